"""Inputs and references for what runs around attention: rotary positions, page tables and the 4-bit
cache.  Bounds:

* rope.  The fixed-point phase is cut to 32 bits (2^-32 turns) and rounded to fp32 (half a turn at
  most: 2^-25 turns), together below 2^-22 radians; the sine and cosine are off by 2^-22 more, and the
  amplitude, the two products and their sum round once each: 2^-20 * amplitude * (|x| + |y|) in all.
  bf16 adds half a step, 2^-8 of the result.
* rope_quantize.  descale: the largest turned value is off by that bound, the division rounds.  A code
  is the nearest e4m3 value to the quotient, but for quotients nearer to a border than the bound.
* append_kv_fp4 is exact: codes and scales equal.  gather_kv_fp4 is exact: one fp32 product, rounded.
* decode_fp4: the bounds of serving_helpers.reference (the 4-bit values are exact in fp16, a weight is
  rounded to fp16 once), and what a block of zeros lets one see: a weight goes into its product as
  2^15 times itself, where fp16's smallest step is 2^-24, so that each weight may be off by 2^-40 of
  its warp's largest whatever its own size, 2^-40 sum_j |v_j| / l in all, with l >= 1 in units of the
  largest.  (Where a dimension's largest weights meet zeros, that is what remains.)
"""
from __future__ import annotations

import numpy as np
import torch

import serving_helpers as S

LEVEL = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6] + [-0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def unpack4(codes):
    """uint8 [..., 64] -> code numbers [..., 128], the low half of a byte first."""
    return np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 128)


def values4(codes, scales):
    """fp64 [..., 128] of packed codes and scale bytes [..., 8], without the descale."""
    return LEVEL[unpack4(codes)] * np.repeat(S.VAL[scales], 16, -1)


def nearest(x, values):
    """Index of the nearest of ascending `values` to x >= 0, the even index in a tie."""
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    a, b = x - values[lo], values[hi] - x
    return np.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def quantise4(x, g):
    """fp64 rows [..., 128] under descales g (broadcast over [..., 1]) -> codes [..., 64], scales
    [..., 8], from the definition.  fp64 decides exactly: values have 8 bits, a scale times a descale
    28, so a quotient is a border or off it by 2^-36 at least."""
    b = x.reshape(*x.shape[:-1], 8, 16)
    g = np.asarray(g, dtype=np.float64)
    s = nearest(np.abs(b).max(-1) / (6 * g), S.VAL[:127]).astype(np.uint8)
    d = (S.VAL[s] * g)[..., None]
    y = np.where(d > 0, np.abs(b) / np.where(d > 0, d, 1), 0)
    c = nearest(y, LEVEL[:8]).astype(np.uint8)
    c = (c | np.where((b < 0), 8, 0).astype(np.uint8)).reshape(x.shape)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


class Cache4(S.Cache):
    """A 4-bit paged cache on the host; everything that no sequence uses has NaN scales."""

    def __init__(self, seed, lens, N2, ps, head=True, nhd=False, spare_cols=1):
        rng = np.random.default_rng(seed)
        self.lens, self.N2, self.ps, self.nhd, self.head = list(lens), N2, ps, nhd, head
        per = [-(-n // ps) for n in lens]
        self.L = max(per + [0]) + spare_cols
        self.P = sum(per) + 2
        perm = rng.permutation(self.P)
        self.table = np.full((len(lens), self.L), 0x7fffffff, dtype=np.int32)
        n_desc = N2 if head else 1
        self.kd = rng.uniform(0.02, 0.03, n_desc).astype(np.float32)
        self.vd = rng.uniform(0.005, 0.02, n_desc).astype(np.float32)
        self.codes, self.scales, pages, scs = {}, {}, {}, {}
        for w, top in (("k", 0x40), ("v", 0x48)):
            self.codes[w] = [rng.integers(0, 256, (N2, n, 64), dtype=np.uint8) for n in lens]
            # scales from subnormal to some ones
            self.scales[w] = [rng.integers(0, top, (N2, n, 8), dtype=np.uint8) for n in lens]
            pages[w] = rng.integers(0, 256, (self.P, N2, ps, 64), dtype=np.uint8)
            scs[w] = np.full((self.P, N2, ps, 8), 0x7f, dtype=np.uint8)
        at = 0
        for b, n in enumerate(lens):
            for i in range(per[b]):
                pg = perm[at]
                at += 1
                self.table[b, i] = pg
                m = min(ps, n - i * ps)
                for w in "kv":
                    pages[w][pg, :, :m] = self.codes[w][b][:, i * ps:i * ps + m]
                    scs[w][pg, :, :m] = self.scales[w][b][:, i * ps:i * ps + m]
        if nhd:
            pages = {w: pages[w].transpose(0, 2, 1, 3) for w in "kv"}
        self.k_pages, self.v_pages = (np.ascontiguousarray(pages[w]) for w in "kv")
        self.k_scales, self.v_scales = scs["k"], scs["v"]

    def device(self):
        import block_sparse_fp8_gb300 as bsa

        t = lambda a: torch.from_numpy(a).cuda()
        kind = bsa.SCALE_PER_HEAD if self.head else bsa.SCALE_PER_TENSOR
        return dict(
            k_pages=t(self.k_pages), v_pages=t(self.v_pages), k_scales=t(self.k_scales),
            v_scales=t(self.v_scales), k_descale=t(self.kd), v_descale=t(self.vd),
            seqused_kv=t(np.array(self.lens, dtype=np.int32)), block_table=t(self.table),
            kinds=dict(kv_layout=bsa.KV_NHD if self.nhd else bsa.KV_HND, k_scale_kind=kind,
                       v_scale_kind=kind))

    def rows(self, b):
        out = []
        for w, d in (("k", self.kd), ("v", self.vd)):
            d = np.broadcast_to(d.astype(np.float64), self.N2)
            out.append(values4(self.codes[w][b], self.scales[w][b]) * d[:, None, None])
        return out


def reference4(cache, q, enabled=None, **kw):
    """serving_helpers.reference with the weights' absolute rounding in the bound of O."""
    O, Z, E, F = S.reference(cache, q, enabled, **kw)
    G = q.shape[1] // cache.N2
    for b, n in enumerate(cache.lens):
        if n:
            E[b] += 2.0 ** -40 * np.repeat(np.abs(cache.rows(b)[1]).sum(1), G, 0)
    return O, Z, E, F


def turned(x, positions, freqs, layout, amplitude):
    """fp64 rows [T, N, 128] rotated by positions [T] and fixed-point freqs uint64 [R/2], and the
    bound of the error before the last rounding."""
    R = 2 * len(freqs)
    with np.errstate(over="ignore"):
        phase = positions.astype(np.int64).astype(np.uint64)[:, None] * freqs.astype(np.uint64)
    a = phase.astype(np.int64).astype(np.float64) * 2.0 ** -64 * 2 * np.pi
    c, s = (np.cos(a) * amplitude)[:, None], (np.sin(a) * amplitude)[:, None]
    y, e = x.astype(np.float64).copy(), np.zeros(x.shape)
    i = (slice(0, R, 2), slice(1, R, 2)) if layout else (slice(0, R // 2), slice(R // 2, R))
    u, v = y[..., i[0]].copy(), y[..., i[1]].copy()
    y[..., i[0]], y[..., i[1]] = u * c - v * s, v * c + u * s
    for j in i:
        e[..., j] = 2.0 ** -20 * abs(amplitude) * (np.abs(u) + np.abs(v))
    return y, e


def assigned(new, old, table, free, count, ps, total):
    """assign_pages, one sequence after another: (cu, used, positions, slots, table, count, status)."""
    B, L = table.shape
    P = len(free)
    table = table.copy()
    cu, used = np.zeros(B + 1, np.int64), np.zeros(B, np.int64)
    positions, slots = np.zeros(total, np.int64), np.full(total, -1, np.int64)
    row = wanted = taken = status = 0
    for b in range(B):
        n, c = max(int(new[b]), 0), int(old[b])
        good = new[b] >= 0 and c >= 0 and c + int(new[b]) <= L * ps
        want = -(-(c + n) // ps) - -(-c // ps) if good else 0
        wanted += want
        good = good and row + n <= total
        some = want == 0 or wanted <= count
        if not good:
            status |= 4
        elif not some:
            status |= 16
        served = good and some
        if served and want:
            for k in range(want):
                page = free[count - 1 - (wanted - want + k)]
                if not 0 <= page < P:
                    status |= 2
                table[b, -(-c // ps) + k] = page
            taken = wanted
        used[b] = c + n if served else max(c, 0)
        for i in range(n):
            if row + i < total:
                positions[row + i] = c + i
                if served:
                    page = table[b, (c + i) // ps]
                    if 0 <= page < P:
                        slots[row + i] = page * ps + (c + i) % ps
                    else:
                        status |= 2
        row += n
        cu[b + 1] = min(row, total)
    return cu, used, positions, slots, table, count - taken, status


def released(lens, keep, table, free, count, ps):
    """release_pages: (lens, free, count, status)."""
    P, L = len(free), table.shape[1]
    free, out, given, status = free.copy(), np.array(lens).copy(), [], 0
    for b in range(len(lens)):
        n = int(lens[b])
        if n < 0 or n > L * ps:
            status |= 4
            continue
        k = min(max(int(keep[b]), 0), n)
        out[b] = k
        for col in range(-(-k // ps), -(-n // ps)):
            page = int(table[b, col])
            if not 0 <= page < P:
                status |= 2
                page = -1
            given.append(page)
    if count + len(given) > P:
        status |= 2
    for j, page in enumerate(given):
        at = count + len(given) - 1 - j
        if at < P:
            free[at] = page
    return out, free, min(count + len(given), P), status
