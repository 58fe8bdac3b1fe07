"""Inputs and fp64 references for the serving operators (decode, gather_kv, merge_states).

The references work on the e4m3 values and descales as they lie in the cache.  Tolerances:

* decode, O (bf16).  The stored result is off by half a bf16 step, 2^-8 |O|.  Each probability is
  rounded to fp16 (2^-11 relative) and each score carries at most (128 + 4) fp32 roundings of
  the terms |q_d k_d| it sums, so with S the largest sum of |q_d k_d| * |softmax_scale| of the
  row a score is off by D = 132 * 2^-24 * S and a probability by D relative, numerator and
  denominator alike; the fp32 sums over n tokens and their split add at most n * 2^-24 of the
  terms' magnitudes.  With A = sum_j p_j |v_j| / l that bounds the error by
  2^-8 |O| + (2^-11 + 2 D + 2 n 2^-24 + 2^-20) A.
* decode, LSE.  D + (n + 4) 2^-24 + 2^-22 |LSE| + 2^-20 (approximate exponentials, the logarithm).
* merge.  fp32 weights: exp of a difference of LSEs, off by 2^-23 |difference| + 2^-22 relative,
  where weights of differences beyond 100 vanish: 2^-8 |O| + 2^-15 A; LSE 2^-22 |LSE| + 2^-15.
* gather_kv is exact: one fp32 product, rounded to nearest.
"""
from __future__ import annotations

import numpy as np
import torch

NEG_FLT_MAX = float(np.finfo(np.float32).min)
TILE = 128


def e4m3_values():
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    x = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8.0) * 2.0 ** (e - 7.0))
    x = np.where((c & 127) == 127, np.nan, x)
    return np.where(c & 128, -x, x)


VAL = e4m3_values()


def finite_codes(rng, shape, spread=1.0):
    """Codes of normal values (numpy's rounding does not matter: any finite code will do)."""
    x = torch.from_numpy((rng.standard_normal(shape) * spread * 60).astype(np.float32))
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


class Cache:
    """A paged cache on the host: logical K/V codes of each sequence, pages in shuffled order,
    everything that no sequence uses filled with NaN codes and NaN descales."""

    def __init__(self, seed, lens, N2, ps, k_tok=True, v_head=True, nhd=False, spread=1.0,
                 spare_cols=1):
        rng = np.random.default_rng(seed)
        self.lens, self.N2, self.ps, self.nhd = list(lens), N2, ps, nhd
        self.k_tok, self.v_head = k_tok, v_head
        per = [-(-n // ps) for n in lens]
        self.L = max(per + [0]) + spare_cols
        self.P = sum(per) + 2
        perm = rng.permutation(self.P)
        self.table = np.full((len(lens), self.L), 0x7fffffff, dtype=np.int32)  # never looked up
        self.k = [finite_codes(rng, (N2, n, 128), spread) for n in lens]
        self.v = [finite_codes(rng, (N2, n, 128)) for n in lens]
        self.kd = [np.exp(rng.uniform(-5.5, -4.5, (N2, n))).astype(np.float32) for n in lens]
        self.k_one = np.array([0.0123], dtype=np.float32)
        self.vd = rng.uniform(0.005, 0.02, N2 if v_head else 1).astype(np.float32)
        kp = np.full((self.P, N2, ps, 128), 0x7f, dtype=np.uint8)
        vp = np.full((self.P, N2, ps, 128), 0xff, dtype=np.uint8)
        kd = np.full((self.P, N2, ps), np.nan, dtype=np.float32)
        at = 0
        for b, n in enumerate(lens):
            for i in range(per[b]):
                pg = perm[at]
                at += 1
                self.table[b, i] = pg
                m = min(ps, n - i * ps)
                kp[pg, :, :m] = self.k[b][:, i * ps:i * ps + m]
                vp[pg, :, :m] = self.v[b][:, i * ps:i * ps + m]
                kd[pg, :, :m] = self.kd[b][:, i * ps:i * ps + m]
        if nhd:
            kp, vp = kp.transpose(0, 2, 1, 3), vp.transpose(0, 2, 1, 3)
        self.k_pages, self.v_pages, self.kd_pages = (np.ascontiguousarray(kp),
                                                     np.ascontiguousarray(vp), kd)

    def device(self):
        import block_sparse_fp8_gb300 as bsa

        t = lambda a: torch.from_numpy(a).cuda()
        return dict(
            k_pages=t(self.k_pages), v_pages=t(self.v_pages),
            k_descale=t(self.kd_pages if self.k_tok else self.k_one), v_descale=t(self.vd),
            seqused_kv=t(np.array(self.lens, dtype=np.int32)), block_table=t(self.table),
            kinds=dict(kv_layout=bsa.KV_NHD if self.nhd else bsa.KV_HND,
                       k_scale_kind=bsa.SCALE_PER_TOKEN_HEAD if self.k_tok
                       else bsa.SCALE_PER_TENSOR,
                       v_scale_kind=bsa.SCALE_PER_HEAD if self.v_head else bsa.SCALE_PER_TENSOR))

    def rows(self, b):
        """fp64 K and V [N2, n, 128] of sequence b."""
        kd = self.kd[b].astype(np.float64) if self.k_tok else np.full(
            self.kd[b].shape, float(self.k_one[0]))
        vd = np.broadcast_to(self.vd.astype(np.float64), self.N2)
        return VAL[self.k[b]] * kd[..., None], VAL[self.v[b]] * vd[:, None, None]


def queries(seed, B, N1, q8, scale=1.0):
    """(device-ready q, q_descale or None, fp64 values)."""
    rng = np.random.default_rng(seed)
    if q8:
        c = finite_codes(rng, (B, N1, 128))
        d = (np.exp(rng.uniform(-5, -4, (B, N1))) * scale).astype(np.float32)
        return torch.from_numpy(c), torch.from_numpy(d), VAL[c] * d.astype(np.float64)[..., None]
    q = torch.from_numpy((rng.standard_normal((B, N1, 128)) * scale).astype(np.float32))
    q = q.to(torch.bfloat16)
    return q, None, q.double().numpy()


def reference(cache, q, enabled=None, scale=1.0 / np.sqrt(128.0), N1=None):
    """fp64 decode.  enabled: bool [B, N1, Kb] or None.  Returns O, LSE and their error bounds."""
    B, N1, _ = q.shape
    G = N1 // cache.N2
    O, E = np.zeros((B, N1, 128)), np.zeros((B, N1, 128))
    Z, F = np.full((N1, B), NEG_FLT_MAX), np.zeros((N1, B))
    for b, n in enumerate(cache.lens):
        k, v = cache.rows(b)
        for h in range(N1):
            on = np.ones(n, dtype=bool)
            if enabled is not None:
                on = np.repeat(enabled[b, h], TILE)[:n]
            if not on.any():
                continue
            kk, vv = k[h // G][on], v[h // G][on]
            s = kk @ q[b, h] * scale
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            O[b, h] = p @ vv / l
            A = p @ np.abs(vv) / l
            S = (np.abs(kk) @ np.abs(q[b, h])).max() * abs(scale)
            D = 132 * 2.0 ** -24 * S
            E[b, h] = 2.0 ** -8 * np.abs(O[b, h]) + (2.0 ** -11 + 2 * D + 2 * n * 2.0 ** -24 +
                                                     2.0 ** -20) * A
            Z[h, b] = m + np.log(l)
            F[h, b] = D + (n + 4) * 2.0 ** -24 + 2.0 ** -22 * abs(Z[h, b]) + 2.0 ** -20
    return O, Z, E, F


def within(got, ref, bound, what):
    """|got - ref| <= bound everywhere; where the reference is NaN (a NaN among the values that
    take part) the result has to be NaN too."""
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, f"{what}: shape {got.shape}, expected {ref.shape}"
    bad = ~((np.abs(got - ref) <= bound) | (np.isnan(got) & np.isnan(ref)))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; first at {i}: got "
                             f"{got[i]}, expected {ref[i]}, bound {bound[i]}")


def index_lists(enabled, rng):
    """bool [B, N1, Kb] -> shuffled index lists with a repeated entry where there is room."""
    B, N1, Kb = enabled.shape
    idx = np.full((B, N1, Kb), -7, dtype=np.int32)     # past a list's length: never read
    cnt = np.zeros((B, N1), dtype=np.int32)
    for b in range(B):
        for h in range(N1):
            t = rng.permutation(np.flatnonzero(enabled[b, h]))
            if 0 < len(t) < Kb:
                t = np.append(t, t[0])
            idx[b, h, :len(t)] = t
            cnt[b, h] = len(t)
    return idx, cnt
