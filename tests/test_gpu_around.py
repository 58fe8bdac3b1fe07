"""Rotary positions, page tables and the 4-bit cache on the GPU against references (bounds and their
derivation: around_helpers.py, serving_helpers.py)."""
import numpy as np
import pytest
import torch

import around_helpers as A
import serving_helpers as S
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def _bf16(rng, shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(
        torch.bfloat16)


def _slice_of(x, extra, at, fill=float("nan")):
    """x [T, N, 128] as a slice of a wider tensor whose other columns hold NaN; (slice, whole)."""
    T, N, D = x.shape
    wide = torch.full((T, N + extra, D), fill, dtype=x.dtype, device="cuda")
    wide[:, at:at + N] = x.cuda()
    return wide[:, at:at + N], wide


def _i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


# ---------------------------------------------------------------------------------------------
# rope
# ---------------------------------------------------------------------------------------------

FAR = [0, 1, -1, 7, 4095, 131071, 500000, 2 ** 31 - 1, -2 ** 31, 12345678]


def _freqs(R, **kw):
    import block_sparse_fp8_gb300 as bsa

    f = bsa.rope_frequencies(R, **kw)
    return f.cuda(), f.numpy().view(np.uint64)


ROPE = [
    # T, N1, N2, R, layout, amplitude
    (1, 1, 0, 128, 0, 1.0),
    (1, 8, 1, 128, 1, 1.0),
    (3, 5, 2, 64, 0, 1.25),
    (7, 9, 3, 96, 0, 1.0),
    (10, 4, 4, 16, 1, 0.5),
    (10, 1, 1, 16, 0, -1.0),
    (33, 32, 8, 80, 1, 1.0),
    (129, 12, 4, 112, 0, 1.0),
    (1000, 64, 8, 128, 0, 1.1),
    (2049, 7, 1, 32, 1, 1.0),
    (6001, 32, 8, 128, 1, 1.0),
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,N1,N2,R,layout,amplitude", ROPE)
def test_rope(T, N1, N2, R, layout, amplitude, wide):
    import block_sparse_fp8_gb300 as bsa

    rng = np.random.default_rng(T + R)
    q, k = _bf16(rng, (T, N1, 128)), _bf16(rng, (T, N2, 128)) if N2 else None
    pos = np.resize(np.array(FAR), T).astype(np.int64)
    pos[len(FAR):] = rng.integers(0, 1 << 20, max(0, T - len(FAR)))
    fd, f = _freqs(R, base=10000.0)
    if wide:
        qd, _ = _slice_of(q, 3, 1)
        kd = _slice_of(k, 2, 0)[0] if N2 else None
        out, out_all = _slice_of(torch.zeros_like(q), 2, 2, fill=5.0)
    else:
        qd, kd, out = q.cuda(), k.cuda() if N2 else None, None
    got = bsa.rope(qd, _i32(pos), fd, k=kd, layout=layout, amplitude=amplitude, out=out)
    torch.cuda.synchronize()
    for x, y in ((q, got[0]), (k, got[1])):
        if x is None:
            assert y is None
            continue
        ref, e = A.turned(x.double().numpy(), pos, f, layout, np.float64(np.float32(amplitude)))
        S.within(y, ref, e + 2.0 ** -8 * np.abs(ref), "rope")
        assert torch.equal(y[..., R:].cpu(), x[..., R:])         # the rest is copied
    if wide:
        assert (out_all[:, :2] == 5).all()
    # where they lie: the same bits
    again = bsa.rope(qd, _i32(pos), fd, k=kd, layout=layout, amplitude=amplitude, out=qd, k_out=kd)
    assert torch.equal(again[0], got[0]) and (k is None or torch.equal(again[1], got[1]))


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("T,N1,N2,R,layout,amplitude", ROPE)
def test_rope_quantize(T, N1, N2, R, layout, amplitude, rule):
    import block_sparse_fp8_gb300 as bsa

    rng = np.random.default_rng(T + R + 1)
    x = _bf16(rng, (T, N1, 128), 3.0)
    x[0, 0] = 0                                             # a zero row: descale 1, zero codes
    pos = np.resize(np.array(FAR), T).astype(np.int64)
    fd, f = _freqs(R, base=500000.0)
    qd, _ = _slice_of(x, 1, 0)
    codes, d = bsa.rope_quantize(qd, _i32(pos), fd, layout=layout, amplitude=amplitude, rule=rule)
    codes, d = codes.cpu().numpy(), d.double().cpu().numpy()
    ref, e = A.turned(x.double().numpy(), pos, f, layout, np.float64(np.float32(amplitude)))
    top, err = np.abs(ref).max(-1) / 448, e.max(-1) / 448
    assert d[0, 0] == 1 and (codes[0, 0] & 127 == 0).all()
    top[0, 0], err[0, 0] = 1, 0
    if rule:
        assert (np.frexp(d)[0] == 0.5).all()
        assert (d >= top - err).all() and (d < 2 * (top + err) * (1 + 2.0 ** -23)).all()
    else:
        assert (np.abs(d - top) <= err + 2.0 ** -23 * top).all()
    y = ref / d[..., None]
    v = np.abs(S.VAL[codes])
    assert np.isfinite(v).all()
    best = S.VAL[:127][A.nearest(np.minimum(np.abs(y), 448), S.VAL[:127])]
    slack = e / d[..., None] + 2.0 ** -22 * np.abs(y)
    assert (np.abs(np.abs(y) - v) <= np.abs(np.abs(y) - best) + 2 * slack).all()
    assert (np.signbit(S.VAL[codes]) == np.signbit(y))[(v > 0) & (np.abs(y) > slack)].all()


def test_rope_agrees_with_quantize_rows():
    """rope_quantize at position 0 is quantize_rows, bit for bit."""
    import block_sparse_fp8_gb300 as bsa

    x = _bf16(np.random.default_rng(4), (70, 6, 128), 2.0).cuda()
    fd, _ = _freqs(128)
    for rule in (bsa.DESCALE_AMAX, bsa.DESCALE_UE8M0):
        a = bsa.rope_quantize(x, torch.zeros(70, dtype=torch.int32, device="cuda"), fd, rule=rule)
        b = bsa.quantize_rows(x, rule=rule)
        assert torch.equal(a[1], b[1]) and torch.equal(a[0] & 127, b[0] & 127)


def test_rope_does_not_spread_nan():
    """A NaN or an infinity in one row leaves the others as they are."""
    import block_sparse_fp8_gb300 as bsa

    x = _bf16(np.random.default_rng(5), (40, 8, 128)).cuda()
    bad = x.clone()
    bad[3, 2, 5], bad[30, 7, 127] = float("nan"), float("inf")
    pos, (fd, _) = _i32(np.arange(40)), _freqs(128)
    a, b = bsa.rope(x, pos, fd)[0], bsa.rope(bad, pos, fd)[0]
    hit = torch.zeros(40, 8, dtype=torch.bool, device="cuda")
    hit[3, 2] = hit[30, 7] = True
    assert torch.equal(a[~hit], b[~hit]) and not torch.isfinite(b[3, 2, 5])


def test_rope_side_by_side():
    """Outputs between the rows of the inputs, in the same wide tensor, are no overlap."""
    import block_sparse_fp8_gb300 as bsa

    x = _bf16(np.random.default_rng(6), (20, 3, 128))
    wide = torch.zeros(20, 9, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:4] = x.cuda()
    pos, (fd, _) = _i32(np.arange(20) * 77), _freqs(64)
    a, ka = bsa.rope(x.cuda(), pos, fd, k=x[:, :2].contiguous().cuda())
    b, kb = bsa.rope(wide[:, 1:4], pos, fd, k=wide[:, 1:3], out=wide[:, 4:7], k_out=wide[:, 7:])
    assert torch.equal(a, b) and torch.equal(ka, kb) and torch.equal(wide[:, 1:4].cpu(), x)
    for bad in (dict(out=wide[:, 3:6]), dict(out=wide[:, :3])):
        with pytest.raises(bsa.BsaError):
            bsa.rope(wide[:, 1:4], pos, fd, **bad)


def test_rope_far_apart_rows():
    """Rows whose places pass 32 bits."""
    import block_sparse_fp8_gb300 as bsa

    T, far = 3, (1 << 31) - 8
    x = _bf16(np.random.default_rng(7), (T, 2, 128)).cuda()
    store = torch.empty((T - 1) * far + 256, dtype=torch.bfloat16, device="cuda")
    q = store.as_strided((T, 2, 128), (far, 128, 1))
    q.copy_(x)
    pos, (fd, _) = _i32([5, 6, 700]), _freqs(128)
    a, _ = bsa.rope(x, pos, fd)
    c = bsa.rope_quantize(q, pos, fd)
    bsa.rope(q, pos, fd, out=q)
    assert torch.equal(q, a)
    d = bsa.rope_quantize(x, pos, fd)
    assert torch.equal(c[0], d[0]) and torch.equal(c[1], d[1])


# ---------------------------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------------------------

def _pages_case(seed, B, ps, hi, old_hi, short=0, spare=5, L=None):
    rng = np.random.default_rng(seed)
    new = rng.integers(0, hi + 1, B)
    old = rng.integers(0, old_hi + 1, B)
    held, need = -(-old // ps), -(-(old + new) // ps)
    L = L or max(int(need.max()) if B else 0, 1) + 1
    P = int(need.sum()) + spare
    perm = rng.permutation(P)
    table = rng.integers(-5, 0, (B, L)).astype(np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    count = P - at
    free = np.full(P, -9, dtype=np.int32)
    free[:count] = perm[at:]
    return new, old, table, free, max(count - short, 0)


def _assign(new, old, table, free, count, ps, total):
    import block_sparse_fp8_gb300 as bsa

    d = dict(table=_i32(table), free=_i32(free), count=_i32([count]))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.full((n,), 77, dtype=torch.int32, device="cuda")
            for n in (len(new) + 1, len(new), total, total)]
    bsa.assign_pages(_i32(new), _i32(old), d["table"], d["free"], d["count"], ps, total, *outs,
                     dev_status=st)
    torch.cuda.synchronize()
    return outs, d, int(st.item())


def _same(got, ref, what):
    got = got.cpu().numpy()
    bad = np.argwhere(got != ref)
    assert got.shape == ref.shape and not len(bad), (what, len(bad), bad[:3], got[tuple(bad[0])],
                                                     ref[tuple(bad[0])])


PAGES = [
    # B, ps, hi, old_hi, total padding
    (1, 32, 1, 0, 0), (1, 64, 1, 64, 3), (1, 32, 5000, 31, 7), (5, 32, 33, 100, 0),
    (17, 64, 0, 200, 4), (300, 32, 1, 500, 9), (1023, 32, 2, 70, 0), (1024, 64, 1, 64, 1),
    (1025, 32, 3, 40, 2), (3000, 32, 1, 33, 5), (2500, 64, 200, 10, 100), (64, 64, 3000, 0, 3),
    (40, 32, 2000, 3000, 0),
]


@pytest.mark.parametrize("B,ps,hi,old_hi,pad", PAGES)
def test_assign_and_release(B, ps, hi, old_hi, pad):
    import block_sparse_fp8_gb300 as bsa

    new, old, table, free, count = _pages_case(B + hi, B, ps, hi, old_hi)
    total = int(new.sum()) + pad
    outs, d, st = _assign(new, old, table, free, count, ps, total)
    cu, used, pos, slots, table2, left, status = A.assigned(new, old, table, free, count, ps, total)
    assert st == status == 0
    for got, ref, what in zip(outs, (cu, used, pos, slots), ("cu", "used", "positions", "slots")):
        _same(got, ref, what)
    _same(d["table"], table2, "table")
    _same(d["free"], free, "free")
    assert int(d["count"]) == left
    # taken back at once: the stack as it was
    left_lens = bsa.release_pages(outs[1], _i32(old), d["table"], d["free"], d["count"], ps)
    _same(left_lens, old, "lens")
    _same(d["free"], free, "free after")
    assert int(d["count"]) == count
    # some kept in part, in place
    rng = np.random.default_rng(B)
    keep = rng.integers(-3, old.max() + 10, B)
    lens = _i32(old)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = A.released(old, keep, table2, free, count, ps)
    bsa.release_pages(lens, _i32(keep), d["table"], d["free"], d["count"], ps, out=lens,
                      dev_status=st)
    _same(lens, ref[0], "lens kept")
    _same(d["free"], ref[1], "free kept")
    assert int(d["count"]) == ref[2] and int(st.item()) == ref[3] == 0


@pytest.mark.parametrize("B,ps,hi,old_hi,short", [
    (1, 32, 100, 10, 50), (8, 64, 500, 100, 20), (2000, 32, 40, 60, 700), (30, 32, 700, 0, 10 ** 6),
    (1100, 32, 1, 64, 7)])
def test_assign_with_too_few_pages(B, ps, hi, old_hi, short):
    new, old, table, free, count = _pages_case(B, B, ps, hi, old_hi, short)
    total = int(new.sum())
    outs, d, st = _assign(new, old, table, free, count, ps, total)
    cu, used, pos, slots, table2, left, status = A.assigned(new, old, table, free, count, ps, total)
    assert st == status == 16
    for got, ref, what in zip(outs, (cu, used, pos, slots), ("cu", "used", "positions", "slots")):
        _same(got, ref, what)
    _same(d["table"], table2, "table")
    assert int(d["count"]) == left


@pytest.mark.parametrize("total_off", [0, -100, 3000])
def test_assign_with_bad_lengths(total_off):
    """Negative lengths, one beyond the table, one at its very end, and too many rows."""
    new, old, table, free, count = _pages_case(3, 40, 32, 60, 100, L=6)
    new[3], old[7], new[11], old[20] = -4, -1, 2 ** 31 - 1, 2 ** 31 - 1
    new[25], old[25] = 192, 0                          # exactly the table's room
    new[26], old[26] = 193, 0
    total = int(np.maximum(new, 0).astype(np.int64)[[i for i in range(40) if i != 11]].sum())
    total = max(0, total + total_off)
    ref = A.assigned(np.where(new > 10 ** 6, 10 ** 6, new), old, table, free, count, 32, total)
    outs, d, st = _assign(new, old, table, free, count, 32, total)
    assert st == ref[6] and st & 4
    for got, r, what in zip(outs, ref, ("cu", "used", "positions", "slots")):
        if what == "positions":                        # of sequences that have one
            ok = ref[3] >= 0
            got, r = got[torch.from_numpy(ok).cuda()], r[ok]
        _same(got, r, what)
    _same(d["table"], ref[4], "table")
    assert int(d["count"]) == ref[5]


def test_assign_and_release_bad_entries():
    """Stack and table entries outside the pool are reported, and their tokens have no slot."""
    import block_sparse_fp8_gb300 as bsa

    new, old, table, free, count = _pages_case(9, 6, 32, 100, 50)
    free[count - 2] = len(free)                        # one past the pool
    held = np.flatnonzero((old % 32 != 0) & (new > 0))
    table[held[0], old[held[0]] // 32] = -1            # a page in use that is none
    total = int(new.sum())
    ref = A.assigned(new, old, table, free, count, 32, total)
    outs, d, st = _assign(new, old, table, free, count, 32, total)
    assert st == ref[6] == 2
    _same(outs[3], ref[3], "slots")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    zero = torch.zeros_like(outs[1])
    ref2 = A.released(ref[1], np.zeros(6), ref[4], free, ref[5], 32)
    bsa.release_pages(outs[1], zero, d["table"], d["free"], d["count"], 32, dev_status=st)
    _same(d["free"], ref2[1], "free")
    assert int(d["count"]) == ref2[2] and int(st.item()) == ref2[3] == 2
    # given back twice: what the stack has no room for is dropped
    before = d["free"].clone()
    bsa.release_pages(outs[1], zero, d["table"], d["free"], d["count"], 32, dev_status=st)
    assert int(d["count"]) == min(len(free), ref2[2] + (ref2[2] - ref[5]))
    assert before.shape == d["free"].shape


def test_assign_and_release_captured():
    """Prompts of many rows, captured: replayed with other lengths, fewer rows and other stacks."""
    import block_sparse_fp8_gb300 as bsa

    B, ps, L, total = 37, 32, 200, 40000
    P = B * L
    rng = np.random.default_rng(17)
    new, old, keep = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    table = torch.full((B, L), -1, dtype=torch.int32, device="cuda")
    free, count = torch.zeros(P, dtype=torch.int32, device="cuda"), _i32([0])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B + 1, B, total, total)]
    left = torch.zeros(B, dtype=torch.int32, device="cuda")

    def both():
        bsa.assign_pages(new, old, table, free, count, ps, total, *outs, dev_status=st)
        bsa.release_pages(outs[1], keep, table, free, count, ps, out=left, dev_status=st)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for hi in (1000, 3, 0, 700):
        n = rng.integers(0, hi + 1, B)
        k = rng.integers(0, n.max() + 2, B)
        stack = rng.permutation(P).astype(np.int32)
        new.copy_(_i32(n)), old.zero_(), keep.copy_(_i32(k)), free.copy_(_i32(stack))
        count.fill_(P)
        graph.replay()
        torch.cuda.synchronize()
        ref = A.assigned(n, np.zeros(B, int), np.full((B, L), -1), stack, P, ps, total)
        for got, want, what in zip(outs, ref, ("cu", "used", "positions", "slots")):
            _same(got, want, what)
        lens, stack2, c2, status = A.released(ref[1], k, ref[4], stack, ref[5], ps)
        _same(left, lens, "left")
        assert int(count) == c2 and int(st.item()) == status == 0
        _same(free[:c2], stack2[:c2], "stack")


def test_assign_nothing():
    """No sequences, or none that gets a token: the padding rows are marked all the same."""
    import block_sparse_fp8_gb300 as bsa

    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    for total in (0, 5, 5000):
        cu, used, pos, slot = bsa.assign_pages(
            e, e, torch.zeros(0, 4, dtype=torch.int32, device="cuda"), _i32([0, 1]), _i32([2]), 32,
            total)
        assert (slot == -1).all() and (pos == 0).all() and slot.numel() == total
        if total:
            assert cu.tolist() == [0]
        count = _i32([2])
        cu, used, pos, slot = bsa.assign_pages(
            _i32([0, 0]), _i32([5, 0]), _i32([[1, -1], [-1, -1]]), _i32([0, 1]), count, 32, total)
        assert cu.tolist() == [0, 0, 0] and used.tolist() == [5, 0] and int(count) == 2
        assert (slot == -1).all() and (pos == 0).all()


# ---------------------------------------------------------------------------------------------
# the 4-bit cache: append and gather
# ---------------------------------------------------------------------------------------------

def _pool4(P, N2, ps, nhd, fill=0xA5):
    shape = (P, ps, N2, 64) if nhd else (P, N2, ps, 64)
    pages = [torch.full(shape, fill, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.full((P, N2, ps, 8), fill, dtype=torch.uint8, device="cuda") for _ in "kv"]
    return pages, scales


def _rows_of(pages, scales, nhd):
    """[P, N2, ps, ...] on the host."""
    p = [x.cpu().numpy() for x in pages]
    return [x.transpose(0, 2, 1, 3) if nhd else x for x in p], [x.cpu().numpy() for x in scales]


def _borders(rng, T, N2, g):
    """bf16 rows whose quotients lie on, or next to, the borders between codes and between scales."""
    x = rng.standard_normal((T, N2, 8, 16))
    top = S.VAL[rng.integers(1, 127, (T, N2, 8, 1))]
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.0, 6.0])
    x = np.where(rng.random(x.shape) < 0.7, mids[rng.integers(0, 9, x.shape)] * np.sign(x), x)
    x[..., 0] = 6
    half = rng.random((T, N2, 8)) < 0.3                # a largest value between two scales
    nxt = S.VAL[np.minimum(np.searchsorted(S.VAL[:127], top[..., 0]) + 1, 126)]
    x = x * top * g.reshape(1, -1, 1, 1)
    x[..., 0] = np.where(half, 3 * (top[..., 0] + nxt) * g.reshape(1, -1, 1), x[..., 0])
    return x.reshape(T, N2, 128)


APPEND = [
    # T, N2, ps, nhd, head, kind of values
    (1, 1, 32, False, True, "normal"), (1, 8, 64, True, True, "normal"),
    (5, 3, 32, True, False, "normal"), (64, 8, 64, False, True, "normal"),
    (77, 1, 64, False, False, "borders"), (100, 5, 32, True, True, "borders"),
    (1000, 2, 32, False, True, "borders"), (40, 4, 64, False, True, "extremes"),
    (513, 8, 32, True, True, "sevenths"), (4097, 8, 64, False, False, "sevenths"),
]


@pytest.mark.parametrize("T,N2,ps,nhd,head,kind", APPEND)
def test_append_and_gather_fp4(T, N2, ps, nhd, head, kind):
    import block_sparse_fp8_gb300 as bsa

    rng = np.random.default_rng(T + N2)
    gk = rng.uniform(0.001, 0.01, N2 if head else 1).astype(np.float32)
    gv = rng.uniform(0.001, 0.01, N2 if head else 1).astype(np.float32)
    if kind == "borders":
        gk = np.exp2(rng.integers(-9, -4, gk.shape)).astype(np.float32)    # exact ties
        x = torch.from_numpy(_borders(rng, T, N2, np.broadcast_to(gk.astype(float), N2)).astype(
            np.float32)).to(torch.bfloat16)
    else:
        x = _bf16(rng, (T, N2, 128), 2.0)
    v = _bf16(rng, (T, N2, 128), 1.5)
    if kind == "sevenths":                              # descales as a largest value gives them
        gk[:] = np.float32(np.float32(x.abs().max().item()) / np.float32(2688))
        gv[:] = np.float32(np.float32(v.abs().max().item()) / np.float32(2688))
    if kind == "extremes":
        x[0] = 0                                        # nothing but zeros
        x[1] *= 2.0 ** -40                              # below the smallest scale
        x[2] *= 1000.0                                  # above the largest
        x[3] = 2.0 ** -30
        x[4], x[5] = torch.finfo(torch.bfloat16).max, -torch.finfo(torch.bfloat16).max
        x[6, :, ::16] = 100.0                           # one of each block stands out
        x[7] = -0.0
        x[8] *= 2.0 ** -9
    P = -(-T // ps) + 3
    slots = rng.permutation(P * ps)[:T].astype(np.int32)
    skip = np.zeros(T, dtype=bool)
    if T > 4:
        skip[[1, T // 2]] = True
        slots[skip] = -1
    pages, scales = _pool4(P, N2, ps, nhd)
    kinds = dict(kv_layout=bsa.KV_NHD if nhd else bsa.KV_HND,
                 k_scale_kind=bsa.SCALE_PER_HEAD if head else bsa.SCALE_PER_TENSOR,
                 v_scale_kind=bsa.SCALE_PER_HEAD if head else bsa.SCALE_PER_TENSOR)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = lambda a: torch.from_numpy(a).cuda()
    bsa.append_kv_fp4(x.cuda(), _slice_of(v, 3, 2)[0], _i32(slots), *pages, *scales, t(gk), t(gv),
                      dev_status=st, **kinds)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    p, s = _rows_of(pages, scales, nhd)
    untouched = np.ones(P * ps, dtype=bool)
    untouched[slots[~skip]] = False
    pg, sl = slots[~skip] // ps, slots[~skip] % ps
    for rows, g, c, e in ((x, gk, p[0], s[0]), (v, gv, p[1], s[1])):
        ref_c, ref_s = A.quantise4(rows.double().numpy()[~skip],
                                   np.broadcast_to(g.astype(np.float64), N2)[:, None])
        got_c, got_s = c[pg, :, sl], e[pg, :, sl]
        assert np.array_equal(got_s, ref_s), np.argwhere(got_s != ref_s)[:3]
        a, b = A.LEVEL[A.unpack4(got_c)], A.LEVEL[A.unpack4(ref_c)]
        assert np.array_equal(a, b), (np.argwhere(a != b)[:3], a[a != b][:3], b[a != b][:3])
        for arr in (c, e):
            flat = arr.transpose(0, 2, 1, 3).reshape(P * ps, -1)
            assert (flat[untouched] == 0xA5).all()
    # and read back, sequence by sequence: runs of consecutive slots
    table = rng.permutation(P).astype(np.int32).reshape(1, P)
    n = P * ps - 5
    cu = np.array([0, n], dtype=np.int32)
    for dtype in (torch.bfloat16, torch.float32):
        for which in ("both", "k", "v"):
            a = [pages[0] if which != "v" else None, pages[1] if which != "k" else None]
            rest = [scales[0] if which != "v" else None, scales[1] if which != "k" else None]
            got = bsa.gather_kv_fp4(*a, *rest, t(gk), t(gv), _i32(cu), _i32(table), n + 2,
                                    cache_starts=_i32([3]), out_dtype=dtype, dev_status=st, **kinds)
            for out, c, e, g, off in ((got[0], p[0], s[0], gk, which == "v"),
                                      (got[1], p[1], s[1], gv, which == "k")):
                if off:
                    assert out is None
                    continue
                at = np.arange(3, 3 + n)
                val = A.values4(c, e)[table[0, at // ps], :, at % ps].astype(np.float32)
                ref = torch.from_numpy(val * np.broadcast_to(g, N2)[:, None]).to(dtype)
                out = out[:n].cpu()
                same = (out == ref) | (torch.isnan(out) & torch.isnan(ref))
                assert same.all()
    assert int(st.item()) == 0


def test_append_fp4_bad_slots():
    """A slot beyond the pool is reported, and nothing is written for it."""
    import block_sparse_fp8_gb300 as bsa

    pages, scales = _pool4(2, 2, 32, False)
    x = _bf16(np.random.default_rng(0), (4, 2, 128)).cuda()
    g = torch.full((1,), 0.001, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.append_kv_fp4(x, x, _i32([64, 2 ** 31 - 1, -1, -2 ** 31]), *pages, *scales, g, g,
                      dev_status=st)
    assert int(st.item()) == bsa.DEV_BAD_PAGE
    assert all((t == 0xA5).all() for t in pages + scales)
    bsa.append_kv_fp4(x, x, _i32([64, 3, -1, 63]), *pages, *scales, g, g)
    assert (pages[0][0, :, 3] != 0xA5).any() and (pages[1][1, :, 31] != 0xA5).any()


def test_gather_fp4_bad_pages_and_rows_behind():
    import block_sparse_fp8_gb300 as bsa

    pages, scales = _pool4(3, 2, 32, False, fill=0x33)
    g = torch.full((2,), 2.0, device="cuda")
    k = torch.full((40, 2, 128), 9.0, device="cuda")
    v = torch.full((40, 2, 128), 9.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.gather_kv_fp4(*pages, *scales, g, g, _i32([0, 33]), _i32([[1, 3]]), 40, k_out=k, v_out=v,
                      dev_status=st)
    assert int(st.item()) == bsa.DEV_BAD_PAGE
    want = 1.5 * S.VAL[0x33] * 2
    assert (k[:32] == want).all() and (k[32] == 0).all() and (k[33:] == 9).all()
    assert (v[:32] == want).all() and (v[32] == 0).all() and (v[33:] == 9).all()


# ---------------------------------------------------------------------------------------------
# decode over it
# ---------------------------------------------------------------------------------------------

def _decode4(cache, q, qd, enabled=None, form="mask", scale=None, dev=None, **kw):
    import block_sparse_fp8_gb300 as bsa

    d = dev or cache.device()
    q, qd = q.cuda(), None if qd is None else qd.cuda()
    B, N1, _ = q.shape
    max_kv = kw.pop("max_kv_len", max(cache.lens + [0]))
    if enabled is not None:
        if form == "mask":
            kw["block_mask"] = torch.from_numpy(enabled.astype(np.uint8) * 3).cuda()
        else:
            idx, cnt = S.index_lists(enabled, np.random.default_rng(3))
            kw["sparse_indices"] = torch.from_numpy(idx).cuda()
            kw["sparse_seq_len"] = torch.from_numpy(cnt).cuda()
    dims = bsa.make_decode_dims(q, d["k_pages"], d["block_table"], max_kv,
                                d["kinds"]["k_scale_kind"], d["kinds"]["v_scale_kind"],
                                d["kinds"]["kv_layout"], sparse=enabled is not None)
    ws = torch.full((bsa.decode_fp4_workspace_size(dims),), 0xff, dtype=torch.uint8, device="cuda")
    out = torch.full((B, N1, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N1, B), float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    expect = kw.pop("status", 0)
    got = bsa.decode_fp4(q, d["k_pages"], d["v_pages"], d["k_scales"], d["v_scales"],
                         d["k_descale"], d["v_descale"], d["seqused_kv"], d["block_table"], max_kv,
                         q_descale=qd, softmax_scale=scale, out=out, lse=lse, dev_status=st,
                         workspace=ws, **d["kinds"], **kw)
    torch.cuda.synchronize()
    assert got[0] is out and got[1] is lse
    assert int(st.item()) == expect
    return out, lse


def _compare(cache, q64, got, enabled=None, what="", scale=None):
    O, Z, E, F = A.reference4(cache, q64, enabled, **({} if scale is None else {"scale": scale}))
    S.within(got[0], O, E, what + " O")
    S.within(got[1], Z, F, what + " LSE")


DENSE = [
    # lens, N1, N2, ps, q8, head, nhd
    ([1], 1, 1, 32, False, True, False),
    ([2, 31], 2, 2, 32, True, True, True),
    ([32, 33, 63, 64, 65], 8, 2, 32, False, True, False),
    ([127, 128, 129], 8, 1, 64, False, False, False),
    ([255, 0, 256, 257, 0], 12, 4, 64, True, False, True),
    ([1000, 1, 517], 7, 1, 32, False, True, True),
    ([300] * 3, 9, 1, 64, False, True, False),
    ([640, 5, 1290], 32, 2, 64, True, True, False),
    ([77], 48, 3, 32, False, True, True),
    ([2048], 5, 5, 64, False, True, False),
    ([200] * 80, 8, 4, 64, True, True, False),
    ([9001, 130], 10, 2, 32, False, True, False),
    ([20000], 16, 1, 64, True, True, True),
]


@pytest.mark.parametrize("lens,N1,N2,ps,q8,head,nhd", DENSE)
def test_decode_fp4_dense(lens, N1, N2, ps, q8, head, nhd):
    cache = A.Cache4(sum(lens) + N1, lens, N2, ps, head, nhd)
    q, qd, q64 = S.queries(N1, len(lens), N1, q8)
    got = _decode4(cache, q, qd)
    _compare(cache, q64, got, what="dense")
    again = _decode4(cache, q, qd)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("form", ["mask", "index"])
@pytest.mark.parametrize("lens,N1,N2,ps,q8,head,nhd", [
    ([700, 130, 0, 1], 8, 2, 32, False, True, False), ([5000, 4000], 16, 1, 64, True, False, True),
    ([1290] * 5, 12, 4, 64, False, True, True), ([9000], 7, 1, 32, True, True, False)])
def test_decode_fp4_sparse(lens, N1, N2, ps, q8, head, nhd, form):
    cache = A.Cache4(sum(lens), lens, N2, ps, head, nhd)
    Kb = -(-max(lens) // 128)
    rng = np.random.default_rng(N1)
    on = rng.random((len(lens), N1, Kb)) < 0.3
    on[0, 0] = False                                   # a head with nothing enabled
    on[-1, :, :] |= rng.random((1, Kb)) < 0.2          # tiles that all heads share
    q, qd, q64 = S.queries(N1, len(lens), N1, q8)
    _compare(cache, q64, _decode4(cache, q, qd, on, form), on, form)


def test_decode_fp4_many_short_sequences():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 300, 301)]
    cache = A.Cache4(11, lens, 2, 32)
    q, qd, q64 = S.queries(12, len(lens), 4, False)
    _compare(cache, q64, _decode4(cache, q, qd), what="many")


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0, 30.0])
def test_decode_fp4_scales(scale):
    """No weight but equal ones, a negative scale, and scores beyond any probability's range."""
    cache = A.Cache4(21, [500, 64, 3], 2, 64)
    q, qd, q64 = S.queries(22, 3, 8, False)
    _compare(cache, q64, _decode4(cache, q, qd, scale=scale), scale=np.float64(np.float32(scale)))


def test_decode_fp4_strided_queries_and_in_place():
    import block_sparse_fp8_gb300 as bsa

    cache = A.Cache4(31, [300, 90, 1], 2, 32)
    q, _, q64 = S.queries(32, 3, 8, False)
    d = cache.device()
    view, _ = _slice_of(q, 5, 2)
    args = (d["k_pages"], d["v_pages"], d["k_scales"], d["v_scales"], d["k_descale"],
            d["v_descale"], d["seqused_kv"], d["block_table"], 300)
    a, la = bsa.decode_fp4(view, *args, **d["kinds"])
    _compare(cache, q64, (a, la))
    own = q.cuda()
    b, none = bsa.decode_fp4(own, *args, out=own, return_lse=False, **d["kinds"])
    assert b is own and none is None and torch.equal(a, b)


def test_decode_fp4_bad_data():
    """Bad pages read as zeros, bad lengths as none; both are reported, nothing else changes."""
    import block_sparse_fp8_gb300 as bsa

    lens = [400, 200, 129]
    cache = A.Cache4(41, lens, 2, 32)
    q, qd, q64 = S.queries(42, 3, 8, False)
    cache.table[0, 2] = cache.P
    cache.table[1, 0] = -1
    for w in "kv":
        cache.codes[w][0][:, 64:96] = 0
        cache.codes[w][1][:, :32] = 0
    _compare(cache, q64, _decode4(cache, q, qd, status=bsa.DEV_BAD_PAGE))
    d = cache.device()
    d["seqused_kv"][0] = 401
    d["seqused_kv"][1] = -1
    got = _decode4(cache, q, qd, dev=d, status=bsa.DEV_BAD_SEQLEN)
    cache.lens = [0, 0, 129]
    _compare(cache, q64, got)


def test_decode_fp4_nan_scale_stays_in_its_heads():
    """A NaN scale of V reaches the heads that enable its tile, and no other."""
    lens = [600]
    cache = A.Cache4(51, lens, 1, 64)
    q, qd, q64 = S.queries(52, 1, 4, False)
    on = np.ones((1, 4, 5), dtype=bool)
    on[0, 1:3, 2] = False
    clean = _decode4(cache, q, qd, on)
    page, slot = cache.table[0, 300 // 64], 300 % 64
    cache.v_scales[page, 0, slot, 3] = 0x7f
    got = _decode4(cache, q, qd, on)
    bad = torch.isnan(got[0]).cpu().numpy()
    assert bad[0, [0, 3]][:, 48:64].all() and bad.sum() == 2 * 16
    assert torch.equal(got[0][:, 1:3], clean[0][:, 1:3]) and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("form", [None, "mask", "index"])
def test_decode_fp4_longest_capacity(form):
    """max_kv_len at the supported limit, as a graph for any length would be captured."""
    cap = 4096 * 128
    lens = [70, 0, 4000]
    cache = A.Cache4(14, lens, 1, 64, spare_cols=0)
    full = np.full((len(lens), cap // 64), 0x7fffffff, dtype=np.int32)
    full[:, :cache.L] = cache.table
    cache.table, cache.L = full, cap // 64
    on = np.random.default_rng(2).random((len(lens), 3, 4096)) < 0.05 if form else None
    q, qd, q64 = S.queries(15, len(lens), 3, False)
    _compare(cache, q64, _decode4(cache, q, qd, on, form, max_kv_len=cap), on, str(form))


def test_decode_fp4_idle_batch():
    """Sequences without a token only, with and without a capacity."""
    cache = A.Cache4(16, [0, 0, 0], 2, 32)
    q, qd, q64 = S.queries(17, 3, 20, True)
    for cap in (0, 32):
        out, lse = _decode4(cache, q, qd, max_kv_len=cap)
        assert (out == 0).all() and (lse == S.NEG_FLT_MAX).all()


def test_fp4_pool_beyond_32_bits():
    """Slots whose bytes lie past 2^32 in the pool, written, read back and decoded over."""
    import block_sparse_fp8_gb300 as bsa

    N2, ps = 8, 64
    P = (1 << 32) // (N2 * ps * 64) + 40
    pages = [torch.empty(P, N2, ps, 64, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.empty(P, N2, ps, 8, dtype=torch.uint8, device="cuda") for _ in "kv"]
    rng = np.random.default_rng(18)
    n = 300
    k, v = _bf16(rng, (n, N2, 128)), _bf16(rng, (n, N2, 128))
    table = (P - 1 - rng.permutation(5)).astype(np.int32).reshape(1, 5)
    at = np.arange(n)
    slots = table[0, at // ps] * ps + at % ps
    g = np.full(N2, 5.0 / 2688, dtype=np.float32)
    gd = torch.from_numpy(g).cuda()
    bsa.append_kv_fp4(k.cuda(), v.cuda(), _i32(slots), *pages, *scales, gd, gd)
    got = bsa.gather_kv_fp4(*pages, *scales, gd, gd, _i32([0, n]), _i32(table), n,
                            out_dtype=torch.float32)
    cache = A.Cache4(1, [0], N2, ps)
    cache.kd = cache.vd = g
    cache.lens = [n]
    for w, x, y in (("k", k, got[0]), ("v", v, got[1])):
        c, e = A.quantise4(x.double().numpy().transpose(1, 0, 2), g.astype(np.float64)[:, None, None])
        cache.codes[w], cache.scales[w] = [c], [e]
        ref = A.values4(c, e).astype(np.float32) * g[:, None, None]
        assert np.array_equal(y.cpu().numpy(), ref.transpose(1, 0, 2))
    q, _, q64 = S.queries(19, 1, 16, False)
    _compare(cache, q64, bsa.decode_fp4(q.cuda(), *pages, *scales, gd, gd, _i32([n]), _i32(table), n))


# ---------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------

def test_calls_on_two_streams_at_once():
    """Every call on a side stream beside the same call on other data on the current one, again and
    again: both come out as they do alone."""
    import block_sparse_fp8_gb300 as bsa

    fd, _ = _freqs(128)
    side = torch.cuda.Stream()

    def data(seed):
        rng = np.random.default_rng(seed)
        lens = [int(x) for x in rng.integers(1, 3000, 6)]
        cache = A.Cache4(seed, lens, 2, 32)
        d = cache.device()
        q, _, _ = S.queries(seed, 6, 16, False)
        n = 500
        x = _bf16(rng, (n, 6, 128)).cuda()
        pages, scales = _pool4(20, 2, 32, False)
        slots = _i32(rng.permutation(20 * 32)[:n])
        new = _i32(rng.integers(0, 900, 6))
        return dict(d=d, q=q.cuda(), x=x, pool=pages + scales, slots=slots, new=new, top=max(lens),
                    pos=_i32(rng.integers(0, 9000, n)), total=int(new.sum()))

    def calls(s, stream):
        d = s["d"]
        o, lse = bsa.decode_fp4(s["q"], d["k_pages"], d["v_pages"], d["k_scales"], d["v_scales"],
                                d["k_descale"], d["v_descale"], d["seqused_kv"], d["block_table"],
                                s["top"], stream=stream, **d["kinds"])
        qr, kr = bsa.rope(s["x"][:, :4], s["pos"], fd, k=s["x"][:, 4:], stream=stream)
        c, e = bsa.rope_quantize(s["x"], s["pos"], fd, stream=stream)
        bsa.append_kv_fp4(kr, s["x"][:, 2:4], s["slots"], *s["pool"], d["k_descale"],
                          d["v_descale"], stream=stream)
        k, v = bsa.gather_kv_fp4(*s["pool"], d["k_descale"], d["v_descale"], s["cu"], s["row"], 640,
                                 stream=stream)
        table, free, count = s["table"].clone(), s["free"].clone(), s["count"].clone()
        outs = bsa.assign_pages(s["new"], s["zero"], table, free, count, 32, s["total"],
                                stream=stream)
        return [o, lse, qr, kr, c, e, k, v, *outs]

    sets = []
    for seed in (81, 82):
        s = data(seed)
        s.update(cu=_i32([0, 640]), row=_i32(np.arange(20).reshape(1, 20)),
                 table=torch.zeros(6, 40, dtype=torch.int32, device="cuda"),
                 free=_i32(np.arange(240)), count=_i32([240]),
                 zero=torch.zeros(6, dtype=torch.int32, device="cuda"))
        sets.append(s)
    alone = [[t.clone() for t in calls(s, None)] for s in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        # what the calls make beside the library's work (clones) is made before the streams part
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b = calls(sets[1], side)
        a = calls(sets[0], None)
        torch.cuda.current_stream().wait_stream(side)
        for got, want in zip(a + b, alone[0] + alone[1]):
            assert torch.equal(got, want)


def test_serving_steps_captured():
    """Prompts admitted, then steps of one token each from one captured graph: pages, rotation,
    append, decode.  Every step against the fp64 attention over what four bits hold."""
    import block_sparse_fp8_gb300 as bsa

    B, N1, N2, ps, L = 5, 8, 2, 32, 12
    P = B * L
    rng = np.random.default_rng(61)
    prompts = np.array([70, 0, 33, 1, 200])
    fd, f = _freqs(128, base=10000.0)
    pages, scales = _pool4(P, N2, ps, False, fill=0x7f)
    g = torch.full((N2,), 5.0 / 2688, device="cuda")
    table = torch.full((B, L), -1, dtype=torch.int32, device="cuda")
    free, count = _i32(rng.permutation(P)), _i32([P])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    history = [[[], []] for _ in range(B)]             # rotated k and v rows as appended

    def place(new, cap, rows):
        """rows [cap, N1 + 2 N2, 128]; returns (rotated q, lengths afterwards)."""
        cu, used, pos, slots = bsa.assign_pages(new, lens, table, free, count, ps, cap,
                                                dev_status=st)
        q, k = bsa.rope(rows[:, :N1], pos, fd, k=rows[:, N1:N1 + N2])
        bsa.append_kv_fp4(k, rows[:, N1 + N2:], slots, *pages, *scales, g, g, dev_status=st)
        lens.copy_(used)
        return q, k, cu, pos

    def remember(k, rows, cu):
        cu = cu.tolist()
        for b in range(B):
            history[b][0].append(k[cu[b]:cu[b + 1]].double().cpu().numpy())
            history[b][1].append(rows[cu[b]:cu[b + 1], N1 + N2:].double().cpu().numpy())

    cap = int(prompts.sum()) + 6
    rows = _bf16(rng, (cap, N1 + 2 * N2, 128)).cuda()
    _, k, cu, pos = place(_i32(prompts), cap, rows)
    remember(k, rows, cu)
    assert pos.tolist()[:70] == list(range(70)) and int(st.item()) == 0

    one = torch.ones(B, dtype=torch.int32, device="cuda")
    step_rows = torch.zeros(B, N1 + 2 * N2, 128, dtype=torch.bfloat16, device="cuda")
    keep = {}

    def step():
        q, k, cu, pos = place(one, B, step_rows)
        # a sequence may sit a step out, so rows are not sequences: the step's own are its first
        out, lse = bsa.decode_fp4(q, *pages, *scales, g, g, lens, table, L * ps, dev_status=st)
        keep.update(q=q, k=k, cu=cu, out=out, lse=lse, pos=pos)

    state = [t.clone() for t in (lens, table, free, count)] + [t.clone() for t in pages + scales]
    step()                                             # warm-up, taken back
    for t, was in zip((lens, table, free, count, *pages, *scales), state):
        t.copy_(was)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, was in zip((lens, table, free, count, *pages, *scales), state):
        t.copy_(was)
    for i in range(35):                                # across a page's end for every sequence
        new = _bf16(rng, (B, N1 + 2 * N2, 128)).cuda()
        step_rows.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        remember(keep["k"], new, keep["cu"])
        if i % 17 and i != 34:
            continue
        cache = A.Cache4(1, [0] * B, N2, ps)           # only its reference is used
        cache.kd = cache.vd = g.cpu().numpy()
        cache.lens = [int(x) for x in lens.tolist()]
        assert cache.lens == [int(p) + i + 1 for p in prompts]
        for w in range(2):
            rows_w = [np.concatenate(h[w]) for h in history]
            both = [A.quantise4(r.transpose(1, 0, 2), cache.kd.astype(np.float64)[:, None, None])
                    for r in rows_w]
            cache.codes["kv"[w]] = [c for c, _ in both]
            cache.scales["kv"[w]] = [s for _, s in both]
        _compare(cache, keep["q"].double().cpu().numpy(), (keep["out"], keep["lse"]), what=f"step {i}")
        # the queries as they were turned
        ref, e = A.turned(new[:, :N1].double().cpu().numpy(),
                          np.array(cache.lens) - 1, f, 0, 1.0)
        S.within(keep["q"], ref, e + 2.0 ** -8 * np.abs(ref), "q")
    assert int(st.item()) == 0
    # everything given back: every page is free again, once
    bsa.release_pages(lens, torch.zeros_like(lens), table, free, count, ps, out=lens)
    assert int(count) == P and sorted(free.tolist()) == list(range(P)) and lens.tolist() == [0] * B


def test_fp4_cache_into_a_prefill():
    """What follows a prompt held in 4 bits: read back, appended to an e4m3 pool, and prefilled over."""
    import block_sparse_fp8_gb300 as bsa

    lens, N2, ps = [150, 64], 2, 32
    cache = A.Cache4(71, lens, N2, ps)
    d = cache.device()
    total, cu = sum(lens), _i32([0, 150, 214])
    k, v = bsa.gather_kv_fp4(d["k_pages"], d["v_pages"], d["k_scales"], d["v_scales"],
                             d["k_descale"], d["v_descale"], cu, d["block_table"], total,
                             **d["kinds"])
    table = _i32(np.arange(10).reshape(2, 5))
    k8 = torch.zeros(10, N2, ps, 128, dtype=torch.uint8, device="cuda")
    v8, kd = torch.zeros_like(k8), torch.zeros(10, N2, ps, device="cuda")
    vs = torch.full((N2,), float(v.abs().max()) / 448, device="cuda")
    bsa.append_kv(k, v, cu, _i32([0, 0]), table, k8, v8, k_descale=kd, v_scale=vs)
    q = _bf16(np.random.default_rng(72), (2, 4, 128)).cuda()
    fd, _ = _freqs(128)
    q8, qd = bsa.rope_quantize(q, _i32([149, 63]), fd)
    out, lse = bsa.prefill(q8, k8, v8, qd, kd, vs, _i32([0, 1, 2]), _i32(lens), table, 1, 150)
    a, la = bsa.decode(q8, k8, v8, kd, vs, _i32(lens), table, 150, q_descale=qd)
    torch.cuda.synchronize()
    # the same rows and queries: the prefill's probabilities are e4m3
    assert torch.allclose(lse, la, rtol=1e-3, atol=1e-3)
    assert (out.float() - a.float()).abs().max() <= 2.0 ** -4 * float(v.abs().max())


# ---------------------------------------------------------------------------------------------
# ends of ranges
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("N1,N2,q8,form", [(8, 2, False, None), (12, 1, False, None),
                                           (4, 1, True, None), (6, 2, False, "mask"),
                                           (16, 1, True, "index")])
@pytest.mark.parametrize("power", [20, 25, 28, 29, 31, 33, 60])
@pytest.mark.parametrize("sign", [1, -1])
def test_decode_fp4_scores_of_any_size(N1, N2, q8, form, power, sign):
    """log2-scores up to 2^power, all above or all below zero: the largest keep their weight.

    Queries are small whole numbers and K's values halves, so the products are exact and two tokens'
    scores are equal or far apart: O is the mean of V over the tokens of the largest score, LSE that
    score plus the logarithm of their number.  O is off by a weight's rounding to fp16, 2^-11, and the
    exponentials', 2^-20, before its own, 2^-8; the LSE by the roundings of the factor (the scale, its
    product with two descales), of the largest score, of two sums and of the product with ln 2 (a
    constant rounded too): 8, 2^-24 each.  What a token t nats below the largest weighs, t >= 14, is off
    by 8 t 2^-24 of it (the factor's roundings), t e^-t 2^-21 < 2^-37.4, and by fp16's smallest step,
    2^-40 of the largest weight: 2^-37 sum_j |v_j| for them all."""
    lens = [500, 64, 3, 1300]
    cache = A.Cache4(power + N1, lens, N2, 32)
    rng = np.random.default_rng(power)
    for b in range(len(lens)):
        cache.codes["k"][b] = rng.integers(0, 256, cache.codes["k"][b].shape, dtype=np.uint8) & 0x77
        cache.scales["k"][b][:] = 0x38                  # one
        for i in range(-(-lens[b] // 32)):
            m = min(32, lens[b] - 32 * i)
            cache.k_pages[cache.table[b, i], :, :m] = cache.codes["k"][b][:, 32 * i:32 * i + m]
            cache.k_scales[cache.table[b, i], :, :m] = 0x38
    q64 = rng.integers(1, 9, (len(lens), N1, 128)).astype(np.float64)
    q, qd = torch.from_numpy(q64).to(torch.bfloat16), None
    if q8:
        qd = torch.from_numpy(rng.uniform(0.5, 2, (len(lens), N1)).astype(np.float32))
        q = torch.from_numpy(q64.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
        q64 = q64 * qd.double().numpy()[..., None]
    scale = float(np.float32(sign * 2.0 ** power / (128 * 8 * 6 * 0.03 * 2)))
    Kb = -(-max(lens) // 128)
    on = np.ones((len(lens), N1, Kb), dtype=bool)
    if form:
        on &= rng.random(on.shape) < 0.6
    got = _decode4(cache, q, qd, on if form else None, form, scale=scale)
    O, Z = np.zeros(q64.shape), np.full((N1, len(lens)), S.NEG_FLT_MAX)
    E, F = np.zeros(q64.shape), np.zeros(Z.shape)
    for b, n in enumerate(lens):
        k, v = cache.rows(b)
        for h in range(N1):
            seen = np.flatnonzero(np.repeat(on[b, h], 128)[:n])
            if not len(seen):
                continue
            # whole halves first: ties are exact
            s = np.rint(2 * (A.values4(cache.codes["k"][b], cache.scales["k"][b])[h * N2 // N1, seen]
                             @ np.rint(q64[b, h] / (1 if qd is None else float(qd[b, h])))))
            unit = 0.5 * float(cache.kd[h * N2 // N1]) * (1 if qd is None else float(qd[b, h])) * scale
            top = (sign * s).max() * sign
            assert abs(unit) > 14
            w = np.exp((s - top) * unit)
            vs = v[h * N2 // N1, seen]
            O[b, h] = (w @ vs) / w.sum()
            E[b, h] = 2.0 ** -8 * np.abs(O[b, h]) + 2.0 ** -37 * np.abs(vs).sum(0) + (
                2.0 ** -11 + 2.0 ** -20) * (w @ np.abs(vs)) / w.sum()
            Z[h, b] = top * unit + np.log(w.sum())
            F[h, b] = 8 * 2.0 ** -24 * abs(Z[h, b]) + 2.0 ** -20
    S.within(got[0], O, E, "O")
    S.within(got[1], Z, F, "LSE")


@pytest.mark.parametrize("g", [2.0 ** -149, 3e-44, 2.0 ** -126, 1e-37, 2.0 ** -122, 1e-36, 7e-32, 3e-20,
                               2.0 ** -60, 0.01, 2.0 ** 60, 4e19, 1e30, 2e37, 1e38, 3.4e38])
def test_append_fp4_with_any_descale(g):
    """Descales from the smallest fp32 number to the largest, blocks below the smallest scale, in the
    middle and above the largest: every code and scale by the definition, and read back exactly."""
    import block_sparse_fp8_gb300 as bsa

    T, N2, ps = 300, 2, 32
    rng = np.random.default_rng(5)
    gg = np.array([g, g], dtype=np.float32)
    gg[1] = np.nextafter(gg[1], np.float32(1))
    top = 2.0 ** rng.uniform(-12, 13, (T, N2, 8, 1)) * 6 * float(gg[0])
    x = rng.uniform(-1, 1, (T, N2, 8, 16)) * top
    x[..., 3] = top[..., 0]
    big = float(torch.finfo(torch.bfloat16).max)
    x = torch.from_numpy(np.clip(x, -big, big).reshape(T, N2, 128)).to(torch.bfloat16)
    x[0], x[1], x[2], x[3] = 1.0, 1e38, -big, 2.0 ** -133
    v = x.flip(0).contiguous()
    P = -(-T // ps)
    pages, scales = _pool4(P, N2, ps, False)
    gd = torch.from_numpy(gg).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.append_kv_fp4(x.cuda(), v.cuda(), _i32(np.arange(T)), *pages, *scales, gd, gd, dev_status=st)
    p, s = _rows_of(pages, scales, False)
    at = np.arange(T)
    for rows, c, e in ((x, p[0], s[0]), (v, p[1], s[1])):
        ref_c, ref_s = A.quantise4(rows.double().numpy(), gg.astype(np.float64)[:, None])
        got_c, got_s = c[at // ps, :, at % ps], e[at // ps, :, at % ps]
        assert np.array_equal(got_s, ref_s), np.argwhere(got_s != ref_s)[:3]
        a, b = A.LEVEL[A.unpack4(got_c)], A.LEVEL[A.unpack4(ref_c)]
        assert np.array_equal(a, b), np.argwhere(a != b)[:3]
    got = bsa.gather_kv_fp4(*pages, *scales, gd, gd, _i32([0, T]), _i32(np.arange(P).reshape(1, P)), T,
                            out_dtype=torch.float32, dev_status=st)
    for out, c, e in zip(got, p, s):
        with np.errstate(over="ignore"):
            ref = A.values4(c, e).astype(np.float32)[at // ps, :, at % ps] * gg[:, None]
        assert np.array_equal(out.cpu().numpy(), ref)
    assert int(st.item()) == 0


def test_assign_pages_without_sequences_writes_the_offset():
    """cu_seqlens has an entry for no sequences too, whatever `total` is, and in a captured call."""
    import block_sparse_fp8_gb300 as bsa

    e, table = torch.zeros(0, dtype=torch.int32, device="cuda"), _i32(np.zeros((0, 4)))
    free, count = _i32([0, 1]), _i32([2])
    for total in (0, 5, 5000):
        cu = _i32([77])
        call = lambda: bsa.assign_pages(e, e, table, free, count, 32, total, cu_seqlens=cu)
        assert call()[0] is cu and cu.tolist() == [0] and count.tolist() == [2]
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            call()
        cu.fill_(77)
        graph.replay()
        assert cu.tolist() == [0]


@pytest.mark.parametrize("B,ps,hi,spare", [(6, 32, 100, 5), (40, 64, 9000, 3), (1500, 32, 70, 9),
                                           (3000, 32, 60, 0), (1, 32, 100000, 2)])
def test_release_of_more_pages_than_the_stack_holds(B, ps, hi, spare):
    """Pages given back twice: the stack is filled to its end, what it has no room for is dropped, and the
    call says so.  Few pages (one CTA) and many (a cluster), lengths out in place of either input."""
    import block_sparse_fp8_gb300 as bsa

    new, old, table, free, count = _pages_case(B + hi, B, ps, hi, 0, spare=spare)
    outs, d, st = _assign(new, old, table, free, count, ps, int(new.sum()))
    ref = A.assigned(new, old, table, free, count, ps, int(new.sum()))
    assert st == 0
    rng = np.random.default_rng(B)
    keep = rng.integers(0, 40, B) * (rng.random(B) < 0.3)
    first = A.released(ref[1], keep, ref[4], free, ref[5], ps)
    again = A.released(ref[1], keep, ref[4], first[1], first[2], ps)
    assert first[3] == 0 and again[3] == bsa.DEV_BAD_PAGE and again[2] == len(free)
    assert (len(free) > 2048) == (B > 6)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = _i32(keep)
    for want, lens, out in ((first, outs[1].clone(), None), (again, outs[1].clone(), k)):
        left = bsa.release_pages(lens, k, d["table"], d["free"], d["count"], ps, out=out,
                                 dev_status=status)
        assert int(status.item()) == want[3] and int(d["count"]) == want[2]
        _same(d["free"], want[1], "free")
        _same(left, want[0], "lens")
        _same(d["table"], ref[4], "table")
        status.zero_()


# ---------------------------------------------------------------------------------------------
# the e4m3 cache behind assign_pages
# ---------------------------------------------------------------------------------------------

class _Pool8:
    """An e4m3 pool, and the bytes that it has to hold."""

    def __init__(self, P, N2, ps, nhd, k_tok=True):
        import block_sparse_fp8_gb300 as bsa

        self.ps, self.nhd, self.k_tok = ps, nhd, k_tok
        shape = (P, ps, N2, 128) if nhd else (P, N2, ps, 128)
        self.k, self.v = (torch.full(shape, 0x55, dtype=torch.uint8, device="cuda") for _ in "kv")
        self.kd = torch.full((P, N2, ps), -7.0, device="cuda")
        self.ks, self.vs = torch.full((1,), 0.02, device="cuda"), torch.linspace(0.02, 0.03, N2).cuda()
        self.kinds = dict(k_scale_kind=bsa.SCALE_PER_TOKEN_HEAD if k_tok else bsa.SCALE_PER_TENSOR,
                          v_scale_kind=bsa.SCALE_PER_HEAD,
                          kv_layout=bsa.KV_NHD if nhd else bsa.KV_HND)
        self.want = [t.clone() for t in (self.k, self.v, self.kd)]

    def append(self, k, v, *where, **kw):
        import block_sparse_fp8_gb300 as bsa

        bsa.append_kv(k, v, *(where or (None,) * 3), self.k, self.v, self.kd, k_scale=self.ks,
                      v_scale=self.vs, **self.kinds, **kw)

    def expect(self, k, v, slots):
        """The rows whose slot is not below zero, by the quantise step's rule."""
        import block_sparse_fp8_gb300 as bsa

        on = torch.from_numpy(np.flatnonzero(slots >= 0)).cuda()
        at = torch.from_numpy(slots[slots >= 0]).cuda()
        pg, sl = at // self.ps, at % self.ps
        e4m3 = lambda x: x.to(torch.float8_e4m3fn).view(torch.uint8)
        codes, d = bsa.quantize_rows(k) if self.k_tok else (e4m3(k.float() / self.ks), None)
        for t, rows in zip(self.want, (codes, e4m3(v.float() / self.vs[:, None]))):
            (t.transpose(1, 2) if self.nhd else t)[pg, :, sl] = rows[on]
        if self.k_tok:
            self.want[2][pg, :, sl] = d[on]

    def check(self, what):
        for got, want, name in zip((self.k, self.v, self.kd), self.want, ("K", "V", "K descales")):
            assert torch.equal(got, want), (what, name, int((got != want).sum()))


@pytest.mark.parametrize("T,N2,ps,nhd,k_tok", [(1, 1, 32, False, True), (77, 5, 32, True, True),
                                               (300, 8, 64, False, False), (1000, 3, 64, True, True)])
def test_append_kv_slots(T, N2, ps, nhd, k_tok):
    """Rows into slots in any order; negative ones skipped, those beyond the pool reported too."""
    import block_sparse_fp8_gb300 as bsa

    rng = np.random.default_rng(T)
    P = -(-T // ps) + 3
    pool = _Pool8(P, N2, ps, nhd, k_tok)
    slots = rng.permutation(P * ps)[:T].astype(np.int32)
    k, v = _bf16(rng, (T, N2, 128)).cuda(), _bf16(rng, (T, N2, 128)).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    skip = slots.copy()
    if T > 4:
        skip[[1, T // 2]] = -1, -2 ** 31
    pool.append(k, v, slot_map=_i32(skip), dev_status=st)
    pool.expect(k, v, skip)
    pool.check("slots")
    assert int(st.item()) == 0
    skip[0] = P * ps
    skip[-1] = 2 ** 31 - 1
    pool.append(v, k, slot_map=_i32(skip), dev_status=st)
    skip[[0, -1]] = -1
    pool.expect(v, k, skip)
    pool.check("beyond the pool")
    assert int(st.item()) == bsa.DEV_BAD_PAGE


@pytest.mark.parametrize("ps,nhd", [(32, False), (64, True)])
def test_pages_for_the_e4m3_cache_captured(ps, nhd):
    """Steps of assign_pages and append_kv from one captured graph, pages given back and assigned to
    others between them: sequences that get no pages, rows behind the last one, sequences that sit out.
    No byte of the pool changes but the served rows'."""
    import block_sparse_fp8_gb300 as bsa

    B, N2, L, P, cap = 6, 2, 8, 14, 200
    rng = np.random.default_rng(ps)
    pool = _Pool8(P, N2, ps, nhd)
    zeros = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    new, lens, st = zeros(B), zeros(B), zeros(1)
    table, free, count = zeros(B, L) - 1, _i32(rng.permutation(P)), _i32([P])
    outs = [zeros(n) for n in (B + 1, B, cap, cap)]
    k, v = (torch.zeros(cap, N2, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")

    def step():
        bsa.assign_pages(new, lens, table, free, count, ps, cap, *outs, dev_status=st)
        pool.append(k, v, slot_map=outs[3], dev_status=st)
        lens.copy_(outs[1])

    step()                                              # nothing to assign: nothing changes
    torch.cuda.synchronize()
    pool.check("warm-up")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    short = 0
    for i in range(40):
        n = rng.integers(0, (40, 2, 90)[i % 3], B) * (rng.random(B) < 0.7)
        state = [t.cpu().numpy() for t in (lens, table, free, count)]
        ref = A.assigned(n, state[0], state[1], state[2], int(state[3][0]), ps, cap)
        new.copy_(_i32(n))
        k.copy_(_bf16(rng, (cap, N2, 128)).cuda())
        v.copy_(_bf16(rng, (cap, N2, 128)).cuda())
        st.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _same(outs[3], ref[3], "slots")
        assert int(st.item()) == ref[6] and ref[6] in (0, 4, 16, 20)
        short += ref[6] >= 16
        pool.expect(k, v, ref[3])
        pool.check(f"step {i}")
        keep = np.where(rng.random(B) < 0.4, rng.integers(0, 60, B), 10 ** 6)
        bsa.release_pages(lens, _i32(keep), table, free, count, ps, out=lens)
    assert short


def test_append_kv_rows_behind_the_last_sequence():
    """Rows from cu_seqlens_new[B] on belong to nobody, whatever the last sequence's table names."""
    rng = np.random.default_rng(7)
    T, B, ps = 120, 2, 32
    pool = _Pool8(8, 2, ps, False)
    k, v = _bf16(rng, (T, 2, 128)).cuda(), _bf16(rng, (T, 2, 128)).cuda()
    table = np.array([[0, 1, 2, 3], [4, 5, 6, 7]])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for cu, cached in (([0, 40, 70], [0, 10]), ([0, 0, 0], [5, 0]), ([0, 33, 33], [40, 128])):
        slots = np.full(T, -1)
        for b in range(B):
            at = cached[b] + np.arange(cu[b + 1] - cu[b])
            slots[cu[b]:cu[b + 1]] = table[b, at // ps] * ps + at % ps
        pool.append(k, v, _i32(cu), _i32(cached), _i32(table), dev_status=st)
        pool.expect(k, v, slots)
        pool.check(str(cu))
        k, v = v, k
    assert int(st.item()) == 0


# ---------------------------------------------------------------------------------------------
# packed queries: a step in which some sequences get no token
# ---------------------------------------------------------------------------------------------

def _decode_any(fp4, d, q, max_kv, **kw):
    """decode() or decode_fp4() over a helper cache's tensors, outputs filled with NaN beforehand."""
    import block_sparse_fp8_gb300 as bsa

    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if kw.get("out") is None:
        kw["out"] = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[1], q.shape[0]), float("nan"), device="cuda")
    kw.update(d["kinds"], lse=lse, dev_status=st)
    if fp4:
        got = bsa.decode_fp4(q, d["k_pages"], d["v_pages"], d["k_scales"], d["v_scales"],
                             d["k_descale"], d["v_descale"], d["seqused_kv"], d["block_table"], max_kv,
                             **kw)
    else:
        got = bsa.decode(q, d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"],
                         d["seqused_kv"], d["block_table"], max_kv, **kw)
    torch.cuda.synchronize()
    return got[0], got[1], int(st.item())


PACKED = [
    # lens, which have a row, rows behind, N1, N2, q8, form
    ([300], [1], 0, 8, 2, False, None),
    ([300], [0], 2, 8, 2, False, None),
    ([300, 7, 40], [1, 0, 1], 0, 8, 2, False, None),
    ([300, 7, 40], [0, 1, 0], 3, 12, 1, True, None),
    ([5000, 0, 129, 2000, 64], [1, 1, 0, 1, 0], 4, 16, 2, True, None),
    ([9000, 1], [0, 1], 1, 6, 2, False, None),
    ([200] * 90, [1, 0, 0] * 30, 50, 8, 4, False, None),
    ([1290, 700, 130, 1], [0, 1, 1, 0], 1, 8, 2, False, "mask"),
    ([1290, 700, 4000, 1], [1, 0, 1, 1], 0, 16, 1, True, "index"),
    ([700, 130, 90], [0, 0, 0], 2, 4, 2, False, "mask"),
]


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("lens,has,behind,N1,N2,q8,form", PACKED)
def test_decode_packed_queries(lens, has, behind, N1, N2, q8, form, fp4):
    """Row for row what decode gives for a row a sequence, those without one counted as empty; the rows
    behind the last sequence's are empty."""
    cache = (A.Cache4 if fp4 else S.Cache)(len(lens) + N1, lens, N2, 32)
    d = cache.device()
    B, max_kv = len(lens), max(lens)
    has = np.array(has)
    cu = np.concatenate([[0], np.cumsum(has)])
    T = int(cu[-1]) + behind
    q, qd, q64 = S.queries(B, max(T, 1), N1, q8)
    q, qd = q[:T].cuda(), None if qd is None else qd[:T].cuda()
    kw = {}
    on = None
    if form:
        on = np.random.default_rng(N1).random((B, N1, -(-max_kv // 128))) < 0.4
        if form == "mask":
            kw["block_mask"] = torch.from_numpy(on.astype(np.uint8)).cuda()
        else:
            idx, cnt = S.index_lists(on, np.random.default_rng(3))
            kw["sparse_indices"], kw["sparse_seq_len"] = (torch.from_numpy(a).cuda() for a in (idx, cnt))
    wide, _ = _slice_of(q, 3, 1) if not q8 else (q, None)
    out, lse, st = _decode_any(fp4, d, wide, max_kv, q_descale=qd, cu_seqlens_q=_i32(cu), **kw)
    assert st == 0
    # a row a sequence
    rows = torch.from_numpy(np.flatnonzero(has)).cuda()
    full = torch.zeros(B, N1, 128, dtype=q.dtype, device="cuda")
    full[rows] = q[:cu[-1]]
    fd = None
    if q8:
        fd = torch.ones(B, N1, device="cuda")
        fd[rows] = qd[:cu[-1]]
    plain = dict(d, seqused_kv=_i32(np.where(has, lens, 0)))
    want, wlse, st = _decode_any(fp4, plain, full, max_kv, q_descale=fd, **kw)
    assert st == 0
    assert torch.equal(out[:cu[-1]], want[rows]) and torch.equal(lse[:, :cu[-1]], wlse[:, rows])
    assert (out[cu[-1]:] == 0).all() and (lse[:, cu[-1]:] == S.NEG_FLT_MAX).all()
    # against the definition
    cache.lens = [n if h else 0 for n, h in zip(lens, has)]
    f64 = np.zeros((B, N1, 128))
    f64[has > 0] = q64[:cu[-1]]
    O, Z, E, F = (A.reference4 if fp4 else S.reference)(cache, f64, on)
    S.within(out[:cu[-1]], O[has > 0], E[has > 0], "O")
    S.within(lse[:, :cu[-1]], Z[:, has > 0], F[:, has > 0], "LSE")
    if not q8:                                          # in place
        own = q.clone()
        again, alse, st = _decode_any(fp4, d, own, max_kv, cu_seqlens_q=_i32(cu), out=own, **kw)
        assert again is own and torch.equal(own, out) and torch.equal(alse, lse) and st == 0


@pytest.mark.parametrize("fp4", [False, True])
def test_decode_packed_bad_rows(fp4):
    """Several rows of a sequence, rows that go back, before the first or beyond the last: reported, empty,
    and the others as they are."""
    import block_sparse_fp8_gb300 as bsa

    lens, N1 = [300, 40, 129, 64], 8
    cache = (A.Cache4 if fp4 else S.Cache)(3, lens, 2, 32)
    d = cache.device()
    q, _, _ = S.queries(4, 6, N1, False)
    q = q.cuda()
    # (rows: whose each is; one that two sequences name is left out)
    for cu, rows in (([0, 1, 3, 4, 5], {0: 0, 3: 2, 4: 3}), ([0, 1, 0, 1, 2], {1: 3}),
                     ([5, 6, 7, 7, 7], {5: 0}), ([-1, 0, 1, 2, 3], {0: 1, 1: 2, 2: 3}),
                     ([2 ** 31 - 1, -2 ** 31, 0, 1, 1], {0: 2}), ([0, 1, 1, 1, 2 ** 31 - 1], {0: 0})):
        out, lse, st = _decode_any(fp4, d, q, 300, cu_seqlens_q=_i32(cu))
        assert st == bsa.DEV_BAD_SEQLEN, cu
        for row, b in rows.items():
            one = torch.zeros(4, N1, 128, dtype=torch.bfloat16, device="cuda")
            one[b] = q[row]
            only = dict(d, seqused_kv=_i32([n if i == b else 0 for i, n in enumerate(lens)]))
            want, wlse, _ = _decode_any(fp4, only, one, 300)
            assert torch.equal(out[row], want[b]) and torch.equal(lse[:, row], wlse[:, b]), cu
        for row in range(max(cu[-1], 0), 6):
            if row not in rows:
                assert (out[row] == 0).all() and (lse[:, row] == S.NEG_FLT_MAX).all(), (cu, row)
    for cu, end in (([0, 1, 3, 4, 5], 3), ([0, 1, 1, 1, 2 ** 31 - 1], 6)):
        out, lse, st = _decode_any(fp4, d, q, 300, cu_seqlens_q=_i32(cu))
        assert (out[1:end] == 0).all() and (lse[:, 1:end] == S.NEG_FLT_MAX).all()


@pytest.mark.parametrize("fp4", [False, True])
def test_decode_packed_nothing(fp4):
    """No sequences: every row is empty; no rows: nothing happens."""
    cache = (A.Cache4 if fp4 else S.Cache)(3, [64], 2, 32)
    d = cache.device()
    q = torch.ones(5, 8, 128, dtype=torch.bfloat16, device="cuda")
    none = dict(d, seqused_kv=d["seqused_kv"][:0], block_table=d["block_table"][:0])
    for T in (5, 1, 0):
        out, lse, st = _decode_any(fp4, none, q[:T], 64, cu_seqlens_q=_i32([0]))
        assert st == 0 and (out == 0).all() and (lse == S.NEG_FLT_MAX).all()
    out, lse, st = _decode_any(fp4, d, q[:0], 64, cu_seqlens_q=_i32([0, 0]))
    assert st == 0 and out.numel() == 0


class _Held:
    """What a cache holds, for the reference: fp64 K and V [N2, n, 128] of each sequence."""

    def __init__(self, N2, rows):
        self.N2, self.held = N2, rows
        self.lens = [r[0].shape[1] for r in rows]

    def rows(self, b):
        return self.held[b]


def test_serving_steps_with_idle_sequences_captured():
    """Steps of a token or none each, whichever sequences sit out, from one captured graph, over the
    4-bit and the e4m3 cache: pages, rotation, append, decode by packed rows.  Every step against the
    fp64 attention over what the caches hold (read back by gather)."""
    import block_sparse_fp8_gb300 as bsa

    B, N1, N2, ps, L = 7, 8, 2, 32, 6
    P = B * L
    rng = np.random.default_rng(91)
    prompts = np.array([70, 0, 33, 1, 150, 64, 5])
    fd, f = _freqs(128)
    pages, scales = _pool4(P, N2, ps, False, fill=0x7f)
    pool = _Pool8(P, N2, ps, True)
    g = torch.full((N2,), 5.0 / 2688, device="cuda")
    zeros = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    table, free, count = zeros(B, L) - 1, _i32(rng.permutation(P)), _i32([P])
    lens, new, st = zeros(B), zeros(B), zeros(1)

    def place(cap, rows):
        cu, used, pos, slots = bsa.assign_pages(new, lens, table, free, count, ps, cap, dev_status=st)
        q, k = bsa.rope(rows[:, :N1], pos, fd, k=rows[:, N1:N1 + N2])
        v = rows[:, N1 + N2:]
        bsa.append_kv_fp4(k, v, slots, *pages, *scales, g, g, dev_status=st)
        pool.append(k, v.contiguous(), slot_map=slots, dev_status=st)
        lens.copy_(used)
        return q, cu, pos

    rows = torch.zeros(B, N1 + 2 * N2, 128, dtype=torch.bfloat16, device="cuda")
    keep = {}

    def step():
        q, cu, pos = place(B, rows)
        a = bsa.decode_fp4(q, *pages, *scales, g, g, lens, table, L * ps, dev_status=st,
                           cu_seqlens_q=cu)
        b = bsa.decode(q, pool.k, pool.v, pool.kd, pool.vs, lens, table, L * ps, dev_status=st,
                       kv_layout=bsa.KV_NHD, cu_seqlens_q=cu)
        keep.update(q=q, cu=cu, pos=pos, fp4=a, e4m3=b)

    new.copy_(_i32(prompts))
    place(int(prompts.sum()) + 3, _bf16(rng, (int(prompts.sum()) + 3, N1 + 2 * N2, 128)).cuda())
    new.zero_()
    step()                                              # nobody gets a token
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    want = prompts.copy()
    for i in range(12):
        n = (rng.random(B) < (0.5, 0.9, 0.2)[i % 3]).astype(int)
        if i == 5:
            n[:] = 0
        want += n
        x = _bf16(rng, (B, N1 + 2 * N2, 128)).cuda()
        rows.copy_(x)
        new.copy_(_i32(n))
        graph.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and lens.tolist() == want.tolist()
        who, T = np.flatnonzero(n), int(n.sum())
        assert keep["cu"].tolist() == [0] + np.cumsum(n).tolist()
        # row r belongs to the r-th sequence with a token, turned at its last position
        ref, e = A.turned(x[:T, :N1].double().cpu().numpy(), want[who] - 1, f, 0, 1.0)
        S.within(keep["q"][:T], ref, e + 2.0 ** -8 * np.abs(ref), "q")
        full = np.zeros((B, N1, 128))
        full[who] = keep["q"][:T].double().cpu().numpy()
        cu = _i32(np.concatenate([[0], np.cumsum(want)]))
        total = int(want.sum())
        for name, kv in (("fp4", bsa.gather_kv_fp4(*pages, *scales, g, g, cu, table, total,
                                                   out_dtype=torch.float32)),
                         ("e4m3", bsa.gather_kv(pool.k, pool.v, pool.kd, pool.vs, cu, table, total,
                                                out_dtype=torch.float32, kv_layout=bsa.KV_NHD))):
            c = cu.tolist()
            kv = [t.double().cpu().numpy().transpose(1, 0, 2) for t in kv]
            held = _Held(N2, [[t[:, c[b]:c[b + 1] if n[b] else c[b]] for t in kv] for b in range(B)])
            O, Z, E, F = (A.reference4 if name == "fp4" else S.reference)(held, full)
            out, lse = keep[name]
            S.within(out[:T], O[who], E[who], f"{name} O {i}")
            S.within(lse[:, :T], Z[:, who], F[:, who], f"{name} LSE {i}")
            assert (out[T:] == 0).all() and (lse[:, T:] == S.NEG_FLT_MAX).all()
