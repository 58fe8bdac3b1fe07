"""decode, gather_kv and merge_states on the GPU: precision of the probabilities, calls on a stream
with memory of their own, mixed batches, and forms in combination (references and bounds that are
not derived here: serving_helpers.py)."""
import numpy as np
import pytest
import torch

import serving_helpers as S
from gpu_helpers import ensure_built
from test_gpu_serving import _compare, _decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


# ---------------------------------------------------------------------------------- precision

def _unit_keys(cache):
    """Every K code +-1 and every K descale 2^-3, in the pages and in the lists."""
    one = lambda c: np.where((c & 0x7f) == 0x7f, c, (c & 0x80) | 0x38).astype(np.uint8)
    cache.k_pages = one(cache.k_pages)
    cache.k = [one(c) for c in cache.k]
    cache.kd_pages = np.where(np.isnan(cache.kd_pages), cache.kd_pages, 0.125).astype(np.float32)
    cache.kd = [np.full_like(d, 0.125) for d in cache.kd]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("lens,N1,N2,form", [
    ([2, 3, 5, 8, 12], 8, 1, None), ([2, 7, 33], 32, 2, None), ([4, 9, 200], 16, 1, "mask"),
    ([3, 6, 140], 8, 1, "index")])
def test_decode_probabilities_keep_their_bits(lens, N1, N2, form, q8):
    """Scores that fp32 holds exactly up to one product: queries and K codes are +-1, so q . k is an
    integer below 2^7, and K's descale is 2^-3.  What is left of a weight's error: the rounding of
    scale * log2(e) and of its product with the integer (|s| log2(e) < 24: 2^-20 each), of the
    reference and of the difference (2^-20 each), 2^-22 of the exponential: together below 2^-18 of
    the weight, 2^-17 of the quotient.  Sums over n tokens add at most n 2^-21 (one fp32 rounding
    and a truncated alignment a term, twice).  With A = sum_j p_j |v_j| / l the result is off by
    2^-8 |O| + (2^-16 + n 2^-21) A, where few tokens of mixed signs make |O| far smaller than A; one
    rounding of the weights to 11 bits is 2^-12 A and stands out."""
    cache = S.Cache(sum(lens) + N1, lens, N2, 32)
    _unit_keys(cache)
    rng = np.random.default_rng(N1)
    sign = rng.choice([-1.0, 1.0], (len(lens), N1, 128))
    if q8:
        q = torch.from_numpy(np.where(sign < 0, 0xb8, 0x38).astype(np.uint8))
        qd = torch.ones(len(lens), N1)
    else:
        q, qd = torch.from_numpy(sign).to(torch.bfloat16), None
    on = None
    if form:
        on = rng.random((len(lens), N1, -(-max(lens) // 128))) < 0.5
        on[:, ::2, 0] = True
    out, lse = _decode(cache, q, qd, on, form or "mask", scale=1.0)
    for b, n in enumerate(lens):
        k, v = cache.rows(b)
        for h in range(N1):
            take = np.ones(n, bool) if on is None else np.repeat(on[b, h], S.TILE)[:n]
            if not take.any():
                assert (out[b, h] == 0).all() and lse[h, b] == S.NEG_FLT_MAX
                continue
            kk, vv = k[h // (N1 // N2)][take], v[h // (N1 // N2)][take]
            s = kk @ sign[b, h]
            p = np.exp(s - s.max())
            O, A = p @ vv / p.sum(), p @ np.abs(vv) / p.sum()
            bound = 2.0 ** -8 * np.abs(O) + (2.0 ** -16 + n * 2.0 ** -21) * A
            S.within(out[b, h], O, bound, f"O of {b}, {h}")
            z = s.max() + np.log(p.sum())
            assert abs(float(lse[h, b]) - z) <= 2.0 ** -16 + n * 2.0 ** -21 + 2.0 ** -22 * abs(z)


# -------------------------------------------------------------------- streams and their memory

def _stream_calls():
    """name -> (call(**kw) on inputs that are ready, check of its result)."""
    import block_sparse_fp8_gb300 as bsa

    cache = S.Cache(3, [3000, 200], 2, 32)
    d = cache.device()
    q, _, q64 = S.queries(4, 2, 8, False)
    q = q.cuda()
    cu = torch.tensor([0, 3000, 3200], dtype=torch.int32, device="cuda")
    rows = [np.concatenate([cache.rows(b)[i].transpose(1, 0, 2) for b in range(2)])
            for i in range(2)]
    g = torch.Generator().manual_seed(5)
    o = [torch.randn(700, 8, 128, generator=g).bfloat16() for _ in range(2)]
    l = [torch.randn(8, 700, generator=g) for _ in range(2)]
    w = torch.softmax(torch.stack(l).double(), 0).transpose(1, 2)[..., None]
    merged = sum(w[i] * o[i].double() for i in range(2)).numpy()
    size = sum(w[i] * o[i].double().abs() for i in range(2)).numpy()
    do, dl = [x.cuda() for x in o], [x.cuda() for x in l]
    x = torch.randn(900, 4, 128, generator=g).bfloat16().cuda()
    codes = tuple(t.cpu() for t in bsa.quantize_rows(x))
    q8, qd = bsa.quantize_rows(torch.randn(300, 8, 128, generator=g).bfloat16().cuda())
    cuq = torch.tensor([0, 200, 300], dtype=torch.int32, device="cuda")
    # the prefill wants zeros in the slots past a sequence's end
    kp, vp = (torch.where(d[n] & 0x7f == 0x7f, 0, d[n]) for n in ("k_pages", "v_pages"))
    kd = d["k_descale"].nan_to_num()

    def prefill(**kw):
        return bsa.prefill(q8, kp, vp, qd, kd, d["v_descale"], cuq, d["seqused_kv"],
                           d["block_table"], 200, 3000, **d["kinds"], **kw)

    ahead = tuple(t.cpu() for t in prefill())

    def same(want):
        def check(got):
            assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))
        return check

    return {
        "decode": (lambda **kw: bsa.decode(
            q, d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"], d["seqused_kv"],
            d["block_table"], 3000, **d["kinds"], **kw),
            lambda got: _compare(cache, q64, got, what="stream")),
        "gather_kv": (lambda **kw: bsa.gather_kv(
            d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"], cu, d["block_table"], 3200,
            out_dtype=torch.float32, **d["kinds"], **kw),
            same([torch.from_numpy(r.astype(np.float32)) for r in rows])),
        "merge_states": (lambda **kw: bsa.merge_states(do, dl, **kw),
                         lambda got: S.within(got[0], merged, 2.0 ** -8 * np.abs(merged) +
                                              2.0 ** -15 * size, "merge")),
        "quantize_rows": (lambda **kw: bsa.quantize_rows(x, **kw), same(codes)),
        "prefill": (prefill, same(ahead)),
    }


STREAM_CALLS = ["decode", "gather_kv", "merge_states", "quantize_rows", "prefill"]


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_call_beside_work_on_freed_memory(name):
    """A call on a stream that does not wait for the current one, where work is still queued on
    memory that has been freed: neither has the other's memory."""
    call, check = _stream_calls()[name]
    sizes = [t.nbytes for t in call()]
    if name == "decode":
        import block_sparse_fp8_gb300 as bsa

        sizes.append(bsa.decode_workspace_size(bsa.DecodeDims(
            2, 8, 2, 128, 32, 3000, 97, 95, 1, 2, 0, 0, 1024, 0)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    kept, freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes], set()
    torch.cuda._sleep(200_000_000)
    for k in kept:
        busy = torch.empty(k.numel(), dtype=torch.uint8, device="cuda")
        freed.add(busy.data_ptr())
        busy.fill_(7)
        k.copy_(busy)
        del busy
    got = call(stream=side)
    assert not freed & {t.data_ptr() for t in got}
    side.synchronize()
    check(got)
    torch.cuda.synchronize()
    check(got)
    assert all((k == 7).all() for k in kept)


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_result_dropped_while_the_current_stream_reads_it(name):
    """A result of another stream, read on the current one and dropped: the other stream's next
    call does not get its memory before that read is done."""
    call, check = _stream_calls()[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)
    copies = [t.clone() for t in got]
    was = {t.data_ptr() for t in got}
    del got
    again = call(stream=side)
    assert not was & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    check(copies)
    check(again)


@pytest.mark.parametrize("name", STREAM_CALLS)
def test_captured_on_a_forked_stream(name):
    """stream= names a stream that a capture has forked; outputs and workspace are the call's own."""
    call, check = _stream_calls()[name]
    call()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(got)


# ------------------------------------------------------------------------------ mixed batches

def test_decode_large_idle_batch():
    """max_kv_len = 0 with more (sequence, KV head) tasks than CTAs: the empty results are shared
    out like those of sequences that could hold a token (the partials' room follows the grid)."""
    import block_sparse_fp8_gb300 as bsa

    cache = S.Cache(20, [0] * 90, 8, 32)
    q, qd, q64 = S.queries(21, 90, 16, False)
    _compare(cache, q64, _decode(cache, q, qd, max_kv_len=0), what="idle")
    none, one = (bsa.decode_workspace_size(bsa.DecodeDims(90, 16, 8, 128, 32, n, 2, 1, 1, 2, 0, 0,
                                                          2048, 0)) for n in (0, 1))
    assert none == one


@pytest.mark.parametrize("form", [None, "mask", "index"])
@pytest.mark.parametrize("lens,N1,N2", [
    ([90] * 200 + [40000] + [70] * 119, 8, 1),             # a partial in about every second run
    ([1, 0, 128] * 55 + [30001], 24, 2),
    ([150] * 60 + [1300] + [150] * 20 + [5000] + [150] * 20, 12, 4),    # four, and twenty
    ([1000 + 3 * i for i in range(40)], 40, 8)])
def test_decode_long_sequences_among_short_ones(lens, N1, N2, form):
    """At least as many tasks as runs, some of them cut by many runs: their joins are shared out."""
    cache = S.Cache(len(lens) + N1, lens, N2, 32)
    on = None
    if form:
        rng = np.random.default_rng(N1)
        on = rng.random((len(lens), N1, -(-max(lens) // 128))) < 0.6
        on[:, :, 0] = True
        on[3, 0] = False
    q, qd, q64 = S.queries(N1 + 1, len(lens), N1, False)
    _compare(cache, q64, _decode(cache, q, qd, on, form or "mask"), on, str(form))


def _device_us(lens, N1, N2):
    """Shortest device time of a captured decode over `lens`, in microseconds."""
    import block_sparse_fp8_gb300 as bsa

    g = torch.Generator(device="cuda").manual_seed(1)
    per = [-(-n // 32) for n in lens]
    P = sum(per)
    kp, vp = (torch.randint(0, 0x78, (P, N2, 32, 128), dtype=torch.uint8, device="cuda",
                            generator=g) for _ in range(2))
    kd = torch.rand(P, N2, 32, device="cuda", generator=g) * 0.01
    table = torch.zeros(len(lens), max(per), dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    table, used = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(len(lens), N1, 128, device="cuda", generator=g).bfloat16()
    call = lambda: bsa.decode(q, kp, vp, kd, torch.ones(N2, device="cuda"), used, table, max(lens))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(10):
            call()
    best = float("inf")
    for _ in range(6):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 100)
    return best


def test_decode_time_does_not_hang_on_the_mix():
    """One sequence of 512K tokens among 319 of 500, against 320 of as many tokens in all: 60 us
    against 50, where the join by the first run's block alone took the first to 150."""
    mixed = _device_us([512 * 1024] + [500] * 319, 16, 1)
    even = _device_us([2137] * 320, 16, 1)
    assert mixed < 2 * even, (mixed, even)


@pytest.mark.parametrize("before", ["copy", "memset", "fork", "nothing"])
@pytest.mark.parametrize("sparse", [False, True])
def test_decode_captured_behind_other_nodes(before, sparse):
    """The programmatic launches as a capture's first nodes, and behind a copy, a memset and a join
    of two streams: every replay waits for what the queries come from."""
    import block_sparse_fp8_gb300 as bsa

    cache = S.Cache(75, [3000, 200], 2, 32)
    d = cache.device()
    q, _, q64 = S.queries(76, 2, 8, False)
    q = q.cuda()
    given = torch.zeros_like(q) if before in ("copy", "fork") else q
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {}
    if sparse:
        kw["block_mask"] = torch.ones(2, 8, 24, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if before == "copy":
            given.copy_(q)
        elif before == "memset":
            word.zero_()
        elif before == "fork":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                given.copy_(q)
                given.add_(0)
            word.add_(1)
            torch.cuda.current_stream().wait_stream(side)
        got = bsa.decode(given, d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"],
                         d["seqused_kv"], d["block_table"], 3000, dev_status=word, **d["kinds"],
                         **kw)
    for _ in range(3):
        if given is not q:
            given.zero_()
        got[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        _compare(cache, q64, got, what=before)


@pytest.mark.parametrize("form", [None, "mask"])
@pytest.mark.parametrize("lens,N1,N2", [([100, 300], 8, 2), ([9000, 10, 700], 12, 1),
                                        ([400] * 90, 16, 4)])
def test_decode_over_its_queries(lens, N1, N2, form):
    """out may be q: a row is written when all that reads its query has been read."""
    import block_sparse_fp8_gb300 as bsa

    cache = S.Cache(sum(lens), lens, N2, 32)
    d = cache.device()
    q, _, q64 = S.queries(N1, len(lens), N1, False)
    kw, on = {}, None
    if form:
        on = np.random.default_rng(1).random((len(lens), N1, -(-max(lens) // 128))) < 0.7
        kw["block_mask"] = torch.from_numpy(on).cuda()
    q = q.cuda()
    got = bsa.decode(q, d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"],
                     d["seqused_kv"], d["block_table"], max(lens), out=q, **d["kinds"], **kw)
    assert got[0] is q
    _compare(cache, q64, got, on, "in place")


# ----------------------------------------------------------------------- forms in combination

@pytest.mark.parametrize("form", ["mask", "index"])
@pytest.mark.parametrize("q8,k_tok,v_head,nhd", [
    (True, True, True, False), (True, False, False, True), (False, False, True, False),
    (True, True, False, True), (False, True, False, False)])
@pytest.mark.parametrize("lens,N1,N2,ps", [([900, 0, 3000], 8, 1, 32), ([130, 2000], 36, 3, 64),
                                           ([300] * 40, 16, 8, 32)])
def test_decode_sparse_types_and_scales(lens, N1, N2, ps, q8, k_tok, v_head, nhd, form):
    """Lists and masks with either type of query, either kind of either scale and either layout, up
    to more tasks than runs."""
    cache = S.Cache(sum(lens) + N1, lens, N2, ps, k_tok, v_head, nhd)
    on = np.random.default_rng(N1).random((len(lens), N1, -(-max(lens) // 128))) < 0.4
    on[0, 0] = False
    q, qd, q64 = S.queries(N1, len(lens), N1, q8)
    _compare(cache, q64, _decode(cache, q, qd, on, form), on, form)


@pytest.mark.parametrize("N1", [12, 24, 28, 40, 48])
@pytest.mark.parametrize("T,n", [(1, 2), (777, 3)])
def test_merge_head_counts(N1, T, n):
    """Head counts that are no power of two."""
    import block_sparse_fp8_gb300 as bsa
    from test_gpu_serving import _merge_reference, _parts

    outs, lses = _parts(T + N1, n, T, N1, 0.2)
    out, lse = bsa.merge_states([o.cuda() for o in outs], [x.cuda() for x in lses])
    O, Z, E, F = _merge_reference(outs, lses)
    S.within(out, O, E, "merge O")
    S.within(lse, Z, F, "merge LSE")


@pytest.mark.parametrize("cuts", [[320], [160, 320], [32, 256, 320]])
def test_prefills_over_parts_of_a_context_merge(cuts):
    """A prompt behind a cached prefix: the prefill over the prefix (in parts, none of them causal)
    and the one over the prompt itself, joined, against the prefill over both; and the decode of
    its last token the same way.  Keys differ in one dimension, by integers, and the softmax
    scale is ln 2, so every probability is a power of two, which the prefill's e4m3 holds.  What
    is left: half a bf16 step of each part, 2^-8 |O_i| with its weight, and of the result, and
    2^-13 of A = sum_j p_j |v_j| for the sums over at most 520 tokens."""
    import block_sparse_fp8_gb300 as bsa

    ps, N1, N2, T, P = 32, 8, 2, 200, 320
    rng = np.random.default_rng(len(cuts))
    n = P + T
    pages = -(-n // ps)
    level = rng.integers(0, 4, (N2, n))
    kp = np.zeros((pages, N2, ps, 128), dtype=np.uint8)
    vp = np.zeros_like(kp)
    v = S.finite_codes(rng, (N2, n, 128))
    for t in range(n):
        kp[t // ps, :, t % ps, 0] = np.array([0x00, 0x38, 0x40, 0x44])[level[:, t]]
        vp[t // ps, :, t % ps] = v[:, t]
    kp, vp = torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda()
    kd, vd = torch.ones(pages, N2, ps, device="cuda"), torch.full((N2,), 0.01, device="cuda")
    q = torch.zeros(T, N1, 128, dtype=torch.uint8, device="cuda")
    q[:, :, 0] = 0x38
    qd = torch.ones(T, N1, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table, scale = torch.arange(pages, dtype=torch.int32, device="cuda"), float(np.log(2.0))

    def part(lo, hi, causal):
        return bsa.prefill(q, kp, vp, qd, kd, vd, i32([0, T]), i32([hi - lo]),
                           table[lo // ps:-(-hi // ps)].view(1, -1).clone(), T, hi - lo,
                           softmax_scale=scale, causal=causal)

    def last(lo, hi):
        return bsa.decode(q[-1:], kp, vp, kd, vd, i32([hi - lo]),
                          table[lo // ps:-(-hi // ps)].view(1, -1).clone(), hi - lo,
                          q_descale=qd[-1:], softmax_scale=scale)

    ends = [0] + cuts
    spans = list(zip(ends, ends[1:])) + [(P, n)]
    parts = [part(a, b, b == n) for a, b in spans]
    joined = bsa.merge_states([x[0] for x in parts], [x[1] for x in parts])
    whole = part(0, n, True)
    lasts = [last(a, b) for a, b in spans]
    joined1 = bsa.merge_states([x[0] for x in lasts], [x[1] for x in lasts])
    whole1 = last(0, n)
    values = S.VAL[v] * np.float64(np.float32(0.01))
    G = N1 // N2
    O, A, R, Z = (np.zeros((T, N1, 128)), np.zeros((T, N1, 128)), np.zeros((T, N1, 128)),
                  np.zeros((N1, T)))
    for t in range(T):
        for g in range(N2):
            m = P + t + 1                                # the tokens that row t sees
            p = 2.0 ** level[g, :m]
            heads = slice(g * G, (g + 1) * G)
            O[t, heads] = p @ values[g, :m] / p.sum()
            A[t, heads] = p @ np.abs(values[g, :m]) / p.sum()
            Z[heads, t] = np.log(p.sum())
            for a, b in spans:                           # the parts' own results, with their weights
                R[t, heads] += np.abs(p[a:b] @ values[g, a:min(b, m)]) / p.sum()
    step, sums, lse = 2.0 ** -8, 2.0 ** -13 * A, np.full_like(Z, 2.0 ** -13)
    S.within(whole[0], O, step * np.abs(O) + sums, "whole O")
    S.within(whole[1], Z, lse, "whole LSE")
    S.within(joined[0], O, step * (np.abs(O) + R) * (1 + 2.0 ** -8) + sums, "joined O")
    S.within(joined[1], Z, lse, "joined LSE")
    S.within(whole1[0], O[-1:], (step * np.abs(O) + sums)[-1:], "last O")
    S.within(joined1[0], O[-1:], (step * (np.abs(O) + R) * (1 + 2.0 ** -8) + sums)[-1:],
             "joined last O")
    S.within(joined1[1], Z[:, -1:], lse[:, -1:], "joined last LSE")


@pytest.mark.parametrize("nhd", [False, True])
@pytest.mark.parametrize("f32", [False, True])
def test_gather_one_head_many_blocks(f32, nhd):
    """One KV head, rows enough for every size of a block's run of tokens."""
    import block_sparse_fp8_gb300 as bsa

    lens = [20000, 0, 1, 60000]
    cache = S.Cache(9, lens, 1, 64, nhd=nhd)
    d = cache.device()
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    k, v = bsa.gather_kv(d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"], cu,
                         d["block_table"], sum(lens), **d["kinds"],
                         out_dtype=torch.float32 if f32 else torch.bfloat16)
    for got, i in ((k, 0), (v, 1)):
        want = np.concatenate([cache.rows(b)[i].transpose(1, 0, 2) for b in range(4)])
        assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).to(got.dtype))


# ------------------------------------------------------------------------------- wide ranges

@pytest.mark.parametrize("power", [4, 16, 17, 18, 19, 20, 21, 22, 23, 24, 40, 100])
@pytest.mark.parametrize("N1,form", [(8, None), (16, "mask")])
def test_decode_large_scores(power, N1, form):
    """Scores far above 2^24, where fp32 holds no odd numbers: integers below 2^7 times 2^power.
    Scores that differ do so by at least 2^(power + 1) > 30, so a row is the mean of V over the
    tokens of its largest score: half a bf16 step, 2^-12 of A for the rest (as above)."""
    lens = [300, 37]
    cache = S.Cache(power, lens, 1, 32)
    _unit_keys(cache)
    cache.kd_pages = np.where(np.isnan(cache.kd_pages), cache.kd_pages, 1.0).astype(np.float32)
    rng = np.random.default_rng(power)
    sign = rng.choice([-1.0, 1.0], (2, N1, 128))
    q = torch.from_numpy(sign * 2.0 ** power).to(torch.bfloat16)
    on = None
    if form:
        on = rng.random((2, N1, 3)) < 0.7
        on[:, :, 0] = True
    out, lse = _decode(cache, q, None, on, scale=1.0)
    for b, n in enumerate(lens):
        k, v = S.VAL[cache.k[b][0]], cache.rows(b)[1][0]
        for h in range(N1):
            take = np.ones(n, bool) if on is None else np.repeat(on[b, h], S.TILE)[:n]
            s = np.where(take, k @ sign[b, h], -np.inf)
            best = s == s.max()
            O, A = v[best].mean(0), np.abs(v[best]).mean(0)
            S.within(out[b, h], O, 2.0 ** -8 * np.abs(O) + 2.0 ** -12 * A, f"O of {b}, {h}")
            z = s.max() * 2.0 ** power + np.log(best.sum())
            assert abs(float(lse[h, b]) - z) <= 2.0 ** -21 * abs(z) + 2.0 ** -15


@pytest.mark.parametrize("vd", [1e-37, 1e-30, 1e30])
@pytest.mark.parametrize("lens", [[300], [20000, 40]])
def test_decode_value_magnitudes(vd, lens):
    """V descales near the ends of fp32's range."""
    cache = S.Cache(7, lens, 2, 32)
    cache.vd[:] = vd
    q, qd, q64 = S.queries(8, len(lens), 8, False)
    _compare(cache, q64, _decode(cache, q, qd), what="values")


@pytest.mark.parametrize("N1", [8, 16])
@pytest.mark.parametrize("form", [None, "mask"])
def test_decode_long_sums_have_no_bias(N1, form):
    """A CTA's sums over 32K tokens, V of one sign (all sequences read the same pages, with queries of
    their own).  A weight is off by less than 2^-20 (scores below 2^4 in fp32, the exponential, two
    fp16 terms), an unbiased fp32 sum by less than that, so a result lies within 2^-19 of the exact
    one and the share of results that round to another bf16 number, whose steps are at least
    2^-8 of it, is below 2 * 2^-19 / 2^-8 = 2^-10.  Sums that lose 2^-25 at each of 1000 products are
    2^-15 off."""
    import block_sparse_fp8_gb300 as bsa

    n, ps, B = 32768, 64, 304
    g = torch.Generator(device="cuda").manual_seed(N1)
    kp = (torch.randn(n // ps, 1, ps, 128, device="cuda", generator=g) * 60).clamp(-448, 448)
    vp = torch.rand(n // ps, 1, ps, 128, device="cuda", generator=g) * 200 + 100
    kp, vp = (x.to(torch.float8_e4m3fn) for x in (kp, vp))
    kd = torch.rand(n // ps, 1, ps, device="cuda", generator=g) * 0.01 + 0.01
    vd = torch.full((1,), 0.01, device="cuda")
    table = torch.arange(n // ps, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    used = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = torch.randn(B, N1, 128, device="cuda", generator=g).bfloat16()
    kw = {}
    if form:
        kw["block_mask"] = torch.ones(B, N1, n // 128, dtype=torch.uint8, device="cuda")
        kw["block_mask"][:, ::2, 1::2] = 0
    out, _ = bsa.decode(q, kp, vp, kd, vd, used, table, n, **kw)
    k = kp.double().view(n, 128) * kd.double().view(n, 1)
    v = vp.double().view(n, 128) * float(vd)
    off = 0
    for h in range(N1):
        s = q[:, h].double() @ k.t() / 128 ** 0.5
        if form and h % 2 == 0:
            s.view(B, -1, 256)[:, :, 128:] = -float("inf")
        want = (torch.softmax(s, 1) @ v).bfloat16()
        off += int((out[:, h] != want).sum())
    assert off < 2.0 ** -10 * out.numel(), off / out.numel()
