"""decode, gather_kv and merge_states on the GPU against fp64 references (bounds and their
derivation: serving_helpers.py)."""
import numpy as np
import pytest
import torch

import serving_helpers as S
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def _cuda(*ts):
    return tuple(None if t is None else t.cuda() for t in ts)


def _decode(cache, q, qd, enabled=None, form="mask", scale=None, dev=None, **kw):
    """One decode into NaN-filled outputs with a NaN-filled workspace; asserts a clean status."""
    import block_sparse_fp8_gb300 as bsa

    d = dev or cache.device()
    q, qd = _cuda(q, qd)
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
    ws = torch.full((bsa.decode_workspace_size(dims),), 0xff, dtype=torch.uint8, device="cuda")
    out = torch.full((B, N1, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N1, B), float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    expect = kw.pop("status", 0)
    got = bsa.decode(q, d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"],
                     d["seqused_kv"], d["block_table"], max_kv, q_descale=qd, softmax_scale=scale,
                     out=out, lse=lse, dev_status=st, workspace=ws, **d["kinds"], **kw)
    torch.cuda.synchronize()
    assert got[0] is out and got[1] is lse
    assert int(st.item()) == expect
    return out, lse


def _compare(cache, q64, got, enabled=None, what="", scale=None):
    O, Z, E, F = S.reference(cache, q64, enabled, **({} if scale is None else {"scale": scale}))
    S.within(got[0], O, E, what + " O")
    S.within(got[1], Z, F, what + " LSE")


DENSE = [
    # lens, N1, N2, ps, q8, k_tok, v_head, nhd
    ([1], 1, 1, 32, False, True, True, False),
    ([2, 31], 2, 2, 32, True, True, True, True),
    ([32, 33, 63, 64, 65], 8, 2, 32, False, True, True, False),
    ([127, 128, 129], 8, 1, 64, False, False, False, False),
    ([255, 0, 256, 257, 0], 12, 4, 64, True, True, False, True),
    ([1000, 1, 517], 7, 1, 32, False, True, True, True),
    ([300] * 3, 9, 1, 64, False, True, True, False),
    ([640, 5, 1290], 32, 2, 64, True, False, True, False),
    ([77], 48, 3, 32, False, True, True, True),
    ([2048], 5, 5, 64, False, True, True, False),
    ([512, 3, 400], 10, 2, 32, False, True, True, False),
    ([200] * 80, 8, 4, 64, True, True, True, False),
    ([9001, 130], 10, 2, 32, False, True, True, False),
    ([20000], 16, 1, 64, True, True, True, True),
]


@pytest.mark.parametrize("lens,N1,N2,ps,q8,k_tok,v_head,nhd", DENSE)
def test_decode_dense(lens, N1, N2, ps, q8, k_tok, v_head, nhd):
    cache = S.Cache(sum(lens) + N1, lens, N2, ps, k_tok, v_head, nhd)
    q, qd, q64 = S.queries(N1, len(lens), N1, q8)
    _compare(cache, q64, _decode(cache, q, qd), what="dense")


def test_decode_many_short_sequences():
    """More sequences than threads of a CTA, one to three tiles each, idle ones among them."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 300, 301)]
    cache = S.Cache(11, lens, 2, 32)
    q, qd, q64 = S.queries(12, len(lens), 4, False)
    _compare(cache, q64, _decode(cache, q, qd), what="many")


def test_decode_thousands_of_tokens_of_one():
    """Far more sequences than CTAs: 5000 of one to three tokens."""
    rng = np.random.default_rng(6)
    lens = [int(x) for x in rng.integers(1, 4, 5000)]
    cache = S.Cache(12, lens, 1, 32)
    q, qd, q64 = S.queries(13, len(lens), 2, True)
    _compare(cache, q64, _decode(cache, q, qd), what="thousands")


@pytest.mark.parametrize("form", [None, "mask", "index"])
def test_decode_longest_capacity(form):
    """max_kv_len at the supported limit, as a graph for any length would be captured, over short
    sequences and over one that fills it."""
    cap = 4096 * 128
    for lens in ([70, 0, 4000], [cap]):
        cache = S.Cache(14, lens, 1, 64, spare_cols=0)
        full = np.full((len(lens), cap // 64), 0x7fffffff, dtype=np.int32)
        full[:, :cache.L] = cache.table
        cache.table, cache.L = full, cap // 64
        on = None
        if form:
            on = np.random.default_rng(2).random((len(lens), 3, 4096)) < 0.02
        q, qd, q64 = S.queries(15, len(lens), 3, False)
        _compare(cache, q64, _decode(cache, q, qd, on, form, max_kv_len=cap), on, str(lens))


def test_decode_shared_pages():
    """Two sequences whose tables name the same pages, one twice in a row."""
    cache = S.Cache(16, [96, 96], 2, 32)
    cache.table[1, 0] = cache.table[1, 2] = cache.table[0, 1]
    for x in (cache.k, cache.v, cache.kd):
        x[1] = x[1].copy()
        x[1][:, :32] = x[1][:, 64:96] = x[0][:, 32:64]
    q, qd, q64 = S.queries(17, 2, 4, False)
    _compare(cache, q64, _decode(cache, q, qd), what="shared")


def test_decode_refuses_a_small_workspace():
    import block_sparse_fp8_gb300 as bsa

    cache = S.Cache(18, [5000], 1, 32)
    d = cache.device()
    q = S.queries(19, 1, 8, False)[0].cuda()
    dims = bsa.make_decode_dims(q, d["k_pages"], d["block_table"], 5000, 1, 2)
    need = bsa.decode_workspace_size(dims)
    for ws in (torch.empty(need - 1, dtype=torch.uint8, device="cuda"),
               torch.empty(need + 64, dtype=torch.uint8, device="cuda")[64:]):
        with pytest.raises(bsa.BsaError) as e:
            _decode_call(bsa, cache, d, q, None, None, ws)
        assert e.value.status == 4
    with pytest.raises(ValueError, match="device"):
        _decode_call(bsa, cache, dict(d, seqused_kv=d["seqused_kv"].cpu()), q, None, None, None)
    with pytest.raises(bsa.BsaError):                    # bf16 queries take no q_descale
        _decode_call(bsa, cache, d, q, None, None, None,
                     q_descale=torch.ones(1, 8, device="cuda"))


def test_decode_all_idle():
    cache = S.Cache(1, [0, 0, 0], 2, 64)
    q, qd, q64 = S.queries(2, 3, 6, False)
    _compare(cache, q64, _decode(cache, q, qd, max_kv_len=64), what="idle")
    _compare(cache, q64, _decode(cache, q, qd, max_kv_len=0), what="idle, no tiles")
    # and with every head's list empty
    on = np.zeros((3, 6, 1), dtype=bool)
    _compare(cache, q64, _decode(cache, q, qd, on, "index", max_kv_len=64), what="idle lists")


@pytest.mark.parametrize("form", ["mask", "index"])
@pytest.mark.parametrize("lens,N1,N2,keep", [
    ([700], 1, 1, 0.5), ([1500, 0, 90], 6, 2, 0.4), ([5000, 257], 16, 1, 0.1),
    ([300, 129], 27, 3, 0.6), ([17000], 8, 1, 0.05)])
def test_decode_sparse(form, lens, N1, N2, keep):
    cache = S.Cache(sum(lens), lens, N2, 32, nhd=form == "index")
    rng = np.random.default_rng(N1)
    Kb = -(-max(lens) // 128)
    on = rng.random((len(lens), N1, Kb)) < keep
    on[0, 0] = False                                   # a head that sees nothing
    q, qd, q64 = S.queries(N1 + 1, len(lens), N1, False)
    _compare(cache, q64, _decode(cache, q, qd, on, form), on, form)


@pytest.mark.parametrize("form", ["mask", "index"])
@pytest.mark.parametrize("N1", [4, 12])
def test_decode_nan_in_a_tile_one_head_masks(N1, form):
    """Every other head masks a tile that holds NaN in K and V; the others of the same KV head read
    it and get NaN, the first are untouched by it."""
    cache = S.Cache(4, [500], 1, 32)
    q, qd, q64 = S.queries(5, 1, N1, False)
    keep, hit = list(range(0, N1, 2)), list(range(1, N1, 2))
    on = np.ones((1, N1, 4), dtype=bool)
    on[0, keep, 1] = False
    d = cache.device()
    pg = int(cache.table[0, 5])                          # tokens 160 .. 191 lie in tile 1
    d["k_pages"][pg, 0, 3] = 0x7f
    d["v_pages"][pg, 0, 4] = 0xff
    out, lse = _decode(cache, q, qd, on, form, dev=d)
    O, Z, E, F = S.reference(cache, q64, on)
    S.within(out[:, keep], O[:, keep], E[:, keep], "masking heads O")
    S.within(lse[keep], Z[keep], F[keep], "masking heads LSE")
    assert torch.isnan(out[:, hit].float()).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_decode_softmax_scale(scale):
    cache = S.Cache(6, [400, 3], 1, 64)
    q, qd, q64 = S.queries(7, 2, 3, False)
    _compare(cache, q64, _decode(cache, q, qd, scale=scale), what=str(scale), scale=scale)


@pytest.mark.parametrize("mag", [1e-30, 1e30])
def test_decode_query_magnitudes(mag):
    """bf16 queries far outside fp16's range, their scale undone by softmax_scale."""
    cache = S.Cache(8, [333], 1, 64)
    q, qd, q64 = S.queries(9, 1, 4, False, scale=mag)
    q[0, 1] = 0                                          # a zero row
    q64[0, 1] = 0
    scale = 0.1 / mag
    _compare(cache, q64, _decode(cache, q, qd, scale=scale), what=str(mag), scale=scale)


def test_decode_rising_scores():
    """Scores whose spread rises and falls along the cache by a factor of 600: the running
    maximum moves often, and most weights underflow against it."""
    cache = S.Cache(10, [3000], 1, 32, spread=1.0)
    cache.kd[0][0] = np.linspace(0.001, 0.6, 3000, dtype=np.float32)
    cache.kd[0][0, 1500:] = np.linspace(0.6, 0.001, 1500, dtype=np.float32)
    for i in range(-(-3000 // 32)):
        m = min(32, 3000 - i * 32)
        cache.kd_pages[cache.table[0, i], 0, :m] = cache.kd[0][0, i * 32:i * 32 + m]
    q, qd, q64 = S.queries(11, 1, 8, False)
    _compare(cache, q64, _decode(cache, q, qd), what="rising")


@pytest.mark.parametrize("q8", [False, True])
def test_decode_strided_queries(q8):
    """q as the first part of a wider projection's output."""
    cache = S.Cache(13, [200, 400, 600], 2, 64)
    q, qd, q64 = S.queries(14, 3, 8, q8)
    wide = torch.zeros(3, 12 * 128 + 16, dtype=q.dtype)
    wide[:, :8 * 128] = q.reshape(3, -1)
    wide = wide.cuda()
    view = wide[:, :8 * 128].unflatten(1, (8, 128))
    _compare(cache, q64, _decode(cache, view, qd), what="strided")


def test_decode_without_lse_and_without_workspace():
    import block_sparse_fp8_gb300 as bsa

    cache = S.Cache(15, [900, 100], 2, 64)
    q, qd, q64 = S.queries(16, 2, 4, False)
    d = cache.device()
    out, lse = bsa.decode(q.cuda(), d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"],
                          d["seqused_kv"], d["block_table"], 900, return_lse=False)
    assert lse is None
    O, _, E, _ = S.reference(cache, q64)
    S.within(out, O, E, "no lse")


def test_decode_page_offsets_beyond_32_bits():
    """Pages that start past 4 GiB of a pool."""
    cache = S.Cache(17, [400, 70], 8, 64)
    d = cache.device()
    shift = (1 << 32) // (8 * 64 * 128) + 1
    big = {n: torch.empty((cache.P + shift,) + tuple(d[n].shape[1:]), dtype=d[n].dtype,
                          device="cuda") for n in ("k_pages", "v_pages", "k_descale")}
    for n in big:
        big[n][shift:] = d[n]
    table = torch.from_numpy(cache.table.astype(np.int64) + shift).clamp(max=2 ** 31 - 1)
    d.update(big, block_table=table.int().cuda())
    q, qd, q64 = S.queries(18, 2, 16, False)
    _compare(cache, q64, _decode(cache, q, qd, dev=d), what="big pool")
    import block_sparse_fp8_gb300 as bsa

    cu = torch.tensor([0, 400, 470], dtype=torch.int32, device="cuda")
    k, v = bsa.gather_kv(d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"], cu,
                         d["block_table"], 470, out_dtype=torch.float32)
    want = np.concatenate([cache.rows(b)[0].transpose(1, 0, 2) for b in range(2)])
    assert np.array_equal(k.cpu().numpy(), want.astype(np.float32))


def test_decode_bad_device_data():
    """Bad lengths, pages and indices: reported, the entry skipped, the other rows unharmed."""
    import block_sparse_fp8_gb300 as bsa

    cache = S.Cache(19, [300, 300, 300], 1, 32)
    q, qd, q64 = S.queries(20, 3, 4, False)
    d = cache.device()
    d["seqused_kv"][0] = -1
    d["seqused_kv"][2] = 301                              # above max_kv_len
    out, lse = _decode(cache, q, qd, dev=d, status=bsa.DEV_BAD_SEQLEN)
    O, Z, E, F = S.reference(cache, q64)
    S.within(out[1:2], O[1:2], E[1:2], "good row")
    assert (out[[0, 2]] == 0).all() and (lse[:, [0, 2]] == S.NEG_FLT_MAX).all()
    # bad pages read as zeros: K = V = 0 there
    d = cache.device()
    d["block_table"][0, 1] = -1
    d["block_table"][2, 0] = cache.P
    out, lse = _decode(cache, q, qd, dev=d, status=bsa.DEV_BAD_PAGE)
    cache.k[0][:, 32:64] = cache.v[0][:, 32:64] = 0
    cache.k[2][:, :32] = cache.v[2][:, :32] = 0
    _compare(cache, q64, (out, lse), what="bad pages")
    # indices out of range, and a length beyond the list
    d = cache.device()
    d["block_table"][0, 1] = cache.table[0, 1]
    idx = torch.zeros(3, 4, 3, dtype=torch.int32)
    cnt = torch.ones(3, 4, dtype=torch.int32)
    idx[1, 2] = torch.tensor([3, -1, 1])
    cnt[1, 2] = 3
    idx[1, 3] = torch.tensor([0, 2, 0])
    cnt[1, 3] = 99
    cnt[1, 1] = -5
    on = np.zeros((3, 4, 3), dtype=bool)
    on[:, :, 0] = True
    on[1, 1:] = [[0, 0, 0], [0, 1, 0], [1, 0, 1]]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = bsa.decode(q.cuda(), d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"],
                          d["seqused_kv"], d["block_table"], 300, sparse_indices=idx.cuda(),
                          sparse_seq_len=cnt.cuda(), dev_status=st, **d["kinds"])
    torch.cuda.synchronize()
    assert int(st.item()) == bsa.DEV_BAD_INDEX
    O, Z, E, F = S.reference(cache, q64, on)
    S.within(out[1], O[1], E[1], "bad indices O")
    S.within(lse[:, 1], Z[:, 1], F[:, 1], "bad indices LSE")


# ------------------------------------------------------------------------------------ streams

def _decode_call(bsa, cache, d, q, out, lse, ws, **kw):
    return bsa.decode(q, d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"],
                      d["seqused_kv"], d["block_table"], max(cache.lens), out=out, lse=lse,
                      workspace=ws, **d["kinds"], **kw)


@pytest.mark.parametrize("sparse", [False, True])
def test_decode_two_graphs_share_a_workspace(sparse):
    """Two captured decodes over different caches with one workspace, replayed in turn, each
    replay the eager result bit for bit; then with longer sequences written in place."""
    import block_sparse_fp8_gb300 as bsa

    graphs = []
    ws = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    for i, lens in enumerate(([5000, 130], [900, 4000])):
        cache = S.Cache(30 + i, lens, 2, 32)
        d = cache.device()
        q, _, q64 = S.queries(40 + i, 2, 8, False)
        q = q.cuda()
        kw, on = {}, None
        if sparse:
            on = np.random.default_rng(i).random((2, 8, -(-max(lens) // 128))) < 0.5
            kw["block_mask"] = torch.from_numpy(on.astype(np.uint8)).cuda()
        eager = _decode_call(bsa, cache, d, q, None, None, None, **kw)
        out, lse = torch.empty_like(eager[0]), torch.empty_like(eager[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _decode_call(bsa, cache, d, q, out, lse, ws, **kw)
        graphs.append((g, out, lse, eager, cache, d, q, q64, kw, on))
    for _ in range(3):
        for g, out, lse, eager, *_ in graphs:
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
    # lengths that changed in place between replays: the split follows them
    g, out, lse, eager, cache, d, q, q64, kw, on = graphs[0]
    cache.lens[0], cache.lens[1] = 700, 0
    cache.k[0], cache.v[0], cache.kd[0] = (x[:, :700] for x in (cache.k[0], cache.v[0],
                                                                cache.kd[0]))
    d["seqused_kv"].copy_(torch.tensor([700, 0], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    _compare(cache, q64, (out, lse), on, "shorter")


@pytest.mark.parametrize("sparse", [False, True])
def test_decode_step_captured_with_its_length_update(sparse):
    """A captured step that lengthens the sequences, appends and decodes, replayed: every replay sees
    the lengths and rows that its own step wrote (bit for bit an eager decode's result)."""
    import block_sparse_fp8_gb300 as bsa

    g = torch.Generator(device="cuda").manual_seed(4)
    B, N1, N2, ps, L = 4, 16, 2, 32, 96
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
    kp, vp = (torch.zeros(B * L, N2, ps, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    kd = torch.ones(B * L, N2, ps, device="cuda")
    vs = torch.full((N2,), 0.012, device="cuda")
    table = torch.randperm(B * L, device="cuda", generator=g).int().view(B, L)
    used = torch.tensor([2500, 10, 127, 1023], dtype=torch.int32, device="cuda")
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), used.cumsum(0).int()])
    T = int(cu[-1])
    bsa.append_kv(rand(T, N2, 128), rand(T, N2, 128), cu, torch.zeros_like(used), table, kp, vp,
                  k_descale=kd, v_scale=vs)
    k1, v1, q = rand(B, N2, 128), rand(B, N2, 128), rand(B, N1, 128)
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    cap = L * ps
    kw = {}
    if sparse:
        kw["block_mask"] = (torch.rand(B, N1, cap // 128, device="cuda", generator=g) < 0.5).byte()
        kw["block_mask"][:, :, 0] = 1
    out = torch.empty(B, N1, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(N1, B, device="cuda")
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")

    def decode(**o):
        return bsa.decode(q, kp, vp, kd, vs, used, table, cap, **o, **kw)

    def step():
        bsa.append_kv(k1, v1, one, used, table, kp, vp, k_descale=kd, v_scale=vs)
        used.add_(1)
        decode(out=out, lse=lse, workspace=ws)
        k1.mul_(-1.01)                                   # the next step's rows
        q.copy_(q.roll(1, 2))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(40):
        graph.replay()
        q.copy_(q.roll(-1, 2))                           # this replay's queries again
        want = decode()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]), i
        q.copy_(q.roll(1, 2))
    assert int(used[1]) == 10 + 41


def test_decode_on_two_streams_at_once():
    import block_sparse_fp8_gb300 as bsa

    jobs = []
    for i in range(2):
        cache = S.Cache(50 + i, [6000 + i, 77], 2, 64)
        q, _, q64 = S.queries(60 + i, 2, 16, False)
        jobs.append((cache, cache.device(), q.cuda(), q64, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = []
        for c, d, q, _, s in jobs:
            with torch.cuda.stream(s):
                got.append(_decode_call(bsa, c, d, q, None, None, None))
    torch.cuda.synchronize()
    for (cache, _, _, q64, _), g in zip(jobs, got):
        _compare(cache, q64, g, what="two streams")


def test_decode_and_merge_on_a_given_stream():
    """stream= names the stream; what the call allocates itself stays its own until that stream is
    through with it."""
    import block_sparse_fp8_gb300 as bsa

    cache = S.Cache(65, [9000, 3000], 2, 64)
    q, _, q64 = S.queries(66, 2, 8, False)
    d, q = cache.device(), q.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                    # the call waits behind this
    got = bsa.decode(q, d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"],
                     d["seqused_kv"], d["block_table"], 9000, stream=side, **d["kinds"])
    both = bsa.merge_states([got[0]], [got[1]], stream=side)
    for _ in range(8):                                   # would take a freed workspace's place
        torch.full((4 << 20,), float("nan"), device="cuda")
    side.synchronize()
    _compare(cache, q64, got, what="given stream")
    _compare(cache, q64, both, what="merge of one")


def test_decode_first_call_inside_a_capture():
    """A fresh process whose first call of the library is captured into a graph."""
    import os
    import subprocess
    import sys

    code = """
import numpy as np, torch
import serving_helpers as S
import block_sparse_fp8_gb300 as bsa
cache = S.Cache(75, [3000, 200], 2, 32)
d = cache.device()
q, _, q64 = S.queries(76, 2, 8, False)
q = q.cuda()
out = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda")
lse = torch.empty(8, 2, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    bsa.decode(q, d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"], d["seqused_kv"],
               d["block_table"], 3000, out=out, lse=lse, **d["kinds"])
g.replay()
torch.cuda.synchronize()
O, Z, E, F = S.reference(cache, q64)
S.within(out, O, E, "O")
S.within(lse, Z, F, "LSE")
print("captured first")
"""
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here]))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env,
                       timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_decode_watchdog():
    """A batch that waits for memory (537 MB).  With a limit below those waits its launches stop
    early and say so; the launch after them, at the default limit, gives the bits of the one
    before them."""
    import block_sparse_fp8_gb300 as bsa

    g = torch.Generator(device="cuda").manual_seed(1)
    B, N1, N2, ps, n = 64, 32, 8, 64, 4096
    P = B * n // ps
    kp, vp = (torch.randint(0, 0x78, (P, N2, ps, 128), dtype=torch.uint8, device="cuda",
                            generator=g) for _ in range(2))
    kd = torch.rand(P, N2, ps, device="cuda", generator=g) * 0.01
    vd = torch.full((N2,), 0.01, device="cuda")
    used = torch.full((B,), n, dtype=torch.int32, device="cuda")
    table = torch.randperm(P, device="cuda", generator=g).int().view(B, -1)
    q = torch.randn(B, N1, 128, device="cuda", generator=g).bfloat16()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: bsa.decode(q, kp, vp, kd, vd, used, table, n, dev_status=st)
    before = call()
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.isfinite(before[0].float()).all()
    try:
        bsa.set_wait_limit_ns(1)
        for _ in range(3):
            st.zero_()
            call()
            torch.cuda.synchronize()
            assert int(st.item()) == bsa.DEV_TIMEOUT
    finally:
        bsa.set_wait_limit_ns(0)
    st.zero_()
    after = call()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(after[0], before[0]) and torch.equal(after[1], before[1])


def test_decode_is_deterministic():
    import block_sparse_fp8_gb300 as bsa

    cache = S.Cache(70, [12000, 300, 5000], 2, 32)
    d = cache.device()
    q = S.queries(71, 3, 16, False)[0].cuda()
    first = _decode_call(bsa, cache, d, q, None, None, None)
    for _ in range(4):
        again = _decode_call(bsa, cache, d, q, None, None, None)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ------------------------------------------------------------------------------------- gather

@pytest.mark.parametrize("nhd", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,starts,N2,ps,k_tok,v_head", [
    ([1], None, 1, 32, True, True), ([0, 33, 0, 64, 1, 0], None, 3, 32, True, False),
    ([400, 100], [1, 129], 8, 64, False, True), ([7] * 70, [90] * 70, 2, 32, True, True),
    ([3000, 0, 129], [0, 5, 31], 5, 64, True, True)])
def test_gather_exact(lens, starts, N2, ps, k_tok, v_head, dtype, nhd):
    import block_sparse_fp8_gb300 as bsa

    st = starts or [0] * len(lens)
    cache = S.Cache(sum(lens) + N2, [a + n for a, n in zip(st, lens)], N2, ps, k_tok, v_head, nhd)
    d = cache.device()
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    T = sum(lens)
    total = T + 5
    k = torch.full((total, N2, 128), 7.0, dtype=dtype, device="cuda")
    v = torch.full_like(k, 9.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cs = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    got = bsa.gather_kv(d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"], cu,
                        d["block_table"], total, cache_starts=cs, k_out=k, v_out=v,
                        dev_status=status, **d["kinds"])
    torch.cuda.synchronize()
    assert got[0] is k and got[1] is v and int(status.item()) == 0
    assert (k[T:] == 7).all() and (v[T:] == 9).all()      # rows behind the last sequence
    parts = [tuple(x[:, a:] for x in cache.rows(b)) for b, a in enumerate(st)]
    for got, which in ((k, 0), (v, 1)):
        want = np.concatenate([p[which].transpose(1, 0, 2) for p in parts]).astype(np.float32)
        want = torch.from_numpy(want).to(dtype)
        assert torch.equal(got[:T].cpu(), want)


def test_gather_fewer_rows_than_tokens():
    """total below cu_seqlens[B]: the rows there are, and nothing behind them."""
    import block_sparse_fp8_gb300 as bsa

    cache = S.Cache(81, [50, 60], 2, 32)
    d = cache.device()
    cu = torch.tensor([0, 50, 110], dtype=torch.int32, device="cuda")
    k = torch.full((90, 2, 128), 5.0, device="cuda")
    bsa.gather_kv(d["k_pages"], None, d["k_descale"], None, cu, d["block_table"], 73,
                  k_out=k[:73])
    want = np.concatenate([cache.rows(b)[0].transpose(1, 0, 2) for b in range(2)])
    assert np.array_equal(k[:73].cpu().numpy(), want[:73].astype(np.float32))
    assert (k[73:] == 5).all()


def test_gather_one_side_and_missing_pages():
    import block_sparse_fp8_gb300 as bsa

    cache = S.Cache(80, [100, 40], 2, 32)
    d = cache.device()
    cu = torch.tensor([0, 100, 140], dtype=torch.int32, device="cuda")
    k, v = bsa.gather_kv(None, d["v_pages"], None, d["v_descale"], cu, d["block_table"], 140)
    assert k is None
    want = np.concatenate([cache.rows(b)[1].transpose(1, 0, 2) for b in range(2)])
    want = torch.from_numpy(want.astype(np.float32)).bfloat16()
    assert torch.equal(v.cpu(), want)
    k, v = bsa.gather_kv(d["k_pages"], None, d["k_descale"], None, cu, d["block_table"], 140)
    assert v is None and torch.isfinite(k).all()
    # a page out of range, and positions before the first and beyond the last column
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d["block_table"][0, 2] = cache.P
    starts = torch.tensor([0, -3], dtype=torch.int32, device="cuda")
    _, v = bsa.gather_kv(d["k_pages"], d["v_pages"], d["k_descale"], d["v_descale"], cu,
                         d["block_table"], 140, cache_starts=starts, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == bsa.DEV_BAD_PAGE
    assert torch.equal(v[:64].cpu(), want[:64]) and torch.equal(v[96:100].cpu(), want[96:100])
    assert (v[64:96] == 0).all() and (v[100:103] == 0).all()
    assert torch.equal(v[103:140].cpu(), want[100:137])
    status.zero_()
    starts = torch.tensor([0, 32 * cache.L - 10], dtype=torch.int32, device="cuda")
    cache2 = cache.device()
    cache2["block_table"][:, 3:] = 0
    bsa.gather_kv(cache2["k_pages"], cache2["v_pages"], cache2["k_descale"],
                  cache2["v_descale"], cu, cache2["block_table"], 140, cache_starts=starts,
                  dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == bsa.DEV_BAD_PAGE


# -------------------------------------------------------------------------------------- merge

def _parts(seed, n, T, N1, empty):
    rng = np.random.default_rng(seed)
    outs = [torch.from_numpy(rng.standard_normal((T, N1, 128)).astype(np.float32)).bfloat16()
            for _ in range(n)]
    lses = [torch.from_numpy((rng.standard_normal((N1, T)) * 3 + 5).astype(np.float32))
            for _ in range(n)]
    for o, l in zip(outs, lses):
        gone = torch.from_numpy(rng.random((N1, T)) < empty)
        l[gone] = S.NEG_FLT_MAX
        o[gone.t()] = float("nan")                       # not to be used
    return outs, lses


def _merge_reference(outs, lses):
    l = np.stack([x.double().numpy() for x in lses])
    l = np.where(l == S.NEG_FLT_MAX, -np.inf, l)
    m = l.max(0)
    some = m > -np.inf
    w = np.where(l > -np.inf, np.exp(l - np.where(some, m, 0)), 0.0)
    t = w.sum(0)
    O = np.zeros(outs[0].shape)
    A = np.zeros(outs[0].shape)
    for wi, o in zip(w, outs):
        f = (wi / np.where(some, t, 1)).T[..., None]
        x = np.where(f > 0, o.double().numpy(), 0.0)
        O += f * x
        A += f * np.abs(x)
    Z = np.where(some, np.where(some, m, 0) + np.log(np.where(some, t, 1)), S.NEG_FLT_MAX)
    return O, Z, 2.0 ** -8 * np.abs(O) + 2.0 ** -15 * A, np.where(
        some, 2.0 ** -22 * np.abs(Z) + 2.0 ** -15, 0.0)


@pytest.mark.parametrize("n,T,N1,empty", [
    (1, 1, 1, 0.0), (2, 3, 5, 0.5), (3, 17, 8, 0.3), (2, 129, 33, 0.1), (8, 9, 64, 0.6),
    (5, 1000, 4, 0.2), (4, 7, 1, 1.0), (2, 2049, 32, 0.05)])
def test_merge(n, T, N1, empty):
    import block_sparse_fp8_gb300 as bsa

    outs, lses = _parts(n * T + N1, n, T, N1, empty)
    out, lse = bsa.merge_states([o.cuda() for o in outs], [x.cuda() for x in lses])
    O, Z, E, F = _merge_reference(outs, lses)
    S.within(out, O, E, "merge O")
    S.within(lse, Z, F, "merge LSE")


def test_merge_in_place_and_odd_lses():
    """Outputs that are one of the inputs; -inf as an empty part; LSEs far apart and large."""
    import block_sparse_fp8_gb300 as bsa

    outs, lses = _parts(90, 3, 40, 6, 0.3)
    lses[0][0, :10] = -float("inf")
    lses[1][1] = 3.0e4
    lses[2][1] = 3.0e4 - 1
    ref_l = [torch.where(x == -float("inf"), torch.full_like(x, S.NEG_FLT_MAX), x) for x in lses]
    O, Z, E, F = _merge_reference(outs, ref_l)
    do, dl = [o.cuda() for o in outs], [x.cuda() for x in lses]
    out, lse = bsa.merge_states(do, dl, out=do[1], lse=dl[2])
    assert out is do[1] and lse is dl[2]
    S.within(out, O, E, "in place O")
    S.within(lse, Z, F, "in place LSE")
    out, lse = bsa.merge_states([o.cuda() for o in outs], [x.cuda() for x in lses],
                                return_lse=False)
    assert lse is None
    S.within(out, O, E, "no lse O")


# ------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("nhd", [False, True])
def test_a_turn_of_serving(nhd):
    """Append a prompt, prefill it, append tokens one by one and decode them; the cache read
    back explains every result, and the decode over two halves of the tiles merges into the
    decode over all of them."""
    import block_sparse_fp8_gb300 as bsa

    lay = bsa.KV_NHD if nhd else bsa.KV_HND
    g = torch.Generator().manual_seed(3)
    B, N1, N2, ps, L, P = 3, 8, 2, 32, 12, 40
    lens = [150, 33, 256]
    T = sum(lens)
    rand = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    shape = (P, ps, N2, 128) if nhd else (P, N2, ps, 128)
    kp, vp = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    kd = torch.zeros(P, N2, ps, device="cuda")
    vs = torch.full((N2,), 5.0 / 448, device="cuda")
    table = torch.randperm(P, generator=g)[:B * L].view(B, L).int().cuda()
    status = i32([0])
    cu = i32(np.cumsum([0] + lens))
    k, v, q = rand(T, N2, 128), rand(T, N2, 128), rand(T, N1, 128)
    bsa.append_kv(k, v, cu, i32([0] * B), table, kp, vp, k_descale=kd, v_scale=vs,
                  kv_layout=lay, dev_status=status)
    q8, qd = bsa.quantize_rows(q)
    used = i32(lens)
    o, lse = bsa.prefill(q8, kp, vp, qd, kd, vs, cu, used, table, max(lens), max(lens),
                         kv_layout=lay, dev_status=status)
    # a decode of the prompts' last rows sees the same keys as the prefill's last rows
    last = [sum(lens[:b + 1]) - 1 for b in range(B)]
    o1, lse1 = bsa.decode(q8[last], kp, vp, kd, vs, used, table, max(lens), q_descale=qd[last],
                          kv_layout=lay, dev_status=status)
    assert (lse1 - lse[:, last]).abs().max() < 1e-3
    # the prefill rounds its probabilities to e4m3: 2^-4 of each, of values up to 5
    assert (o1.float() - o[last].float()).abs().max() < 2.0 ** -4 * 5
    for step in range(3):
        k1, v1, q1 = rand(B, N2, 128), rand(B, N2, 128), rand(B, N1, 128)
        bsa.append_kv(k1, v1, i32([0, 1, 2, 3]), used, table, kp, vp, k_descale=kd, v_scale=vs,
                      kv_layout=lay, dev_status=status)
        used += 1
        top = max(lens) + step + 1
        o, lse = bsa.decode(q1, kp, vp, kd, vs, used, table, top, kv_layout=lay,
                            dev_status=status)
        n = [x + step + 1 for x in lens]
        kk, vv = bsa.gather_kv(kp, vp, kd, vs, i32(np.cumsum([0] + n)), table, sum(n),
                               out_dtype=torch.float32, kv_layout=lay, dev_status=status)
        at = 0
        for b in range(B):
            kb, vb = (x[at:at + n[b]].double().cpu().repeat_interleave(N1 // N2, 1)
                      for x in (kk, vv))
            at += n[b]
            s = torch.einsum("hd,nhd->hn", q1[b].double().cpu(), kb) / np.sqrt(128)
            p = torch.softmax(s, 1)
            want = torch.einsum("hn,nhd->hd", p, vb)
            size = torch.einsum("hn,nhd->hd", p, vb.abs())
            # half a bf16 step of the result; fp16 probabilities and fp32 scores (|s| sums < 2^5)
            bound = 2.0 ** -8 * want.abs() + 2.0 ** -10 * size
            assert ((o[b].double().cpu() - want).abs() <= bound).all()
            assert (lse[:, b].double().cpu() - torch.logsumexp(s, 1)).abs().max() < 1e-4
        Kb = -(-top // 128)
        first = torch.zeros(B, N1, Kb, dtype=torch.uint8, device="cuda")
        first[:, :, ::2] = 1
        first[:, 1] = 1 - first[:, 1]
        halves = [bsa.decode(q1, kp, vp, kd, vs, used, table, top, block_mask=m, kv_layout=lay,
                             dev_status=status) for m in (first, 1 - first)]
        om, lm = bsa.merge_states([x[0] for x in halves], [x[1] for x in halves])
        # each half is off by half a bf16 step of its own, values up to 5 in the sequences
        assert (om.float() - o.float()).abs().max() < 3 * 2.0 ** -8 * 5
        assert (lm - lse).abs().max() < 1e-4
    assert int(status.item()) == 0
