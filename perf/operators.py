"""The serving operators beside the prefill: measured cases, plain forms and exact results.

Three operators over the paged e4m3 cache that ``append_kv`` writes and ``prefill`` reads:

* ``decode``        attention of one new token per sequence over the whole cache
* ``gather_kv``     the cache read back into contiguous bf16 / fp32 rows
* ``merge_states``  the join of attention results (O, LSE) over disjoint parts of a cache

``run`` with ``own`` false is the plain form: elementary torch operations in fp32, rounded once.
With ``own`` true it makes the calls a user of ``block_sparse_fp8_gb300`` makes.
"""
import math

import numpy as np
import torch

own = False

D = 128
TILE = 128
NO_KEY = torch.finfo(torch.float32).min      # LSE of a row without a visible key


def listed():
    return [
        # one chat turn just begun: a single short sequence, where latency is all
        dict(name="decode_first_tokens", op="decode", B=1, N1=32, N2=8, ps=64, lo=300, hi=300,
             empty=False, q8=False, k_tok=True, v_head=True, nhd=False, sparse="", keep=1.0),
        # a small mixed batch, lengths from one token to some thousands, one slot idle
        dict(name="decode_ragged_16", op="decode", B=16, N1=32, N2=8, ps=32, lo=1, hi=4097,
             empty=True, q8=True, k_tok=True, v_head=True, nhd=True, sparse="", keep=1.0),
        # a full serving batch at the lengths of the default prefill workload
        dict(name="decode_batch_64", op="decode", B=64, N1=64, N2=8, ps=32, lo=8200, hi=16384,
             empty=False, q8=False, k_tok=True, v_head=True, nhd=False, sparse="", keep=1.0),
        # two users with very long contexts: the cache's length has to be split
        dict(name="decode_long_2x128k", op="decode", B=2, N1=32, N2=4, ps=64, lo=131071, hi=131071,
             empty=False, q8=False, k_tok=False, v_head=False, nhd=False, sparse="", keep=1.0),
        # block-sparse decode: each KV head's query heads share a list of a quarter of the tiles
        dict(name="decode_index_8x64k", op="decode", B=8, N1=64, N2=8, ps=32, lo=50000, hi=65536,
             empty=False, q8=True, k_tok=True, v_head=True, nhd=False, sparse="index", keep=0.25),
        # block mask, a pattern for every query head, some heads with nothing enabled, 16 to 1
        dict(name="decode_mask_4x16k", op="decode", B=4, N1=32, N2=2, ps=64, lo=3000, hi=16384,
             empty=False, q8=False, k_tok=True, v_head=True, nhd=False, sparse="mask", keep=0.2),
        # a short system prompt taken out of the cache
        dict(name="gather_prompt", op="gather", B=1, N2=8, ps=64, lo=77, hi=77, start=0,
             k_tok=True, v_head=True, nhd=False, f32=False),
        # the tails of a mixed batch behind a common prefix
        dict(name="gather_tails_8", op="gather", B=8, N2=8, ps=32, lo=100, hi=5000, start=1000,
             k_tok=False, v_head=True, nhd=False, f32=True),
        # whole long sequences, moved to a bf16 cache elsewhere
        dict(name="gather_4x64k", op="gather", B=4, N2=8, ps=64, lo=65536, hi=65536, start=0,
             k_tok=True, v_head=True, nhd=True, f32=False),
        # decode rows over a shared prefix joined with the rows over each one's own suffix
        dict(name="merge_decode_16", op="merge", T=16, N1=32, n=2, empty=0.1),
        # a prefill chunk over the cache before it and over itself
        dict(name="merge_chunk_8k", op="merge", T=8192, N1=32, n=2, empty=0.05),
        # a long prefill over a context that was cut into five
        dict(name="merge_context_5", op="merge", T=16384, N1=64, n=5, empty=0.05),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "gather", "merge"])
    if op == "decode":
        N2 = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 5, 7, 8, 16])
        B = _log_int(rng, 1, 64)
        # token-heads of the padded batch at most those of the full serving batch
        top = min(131071, (64 * 8 * 12000) // (B * N2 * max(1, G // 8)))
        hi = _log_int(rng, 100, max(top, 200))
        lo = rng.choice([1, hi // 2 + 1, hi])
        sparse = rng.choice(["", "", "index", "mask"])
        return dict(op=op, B=B, N1=N2 * G, N2=N2, ps=rng.choice([32, 64]), lo=lo, hi=hi,
                    empty=B > 2 and rng.random() < 0.3, q8=rng.random() < 0.5,
                    k_tok=rng.random() < 0.7, v_head=rng.random() < 0.7, nhd=rng.random() < 0.4,
                    sparse=sparse, keep=rng.choice([0.1, 0.25, 0.5]) if sparse else 1.0)
    if op == "gather":
        N2 = rng.choice([1, 2, 4, 8])
        B = _log_int(rng, 1, 32)
        hi = _log_int(rng, 30, max(60, min(65536, 2000000 // (B * N2))))
        return dict(op=op, B=B, N2=N2, ps=rng.choice([32, 64]), lo=rng.choice([1, hi // 2 + 1, hi]),
                    hi=hi, start=rng.choice([0, 1, 129, 1000]), k_tok=rng.random() < 0.6,
                    v_head=rng.random() < 0.6, nhd=rng.random() < 0.5, f32=rng.random() < 0.4)
    n = rng.choice([2, 2, 3, 4, 5, 8])
    N1 = rng.choice([1, 8, 24, 32, 64])
    return dict(op=op, T=_log_int(rng, 1, 1000000 * 5 // (N1 * n)), N1=N1, n=n,
                empty=rng.choice([0.0, 0.05, 0.5]))


def lengths(case):
    """The sequences' lengths: spread over [lo, hi] by multiples of the golden ratio, the first
    the longest; an idle slot has none."""
    lo, hi, B = case["lo"], case["hi"], case["B"]
    lens = [hi] + [lo + int((hi - lo + 1) * ((b * 0.6180339887498949) % 1.0)) for b in range(1, B)]
    if case.get("empty"):
        lens[B // 2] = 0
    return lens


def _kept(case, n):
    """Tiles of an n-tile sequence on one list."""
    return min(n, max(2, math.ceil(case["keep"] * n)))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _quantise(x):
    """fp32 rows -> (e4m3 codes as bytes, descale amax / 448)."""
    d = x.abs().amax(-1, keepdim=True) / 448.0
    d = torch.where(d > 0, d, torch.ones_like(d))
    return (x / d).to(torch.float8_e4m3fn).view(torch.uint8), d[..., 0]


def _cache(case, lens, gen):
    """A pool of pages in shuffled order holding `lens` tokens of each sequence."""
    B, N2, ps = case["B"], case["N2"], case["ps"]
    per = [-(-n // ps) for n in lens]
    L = max(max(per), 1)
    P = sum(per) + 3
    perm = torch.randperm(P, generator=gen, device="cuda")
    table = torch.zeros(B, L, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n].int()
        at += n
    k_pages = torch.empty(P, N2, ps, D, dtype=torch.uint8, device="cuda")
    v_pages = torch.empty_like(k_pages)
    kd = torch.empty(P, N2, ps, dtype=torch.float32, device="cuda")
    channel = torch.ones(N2, 1, D, device="cuda")
    channel[:, 0, ::61] = 4.0                               # channels that stand out
    v_scale = 0.5 + torch.arange(N2, device="cuda") / N2     # heads of unlike size
    v_desc = v_scale * (6.0 / 448.0)
    if not case["v_head"]:
        v_desc = v_desc.amax().reshape(1)
    k_desc1 = torch.full((1,), 6.0 * 4.0 / 448.0, device="cuda")
    step = max(1, (1 << 27) // (N2 * ps * D))
    for p0 in range(0, P, step):
        m = min(step, P - p0)
        x = torch.randn(m, N2, ps, D, generator=gen, device="cuda") * channel
        if case["k_tok"]:
            k_pages[p0:p0 + m], kd[p0:p0 + m] = _quantise(x)
        else:
            k_pages[p0:p0 + m] = (x / k_desc1).clamp(-448, 448).to(
                torch.float8_e4m3fn).view(torch.uint8)
        x = torch.randn(m, N2, ps, D, generator=gen, device="cuda") * v_scale[:, None, None]
        v_pages[p0:p0 + m] = (x / v_desc.view(-1, 1, 1)).clamp(-448, 448).to(
            torch.float8_e4m3fn).view(torch.uint8)
    # slots past a sequence's last token hold zeros
    for b, n in enumerate(lens):
        if n % ps:
            pg = int(table[b, n // ps])
            k_pages[pg, :, n % ps:] = 0
            v_pages[pg, :, n % ps:] = 0
            kd[pg, :, n % ps:] = 0
    if case["nhd"]:
        k_pages = k_pages.transpose(1, 2).contiguous()
        v_pages = v_pages.transpose(1, 2).contiguous()
    return dict(k_pages=k_pages, v_pages=v_pages, k_descale=kd if case["k_tok"] else k_desc1,
                v_descale=v_desc, block_table=table)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = np.random.default_rng(seed)
    if case["op"] == "merge":
        T, N1, n = case["T"], case["N1"], case["n"]
        outs, lses = [], []
        for _ in range(n):
            o = torch.randn(T, N1, D, generator=gen, device="cuda", dtype=torch.bfloat16) * 0.1
            l = torch.randn(N1, T, generator=gen, device="cuda") * 2.0 + 8.0
            gone = torch.rand(N1, T, generator=gen, device="cuda") < case["empty"]
            o[gone.t()] = 0
            outs.append(o)
            lses.append(torch.where(gone, torch.full_like(l, NO_KEY), l))
        return dict(outs=outs, lses=lses)
    lens = lengths(case)
    if case["op"] == "gather":
        start = case["start"]
        s = _cache(case, [start + n for n in lens], gen)
        s["cu_seqlens"] = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
        s["cache_starts"] = torch.full((case["B"],), start, dtype=torch.int32, device="cuda")
        s["total"] = sum(lens)
        return s
    B, N1, N2 = case["B"], case["N1"], case["N2"]
    G = N1 // N2
    s = _cache(case, lens, gen)
    q = torch.randn(B, N1, D, generator=gen, device="cuda") * 1.5
    if case["q8"]:
        s["q"], s["q_descale"] = _quantise(q)
    else:
        s["q"], s["q_descale"] = q.to(torch.bfloat16), None
    s["seqused_kv"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["max_kv_len"] = max(lens)
    s["block_mask"] = s["sparse_indices"] = s["sparse_seq_len"] = None
    Kb = -(-max(lens) // TILE)
    if case["sparse"] == "index":
        idx = np.full((B, N1, Kb), -1, dtype=np.int32)
        cnt = np.zeros((B, N1), dtype=np.int32)
        for b, n in enumerate(lens):
            nt = -(-n // TILE)
            m = _kept(case, nt)
            for g in range(N2):
                if m:
                    # the first and the last tile, and others at random, in no order
                    mid = host.permutation(max(nt - 2, 0))[:max(m - 2, 0)] + 1
                    t = np.concatenate([[0, nt - 1][:m], mid]) if nt > 1 else np.zeros(1)
                    idx[b, g * G:(g + 1) * G, :m] = host.permutation(t)
            cnt[b] = m
        s["sparse_indices"] = torch.from_numpy(idx).cuda()
        s["sparse_seq_len"] = torch.from_numpy(cnt).cuda()
    elif case["sparse"] == "mask":
        mask = (host.random((B, N1, Kb)) < case["keep"]).astype(np.uint8)
        mask[:, :, 0] = 1
        for b, n in enumerate(lens):
            mask[b, :, max(-(-n // TILE) - 1, 0):] = 1
        mask[0, 0] = 0                                       # a head with nothing enabled
        s["block_mask"] = torch.from_numpy(mask).cuda()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import block_sparse_fp8_gb300 as bsa

    # what a serving loop keeps from step to step: outputs, workspace, status word
    if case["op"] == "decode":
        B, N1 = case["B"], case["N1"]
        layout = bsa.KV_NHD if case["nhd"] else bsa.KV_HND
        k_kind = bsa.SCALE_PER_TOKEN_HEAD if case["k_tok"] else bsa.SCALE_PER_TENSOR
        v_kind = bsa.SCALE_PER_HEAD if case["v_head"] else bsa.SCALE_PER_TENSOR
        dims = bsa.make_decode_dims(s["q"], s["k_pages"], s["block_table"], s["max_kv_len"], k_kind,
                                    v_kind, kv_layout=layout, sparse=bool(case["sparse"]))
        s["kinds"] = dict(k_scale_kind=k_kind, v_scale_kind=v_kind, kv_layout=layout)
        s["workspace"] = torch.empty(bsa.decode_workspace_size(dims), dtype=torch.uint8,
                                     device="cuda")
        s["out"] = torch.empty(B, N1, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(N1, B, dtype=torch.float32, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    elif case["op"] == "gather":
        s["kinds"] = dict(
            k_scale_kind=bsa.SCALE_PER_TOKEN_HEAD if case["k_tok"] else bsa.SCALE_PER_TENSOR,
            v_scale_kind=bsa.SCALE_PER_HEAD if case["v_head"] else bsa.SCALE_PER_TENSOR,
            kv_layout=bsa.KV_NHD if case["nhd"] else bsa.KV_HND)
        dtype = torch.float32 if case["f32"] else torch.bfloat16
        s["k_out"] = torch.empty(s["total"], case["N2"], D, dtype=dtype, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        s["out"] = torch.empty_like(s["outs"][0])
        s["lse"] = torch.empty_like(s["lses"][0])
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"decode": _own_decode, "gather": _own_gather, "merge": _own_merge}[op](state)
    return {"decode": _plain_decode, "gather": _plain_gather, "merge": _plain_merge}[op](state)


def _own_decode(s):
    import block_sparse_fp8_gb300 as bsa

    return bsa.decode(s["q"], s["k_pages"], s["v_pages"], s["k_descale"], s["v_descale"],
                      s["seqused_kv"], s["block_table"], s["max_kv_len"], q_descale=s["q_descale"],
                      block_mask=s["block_mask"], sparse_indices=s["sparse_indices"],
                      sparse_seq_len=s["sparse_seq_len"], out=s["out"], lse=s["lse"],
                      dev_status=s["status"], workspace=s["workspace"], **s["kinds"])


def _own_gather(s):
    import block_sparse_fp8_gb300 as bsa

    return bsa.gather_kv(s["k_pages"], s["v_pages"], s["k_descale"], s["v_descale"],
                         s["cu_seqlens"], s["block_table"], s["total"],
                         cache_starts=s["cache_starts"], k_out=s["k_out"], v_out=s["v_out"],
                         dev_status=s["status"], **s["kinds"])


def _own_merge(s):
    import block_sparse_fp8_gb300 as bsa

    return bsa.merge_states(s["outs"], s["lses"], out=s["out"], lse=s["lse"])


def _values(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float32)


def _plain_decode(s):
    case = s["case"]
    B, N1, N2, ps = case["B"], case["N1"], case["N2"], case["ps"]
    G = N1 // N2
    L = s["block_table"].shape[1]
    n = L * ps
    pages = s["block_table"].long()
    token = torch.arange(n, device="cuda")
    live = token < s["seqused_kv"][:, None]                            # [B, n]
    k, v = s["k_pages"][pages], s["v_pages"][pages]                    # [B, L, ...]
    if case["nhd"]:
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    k = _values(k).transpose(1, 2).reshape(B, N2, n, D)
    q = _values(s["q"]) * s["q_descale"][..., None] if case["q8"] else s["q"].float()
    x = torch.matmul(q.view(B, N2, G, D), k.transpose(2, 3))           # [B, N2, G, n]
    del k
    if case["k_tok"]:
        x = x * s["k_descale"][pages].transpose(1, 2).reshape(B, N2, 1, n)
    else:
        x = x * s["k_descale"]
    x = x * (1.0 / math.sqrt(D))
    on = live[:, None, None, :]
    Kb = -(-s["max_kv_len"] // TILE)
    mask = s["block_mask"]
    if s["sparse_indices"] is not None:
        taken = torch.arange(Kb, device="cuda") < s["sparse_seq_len"][..., None]
        # entries past a list's length go to a tile that does not exist
        idx = torch.where(taken, s["sparse_indices"], torch.full_like(s["sparse_indices"], Kb))
        mask = torch.zeros(B, N1, Kb + 1, dtype=torch.uint8, device="cuda")
        mask.scatter_(2, idx.long(), 1)
    if mask is not None:
        tile = (token // TILE).clamp(max=Kb - 1)
        on = on & (mask[:, :, tile] != 0).view(B, N2, G, n)
    x = torch.where(on, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    del x
    total = p.sum(-1, keepdim=True)
    v = _values(v).transpose(1, 2).reshape(B, N2, n, D)
    v = torch.where(live[:, None, :, None], v, torch.zeros_like(v))
    o = torch.matmul(p, v)
    some = total > 0
    o = torch.where(some, o / torch.where(some, total, torch.ones_like(total)), torch.zeros_like(o))
    o = o * (s["v_descale"].view(1, N2, 1, 1) if case["v_head"] else s["v_descale"])
    lse = torch.where(some, m + torch.log(total), torch.full_like(m, NO_KEY))
    return o.view(B, N1, D).to(torch.bfloat16), lse.view(B, N1).t().contiguous()


def _plain_gather(s):
    case = s["case"]
    ps = case["ps"]
    row = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(s["cu_seqlens"].long(), row, right=True) - 1
    pos = row - s["cu_seqlens"].long()[seq] + s["cache_starts"].long()[seq]
    page = s["block_table"][seq, pos // ps].long()
    slot = pos % ps
    at = (page, slot) if case["nhd"] else (page, slice(None), slot)
    dtype = torch.float32 if case["f32"] else torch.bfloat16
    k = _values(s["k_pages"][at])
    k = k * (s["k_descale"][page, :, slot][..., None] if case["k_tok"] else s["k_descale"])
    v = _values(s["v_pages"][at])
    v = v * (s["v_descale"][:, None] if case["v_head"] else s["v_descale"])
    return k.to(dtype), v.to(dtype)


def _plain_merge(s):
    l = torch.stack(s["lses"])                                         # [n, N1, T]
    m = l.amax(0)
    w = torch.where(l == NO_KEY, torch.zeros_like(l), torch.exp(l - m))
    total = w.sum(0)
    some = total > 0
    w = w / torch.where(some, total, torch.ones_like(total))
    o = torch.zeros(s["outs"][0].shape, dtype=torch.float32, device="cuda")
    for i, part in enumerate(s["outs"]):
        o = o + w[i].t()[..., None] * part.float()
    lse = torch.where(some, m + torch.log(torch.where(some, total, torch.ones_like(total))),
                      torch.full_like(m, NO_KEY))
    return o.to(torch.bfloat16), lse


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------------------------

def _e4m3_table():
    """The value of each e4m3 byte, from its sign, exponent and fraction."""
    val = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if (c & 127) == 127:
            x = math.nan
        val.append(-x if c & 128 else x)
    return torch.tensor(val, dtype=torch.float64, device="cuda")


def _sequence(s, case, table, b, first, n, which):
    """Rows first .. first + n of sequence b: fp64 [N2, n, D]."""
    ps = case["ps"]
    l0, l1 = first // ps, -(-(first + n) // ps)
    pg = s["block_table"][b, l0:l1].long()
    c = table[s[which + "_pages"][pg].long()]                          # [pages, ...]
    c = c.permute(2, 0, 1, 3) if case["nhd"] else c.permute(1, 0, 2, 3)
    c = c.reshape(case["N2"], -1, D)
    if which == "v":
        c = c * s["v_descale"].double().view(-1, 1, 1)
    elif case["k_tok"]:
        c = c * s["k_descale"][pg].double().permute(1, 0, 2).reshape(case["N2"], -1, 1)
    else:
        c = c * s["k_descale"].double()
    off = first - l0 * ps
    return c[:, off:off + n]


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "merge":
        l = torch.stack([x.double() for x in s["lses"]], -1)           # [N1, T, n]
        l[l == NO_KEY] = -math.inf
        lse = torch.logsumexp(l, -1)
        out = torch.zeros(case["T"], case["N1"], D, dtype=torch.float64, device="cuda")
        for i, part in enumerate(s["outs"]):
            w = torch.exp(l[..., i] - lse)
            w[lse == -math.inf] = 0
            out += w.t().unsqueeze(-1) * part.double()
        lse[lse == -math.inf] = NO_KEY
        return out, lse
    table = _e4m3_table()
    lens = lengths(case)
    if case["op"] == "gather":
        both = []
        for which in "kv":
            rows = [_sequence(s, case, table, b, case["start"], n, which).transpose(0, 1)
                    for b, n in enumerate(lens) if n]
            both.append(torch.cat(rows))
        return tuple(both)
    B, N1, N2 = case["B"], case["N1"], case["N2"]
    G = N1 // N2
    out = torch.zeros(B, N1, D, dtype=torch.float64, device="cuda")
    lse = torch.full((N1, B), NO_KEY, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        q = table[s["q"][b].long()] * s["q_descale"][b].double()[:, None] if case["q8"] else \
            s["q"][b].double()
        k = _sequence(s, case, table, b, 0, n, "k")
        x = torch.einsum("hgd,hnd->hgn", q.view(N2, G, D), k).reshape(N1, n) / math.sqrt(D)
        del k
        nt = -(-n // TILE)
        if case["sparse"]:
            on = torch.zeros(N1, nt, dtype=torch.bool, device="cuda")
            if case["sparse"] == "mask":
                on = s["block_mask"][b, :, :nt] != 0
            else:
                for h in range(N1):
                    on[h, s["sparse_indices"][b, h, :_kept(case, nt)].long()] = True
            x[~on.repeat_interleave(TILE, 1)[:, :n]] = -math.inf
        z = torch.logsumexp(x, -1)
        some = z > -math.inf
        p = torch.exp(x - z[:, None])
        p[~some] = 0
        v = _sequence(s, case, table, b, 0, n, "v")
        out[b] = torch.einsum("hgn,hnd->hgd", p.view(N2, G, n), v).reshape(N1, D)
        lse[some, b] = z[some]
    return out, lse


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "merge":
        rows = case["T"] * case["N1"]
        return dict(bytes=rows * (case["n"] + 1) * (2 * D + 4), flops=rows * case["n"] * 2 * D)
    lens = lengths(case)
    N2, ps = case["N2"], case["ps"]
    desc = 4 if case["k_tok"] else 0
    if case["op"] == "gather":
        rows = sum(lens) * N2
        table = sum(-(-n // ps) for n in lens) * 4
        return dict(bytes=rows * (2 * D + desc + 2 * D * (4 if case["f32"] else 2)) + table,
                    flops=rows * 2 * D)
    B, N1 = case["B"], case["N1"]
    G = N1 // N2
    size = 0.0                                   # tokens of a KV head that some query head needs
    pairs = 0.0                                  # (query head, token) pairs
    lists = 0
    for n in lens:
        nt = -(-n // TILE)
        if case["sparse"] == "index":
            # the last tile, on every list, may be short
            t = _kept(case, nt) * TILE - (nt * TILE - n)
            size += t * N2
            pairs += t * N1
            lists += _kept(case, nt) * 4 * N1
        elif case["sparse"] == "mask":
            size += n * N2 * (1 - (1 - case["keep"]) ** G)
            pairs += n * N1 * case["keep"]
            lists += nt * N1
        else:
            size += n * N2
            pairs += n * N1
    nbytes = size * (2 * D + desc) + lists + sum(-(-n // ps) for n in lens) * 4
    nbytes += B * N1 * (D * (1 if case["q8"] else 2) + (4 if case["q8"] else 0) + 2 * D + 4)
    return dict(bytes=int(nbytes), flops=int(pairs * 4 * D))
