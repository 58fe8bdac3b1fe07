"""What a serving loop runs around attention: measured cases, plain forms and exact results.

* ``rope`` / ``rope_quantize``        rotary positions of Q and K, and of Q on its way to e4m3
* ``assign_pages`` / ``release_pages``  block tables and slot maps from the requests' lengths
* ``append_kv_fp4`` / ``gather_kv_fp4``  tokens into a cache held in 4 bits, and out of it again
* ``decode_fp4``                      attention of one new token per sequence over that cache

The 4-bit cache: e2m1 codes, two to a byte, an e4m3 scale for every 16 of them, and one fp32 descale
per tensor or KV head: value = code * scale * descale.

``run`` with ``own`` false is the plain form: elementary torch operations in fp32 (the angles in
fp64), rounded once.  With ``own`` true it makes the calls a user of ``block_sparse_fp8_gb300`` makes.
"""
import math

import numpy as np
import torch

own = False

D = 128
TILE = 128
BLOCK = 16                                   # codes to a scale
NO_KEY = torch.finfo(torch.float32).min      # LSE of a row without a visible key
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # a decode step of a small batch: one token each, anywhere in its context
        dict(name="rope_step_16", op="rope", T=16, N1=32, N2=8, R=128, inter=False, far=40000,
             scaling="none", factor=1.0),
        # a prefill chunk far into a stretched context, half of each head rotated in pairs
        dict(name="rope_chunk_8k", op="rope", T=8192, N1=32, N2=8, R=64, inter=True, far=500000,
             scaling="parts", factor=8.0),
        # the queries of a decode step on their way to e4m3
        dict(name="rope_q8_step_64", op="ropeq", T=64, N1=64, R=128, inter=False, far=130000,
             scaling="linear", factor=4.0, ue8m0=True),
        # the queries of a long prefill on their way to e4m3
        dict(name="rope_q8_16k", op="ropeq", T=16384, N1=64, R=128, inter=False, far=16384,
             scaling="none", factor=1.0, ue8m0=False),
        # a decode step of a full server: a token or none each, taken back once (a rejected draft)
        dict(name="pages_step_256", op="pages", B=256, ps=32, lo=0, hi=1, old=16000),
        # prompts admitted at once, and taken back (a batch that is put off)
        dict(name="pages_prompts_64", op="pages", B=64, ps=64, lo=700, hi=16384, old=0),
        # a decode step's tokens stored, and read back
        dict(name="store_step_64", op="store", T=64, N2=8, ps=64, B=64, nhd=False, head=True),
        # prompts stored, and read back for a prefill of what follows them
        dict(name="store_prompts_64k", op="store", T=65537, N2=8, ps=32, B=7, nhd=True, head=False),
        # one chat turn just begun: a single short sequence, where latency is all
        dict(name="decode4_first_tokens", op="decode", B=1, N1=32, N2=8, ps=64, lo=300, hi=300,
             empty=False, q8=False, head=True, nhd=False, sparse="", keep=1.0),
        # a full serving batch at the lengths of the default prefill workload
        dict(name="decode4_batch_64", op="decode", B=64, N1=64, N2=8, ps=32, lo=8200, hi=16384,
             empty=False, q8=False, head=True, nhd=False, sparse="", keep=1.0),
        # two users with very long contexts: the cache's length has to be split
        dict(name="decode4_long_2x128k", op="decode", B=2, N1=32, N2=4, ps=64, lo=131071, hi=131071,
             empty=False, q8=True, head=False, nhd=True, sparse="", keep=1.0),
        # block-sparse decode: each KV head's query heads share a list of a quarter of the tiles
        dict(name="decode4_index_8x64k", op="decode", B=8, N1=64, N2=8, ps=32, lo=50000, hi=65536,
             empty=True, q8=True, head=True, nhd=False, sparse="index", keep=0.25),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rope(rng, heads):
    return dict(T=_log_int(rng, 1, 800000 // heads), R=rng.choice([16, 32, 64, 80, 96, 128, 128]),
                inter=rng.random() < 0.4, far=_log_int(rng, 100, 1000000),
                **rng.choice([dict(scaling="none", factor=1.0), dict(scaling="linear", factor=4.0),
                              dict(scaling="base", factor=2.0), dict(scaling="parts", factor=8.0)]))


def draw(rng):
    op = rng.choice(["rope", "ropeq", "pages", "store", "decode", "decode", "decode"])
    if op == "rope":
        N2 = rng.choice([1, 2, 4, 5, 8])
        N1 = N2 * rng.choice([1, 3, 4, 8])
        return dict(op=op, N1=N1, N2=N2, **_draw_rope(rng, N1 + N2))
    if op == "ropeq":
        N1 = rng.choice([1, 7, 8, 24, 32, 64])
        more = _draw_rope(rng, N1)
        # descales that are powers of two for few rows only: among a million rows there is one whose
        # largest value lies next to such a power, and the last bit of a sine decides
        return dict(op=op, N1=N1, ue8m0=rng.random() < 0.5 and more["T"] * N1 <= 5000, **more)
    if op == "pages":
        B = _log_int(rng, 1, 2000)
        hi = _log_int(rng, 1, max(1, min(65536, 600000 // B)))
        return dict(op=op, B=B, ps=rng.choice([32, 64]), lo=rng.choice([0, hi // 2, hi]), hi=hi,
                    old=rng.choice([0, 100, min(16000, 4000000 // B)]))
    if op == "store":
        N2 = rng.choice([1, 2, 4, 8])
        T = _log_int(rng, 1, 524288 // N2)
        return dict(op=op, T=T, N2=N2, ps=rng.choice([32, 64]), B=min(T, _log_int(rng, 1, 64)),
                    nhd=rng.random() < 0.5, head=rng.random() < 0.6)
    N2 = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 7, 8, 16])
    B = _log_int(rng, 1, 64)
    # token-heads of the padded batch at most those of the full serving batch
    top = min(131071, (64 * 8 * 12000) // (B * N2 * max(1, G // 8)))
    hi = _log_int(rng, 100, max(top, 200))
    sparse = rng.choice(["", "", "index", "mask"])
    return dict(op=op, B=B, N1=N2 * G, N2=N2, ps=rng.choice([32, 64]),
                lo=rng.choice([1, hi // 2 + 1, hi]), hi=hi, empty=B > 2 and rng.random() < 0.3,
                q8=rng.random() < 0.5, head=rng.random() < 0.7, nhd=rng.random() < 0.4,
                sparse=sparse, keep=rng.choice([0.1, 0.25, 0.5]) if sparse else 1.0)


def lengths(case):
    """The sequences' lengths: spread over [lo, hi] by multiples of the golden ratio, the first
    the longest; an idle slot has none."""
    lo, hi, B = case["lo"], case["hi"], case["B"]
    lens = [hi] + [lo + int((hi - lo + 1) * ((b * 0.6180339887498949) % 1.0)) for b in range(1, B)]
    if case.get("empty"):
        lens[B // 2] = 0
    return lens


def _shares(total, B):
    """`total` tokens in B unlike shares of one at least."""
    extra = total - B
    at = [extra * b * (b + 3) // (B * (B + 3)) for b in range(B + 1)]
    return [1 + at[b + 1] - at[b] for b in range(B)]


def _kept(case, n):
    """Tiles of an n-tile sequence on one list."""
    return min(n, max(2, math.ceil(case["keep"] * n)))


# ---------------------------------------------------------------------------------------------
# rotary frequencies, in radians a position
# ---------------------------------------------------------------------------------------------

BASE, CONTEXT, SLOW, FAST = 10000.0, 8192, 1.0, 32.0


def _inv_freq(case):
    R, s = case["R"], case["factor"]
    base = BASE * s ** (R / (R - 2)) if case["scaling"] == "base" else BASE
    f = torch.tensor([base ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float64)
    if case["scaling"] == "linear":
        f = f / s
    elif case["scaling"] == "parts":
        # as trained where a dimension turns often within the context, stretched where hardly once
        w = ((CONTEXT * f / (2 * math.pi) - SLOW) / (FAST - SLOW)).clamp(0, 1)
        f = f * w + f / s * (1 - w)
    return f.cuda()


def _amplitude(case):
    return 1.0 + 0.1 * math.log(case["factor"]) if case["scaling"] == "parts" else 1.0


# ---------------------------------------------------------------------------------------------
# four bits
# ---------------------------------------------------------------------------------------------

def _e2m1(y):
    """The nearest e2m1 code of each value, ties to the even code, 6 the largest."""
    a = y.abs()
    c = (a > 0.25).to(torch.uint8)
    for at, closed in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                       (5.0, False)):
        c += (a >= at) if closed else (a > at)
    return c + 8 * (y < 0).to(torch.uint8)


def _quantise4(x, g):
    """fp32 [..., 128], descale (broadcast) -> packed codes [..., 64], scales as bytes [..., 8].
    The quotients in fp64: descales are often some largest value over 6 * 448, a multiple of 7, and
    then many values lie next to the borders at 7/4 and 7/2."""
    b = x.unflatten(-1, (D // BLOCK, BLOCK))
    g = torch.as_tensor(g, dtype=torch.float64, device=x.device)[..., None]
    t = (b.abs().amax(-1) / (g * 6.0)).clamp(max=448.0)
    # to fp32 by cutting off, with the last bit set where something was cut off: what is next to a
    # border between two scales stays on its side of it
    s = t.to(torch.float32)
    s = torch.where(s.double() > t, torch.nextafter(s, torch.zeros_like(s)), s)
    s = (s.view(torch.int32) | (s.double() < t).to(torch.int32)).view(torch.float32)
    s = s.to(torch.float8_e4m3fn)
    d = (s.to(torch.float64) * g)[..., None]
    c = _e2m1(torch.where(d > 0, b / torch.where(d > 0, d, torch.ones_like(d)),
                          torch.zeros_like(d))).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), s.view(torch.uint8)


def _values4(codes, scales):
    """Packed codes [..., 64] and scales [..., 8] -> fp32 [..., 128], without the descale."""
    level = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = level[c.int()].unflatten(-1, (D // BLOCK, BLOCK))
    return (v * scales.view(torch.float8_e4m3fn).to(torch.float32)[..., None]).flatten(-2)


def _quantise8(x):
    """fp32 rows -> (e4m3 codes as bytes, descale amax / 448)."""
    d = x.abs().amax(-1, keepdim=True) / 448.0
    d = torch.where(d > 0, d, torch.ones_like(d))
    return (x / d).to(torch.float8_e4m3fn).view(torch.uint8), d[..., 0]


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _tables(lens, ps, gen, spare=3):
    """Pages of `lens` tokens in shuffled order: table [B, L], pages in all."""
    per = np.array([-(-n // ps) for n in lens])
    P, L = int(per.sum()) + spare, max(int(per.max()), 1)
    perm = torch.randperm(P, generator=gen, device="cuda").int()
    first = torch.from_numpy(np.cumsum(per) - per).cuda()
    col = torch.arange(L, device="cuda")
    held = col < torch.from_numpy(per).cuda()[:, None]
    at = (first[:, None] + col).clamp(max=P - 1)
    return torch.where(held, perm[at], torch.zeros_like(perm[at])), P, perm


def _cache4(case, lens, gen):
    """A pool of 4-bit pages in shuffled order holding `lens` tokens of each sequence."""
    N2, ps = case["N2"], case["ps"]
    table, P, _ = _tables(lens, ps, gen)
    pool = dict(block_table=table)
    channel = torch.ones(N2, 1, D, device="cuda")
    channel[:, 0, ::61] = 4.0                               # channels that stand out
    v_size = 0.5 + torch.arange(N2, device="cuda") / N2      # heads of unlike size
    pool["k_descale"] = torch.full((N2,), 20.0 / (6 * 448), device="cuda")
    pool["v_descale"] = v_size * (6.0 / (6 * 448))
    if not case["head"]:
        pool["k_descale"] = pool["k_descale"][:1].clone()
        pool["v_descale"] = pool["v_descale"].amax().reshape(1)
    step = max(1, (1 << 26) // (N2 * ps * D))
    for which, size in (("k", channel), ("v", v_size[:, None, None])):
        codes = torch.empty(P, N2, ps, D // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(P, N2, ps, D // BLOCK, dtype=torch.uint8, device="cuda")
        for p0 in range(0, P, step):
            m = min(step, P - p0)
            x = torch.randn(m, N2, ps, D, generator=gen, device="cuda") * size
            codes[p0:p0 + m], scales[p0:p0 + m] = _quantise4(
                x, pool[which + "_descale"].view(-1, 1))
        pool[which + "_pages"] = codes.transpose(1, 2).contiguous() if case["nhd"] else codes
        pool[which + "_scales"] = scales
    return pool


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = np.random.default_rng(seed)
    op = case["op"]
    if op in ("rope", "ropeq"):
        T, N1, N2 = case["T"], case["N1"], case.get("N2", 0)
        # q and k as a projection leaves them: side by side, v behind them
        wide = torch.randn(T, N1 + 2 * N2, D, generator=gen, device="cuda", dtype=torch.bfloat16)
        far = torch.randint(0, case["far"] + 1, (), generator=gen, device="cuda")
        pos = (far + torch.arange(T, device="cuda")) % (case["far"] + 1) if T > 256 else \
            torch.randint(0, case["far"] + 1, (T,), generator=gen, device="cuda")
        return dict(q=wide[:, :N1], k=wide[:, N1:N1 + N2], positions=pos.int())
    if op == "pages":
        B, ps = case["B"], case["ps"]
        new = host.permutation(np.array(lengths(case)))
        span = case["old"] - case["old"] // 2 + 1
        old = host.permutation(case["old"] // 2 + (np.arange(B) * 0.6180339887498949 % 1 * span)
                               .astype(np.int64))
        table, P, perm = _tables(list(old), ps, gen, spare=int((-(-new // ps)).sum()) + 5)
        L = max(1, -(-(case["old"] + case["hi"]) // ps))
        wide = torch.full((B, L), -1, dtype=torch.int32, device="cuda")
        n = min(table.shape[1], wide.shape[1])
        per = torch.from_numpy(-(-old // ps)).cuda()
        held = torch.arange(n, device="cuda") < per[:, None]
        wide[:, :n] = torch.where(held, table[:, :n], wide[:, :n])
        used = int((-(-old // ps)).sum())
        free = torch.cat([perm[used:], torch.full((used,), -1, dtype=torch.int32, device="cuda")])
        i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()
        return dict(new_lens=i32(new), cache_seqlens=i32(old), block_table=wide, free_pages=free,
                    free_count=i32([P - used]), total=int(new.sum()) + 3)   # padded by three
    if op == "store":
        T, N2, ps = case["T"], case["N2"], case["ps"]
        lens = _shares(T, case["B"])
        old = [int(x) for x in host.integers(0, 2 * ps, case["B"])]
        table, P, _ = _tables([a + b for a, b in zip(old, lens)], ps, gen)
        seq = torch.from_numpy(np.repeat(np.arange(case["B"]), lens)).cuda()
        cu = torch.tensor(np.cumsum([0] + lens), device="cuda")
        starts = torch.tensor(old, device="cuda")
        pos = torch.arange(T, device="cuda") - cu[seq] + starts[seq]
        slot = table[seq, pos // ps].long() * ps + pos % ps
        wide = torch.randn(T, 2 * N2, D, generator=gen, device="cuda", dtype=torch.bfloat16)
        head = N2 if case["head"] else 1
        g = (0.6 + torch.arange(head, device="cuda") / head) * (5.0 / (6 * 448))
        return dict(k=wide[:, :N2].contiguous(), v=wide[:, N2:], slot_map=slot.int(), pages=P,
                    block_table=table, cu_seqlens=cu.int(), cache_starts=starts.int(),
                    k_descale=g, v_descale=g * 1.25)
    lens = lengths(case)
    B, N1, N2 = case["B"], case["N1"], case["N2"]
    G = N1 // N2
    s = _cache4(case, lens, gen)
    q = torch.randn(B, N1, D, generator=gen, device="cuda") * 1.5
    if case["q8"]:
        s["q"], s["q_descale"] = _quantise8(q)
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
            for g in range(N2 if m else 0):
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
    op = case["op"]
    # what a serving loop keeps from step to step: frequencies, pool, outputs, workspace, status word
    if op in ("rope", "ropeq"):
        s["inv_freq"] = _inv_freq(case)
    if op == "store":
        shape = (s["pages"], case["ps"], case["N2"]) if case["nhd"] else (
            s["pages"], case["N2"], case["ps"])
        for which in "kv":
            s[which + "_pages"] = torch.zeros(*shape, D // 2, dtype=torch.uint8, device="cuda")
            s[which + "_scales"] = torch.zeros(s["pages"], case["N2"], case["ps"], D // BLOCK,
                                               dtype=torch.uint8, device="cuda")
    if not own:
        return s
    import block_sparse_fp8_gb300 as bsa

    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    layout = bsa.KV_NHD if case.get("nhd") else bsa.KV_HND
    kind = bsa.SCALE_PER_HEAD if case.get("head") else bsa.SCALE_PER_TENSOR
    s["kinds"] = dict(k_scale_kind=kind, v_scale_kind=kind, kv_layout=layout)
    if op in ("rope", "ropeq"):
        scaling = {"none": bsa.ROPE_NONE, "linear": bsa.ROPE_LINEAR, "base": bsa.ROPE_BASE,
                   "parts": bsa.ROPE_PARTS}[case["scaling"]]
        s["freqs"] = bsa.rope_frequencies(case["R"], base=BASE, scaling=scaling,
                                          factor=case["factor"], context=CONTEXT, device="cuda")
        s["how"] = dict(layout=bsa.ROPE_INTERLEAVED if case["inter"] else bsa.ROPE_HALF,
                        amplitude=_amplitude(case))
        if op == "rope":
            s["q_out"] = torch.empty(case["T"], case["N1"], D, dtype=torch.bfloat16, device="cuda")
            s["k_out"] = torch.empty(case["T"], case["N2"], D, dtype=torch.bfloat16, device="cuda")
        else:
            s["codes"] = torch.empty(case["T"], case["N1"], D, dtype=torch.uint8, device="cuda")
            s["descale"] = torch.empty(case["T"], case["N1"], device="cuda")
            s["rule"] = bsa.DESCALE_UE8M0 if case["ue8m0"] else bsa.DESCALE_AMAX
    elif op == "pages":
        B = case["B"]
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
        s["out"] = dict(cu_seqlens=i32(B + 1), seqused_kv=i32(B), positions=i32(s["total"]),
                        slot_map=i32(s["total"]))
        s["left"] = i32(B)
    elif op == "store":
        s["k_out"] = torch.empty(case["T"], case["N2"], D, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
    else:
        B, N1 = case["B"], case["N1"]
        dims = bsa.make_decode_dims(s["q"], s["k_pages"], s["block_table"], s["max_kv_len"], kind,
                                    kind, kv_layout=layout, sparse=bool(case["sparse"]))
        s["workspace"] = torch.empty(bsa.decode_fp4_workspace_size(dims), dtype=torch.uint8,
                                     device="cuda")
        s["out"] = torch.empty(B, N1, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(N1, B, dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "ropeq": _own_ropeq, "pages": _own_pages, "store": _own_store,
                "decode": _own_decode}[op](state)
    return {"rope": _plain_rope, "ropeq": _plain_ropeq, "pages": _plain_pages,
            "store": _plain_store, "decode": _plain_decode}[op](state)


def _own_rope(s):
    import block_sparse_fp8_gb300 as bsa

    return bsa.rope(s["q"], s["positions"], s["freqs"], k=s["k"], out=s["q_out"], k_out=s["k_out"],
                    **s["how"])


def _own_ropeq(s):
    import block_sparse_fp8_gb300 as bsa

    codes, descale = bsa.rope_quantize(s["q"], s["positions"], s["freqs"], codes=s["codes"],
                                       descale=s["descale"], rule=s["rule"], **s["how"])
    return codes.view(torch.float8_e4m3fn), descale


def _own_pages(s):
    import block_sparse_fp8_gb300 as bsa

    o = s["out"]
    bsa.assign_pages(s["new_lens"], s["cache_seqlens"], s["block_table"], s["free_pages"],
                     s["free_count"], s["case"]["ps"], s["total"], dev_status=s["status"], **o)
    bsa.release_pages(o["seqused_kv"], s["cache_seqlens"], s["block_table"], s["free_pages"],
                      s["free_count"], s["case"]["ps"], out=s["left"], dev_status=s["status"])
    return dict(o, left=s["left"], block_table=s["block_table"], free_pages=s["free_pages"],
                free_count=s["free_count"])


def _own_store(s):
    import block_sparse_fp8_gb300 as bsa

    bsa.append_kv_fp4(s["k"], s["v"], s["slot_map"], s["k_pages"], s["v_pages"], s["k_scales"],
                      s["v_scales"], s["k_descale"], s["v_descale"], dev_status=s["status"],
                      **s["kinds"])
    return bsa.gather_kv_fp4(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"],
                             s["k_descale"], s["v_descale"], s["cu_seqlens"], s["block_table"],
                             s["case"]["T"], cache_starts=s["cache_starts"], k_out=s["k_out"],
                             v_out=s["v_out"], dev_status=s["status"], **s["kinds"])


def _own_decode(s):
    import block_sparse_fp8_gb300 as bsa

    return bsa.decode_fp4(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"],
                          s["k_descale"], s["v_descale"], s["seqused_kv"], s["block_table"],
                          s["max_kv_len"], q_descale=s["q_descale"], block_mask=s["block_mask"],
                          sparse_indices=s["sparse_indices"], sparse_seq_len=s["sparse_seq_len"],
                          out=s["out"], lse=s["lse"], dev_status=s["status"],
                          workspace=s["workspace"], **s["kinds"])


def _rotated(x, s):
    """fp32 rows [T, N, 128] of bf16 ones, rotated."""
    case = s["case"]
    R = case["R"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]             # [T, R / 2]
    a = _amplitude(case)
    c = (torch.cos(angle) * a).float()[:, None]
    sn = (torch.sin(angle) * a).float()[:, None]
    x = x.float()
    if case["inter"]:
        u, v = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack((u * c - v * sn, v * c + u * sn), -1).flatten(-2)
    else:
        u, v = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat((u * c - v * sn, v * c + u * sn), -1)
    return torch.cat((turned, x[..., R:]), -1)


def _plain_rope(s):
    return _rotated(s["q"], s).to(torch.bfloat16), _rotated(s["k"], s).to(torch.bfloat16)


def _plain_ropeq(s):
    x = _rotated(s["q"], s)
    d = x.abs().amax(-1, keepdim=True) / 448.0
    if s["case"]["ue8m0"]:
        m, e = torch.frexp(d)                        # d = m 2^e, m in [1/2, 1)
        d = torch.ldexp(torch.ones_like(d), torch.where(m == 0.5, e - 1, e))
    return (x / d).clamp(-448, 448).to(torch.float8_e4m3fn), d[..., 0]


def _plain_pages(s):
    ps, total = s["case"]["ps"], s["total"]
    new, old = s["new_lens"].long(), s["cache_seqlens"].long()
    free = s["free_count"].long()
    have, need = (old + ps - 1) // ps, (old + new + ps - 1) // ps
    want = need - have
    ends = torch.cumsum(want, 0)
    served = ends <= free
    cu = torch.cat((torch.zeros_like(new[:1]), torch.cumsum(new, 0)))
    used = torch.where(served, old + new, old)
    # the pages: the j-th that is taken comes from the j-th place below the stack's top
    table = s["block_table"]
    col = torch.arange(table.shape[1], device="cuda")
    fresh = served[:, None] & (col >= have[:, None]) & (col < need[:, None])
    j = (ends - want)[:, None] + col - have[:, None]
    top = (free - 1 - j).clamp(0, s["free_pages"].numel() - 1)
    table = torch.where(fresh, s["free_pages"][top], table)
    row = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu, row, right=True) - 1
    live = seq < new.numel()
    seq = seq.clamp(max=new.numel() - 1)
    pos = row - cu[seq] + old[seq]
    col = (pos // ps).clamp(max=table.shape[1] - 1)
    slot = torch.where(live & served[seq], table[seq, col].long() * ps + pos % ps,
                       torch.full_like(pos, -1))
    # and all taken back: the same pages to the same places, so that the stack is as it was
    left = torch.minimum(old, used)
    i32 = lambda x: x.to(torch.int32)
    return dict(cu_seqlens=i32(cu), seqused_kv=i32(used),
                positions=i32(torch.where(live, pos, torch.zeros_like(pos))), slot_map=i32(slot),
                left=i32(left), block_table=table, free_pages=s["free_pages"],
                free_count=s["free_count"])


def _at(case, page, slot):
    return (page, slot) if case["nhd"] else (page, slice(None), slot)


def _plain_store(s):
    case = s["case"]
    ps = case["ps"]
    page, slot = s["slot_map"].long() // ps, s["slot_map"].long() % ps
    row = torch.arange(case["T"], device="cuda")
    seq = torch.searchsorted(s["cu_seqlens"].long(), row, right=True) - 1
    pos = row - s["cu_seqlens"].long()[seq] + s["cache_starts"].long()[seq]
    from_page, from_slot = s["block_table"][seq, pos // ps].long(), pos % ps
    got = []
    for which in "kv":
        g = s[which + "_descale"]
        codes, scales = s[which + "_pages"], s[which + "_scales"]
        c, e = _quantise4(s[which].float(), g)
        codes[_at(case, page, slot)] = c
        scales[page, :, slot] = e
        x = _values4(codes[_at(case, from_page, from_slot)], scales[from_page, :, from_slot])
        got.append((x * g[:, None]).to(torch.bfloat16))
    return got[0], got[1]


def _plain_decode(s):
    case = s["case"]
    B, N1, N2, ps = case["B"], case["N1"], case["N2"], case["ps"]
    G = N1 // N2
    pages = s["block_table"].long()
    n = pages.shape[1] * ps
    token = torch.arange(n, device="cuda")
    live = token < s["seqused_kv"][:, None]                            # [B, n]

    def rows(which):
        c = s[which + "_pages"][pages]                                 # [B, L, ...]
        c = (c.transpose(2, 3) if case["nhd"] else c).transpose(1, 2).reshape(B, N2, n, D // 2)
        e = s[which + "_scales"][pages].transpose(1, 2).reshape(B, N2, n, D // BLOCK)
        return _values4(c, e) * s[which + "_descale"].view(1, -1, 1, 1)

    q = s["q"].view(torch.float8_e4m3fn).float() * s["q_descale"][..., None] if case["q8"] else \
        s["q"].float()
    x = torch.matmul(q.view(B, N2, G, D), rows("k").transpose(2, 3)) * (1.0 / math.sqrt(D))
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
    o = torch.matmul(p, rows("v") * live[:, None, :, None])
    some = total > 0
    one = torch.where(some, total, torch.ones_like(total))
    o = torch.where(some, o / one, torch.zeros_like(o))
    lse = torch.where(some, m + torch.log(one), torch.full_like(m, NO_KEY))
    return o.view(B, N1, D).to(torch.bfloat16), lse.view(B, N1).t().contiguous()


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
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


def _nearest(x, values):
    """The nearest of ascending `values` to each x >= 0 (fp64), the one of even index in a tie."""
    hi = torch.searchsorted(values, x).clamp(max=values.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    a, b = x - values[lo], values[hi] - x
    return values[torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)]


def _stored(x, g):
    """What four bits hold of fp64 rows [..., 128] under descales g."""
    e4m3 = _e4m3_table()[:127]
    b = x.view(*x.shape[:-1], D // BLOCK, BLOCK)
    s = _nearest(b.abs().amax(-1, keepdim=True) / (6 * g), e4m3)
    y = torch.where(s > 0, b.abs() / (s * g), torch.zeros_like(b))
    level = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    return (_nearest(y, level) * s * g * torch.sign(b)).view(x.shape)


def _turned(x, positions, case):
    """fp64 rows rotated, as products of complex numbers."""
    R, x = case["R"], x.double()
    i = torch.arange(R // 2, device="cuda", dtype=torch.float64)
    s = case["factor"]
    f = torch.exp(-2.0 * i / R * (math.log(BASE) + (
        math.log(s) * R / (R - 2) if case["scaling"] == "base" else 0.0)))
    if case["scaling"] == "linear":
        f = f / s
    elif case["scaling"] == "parts":
        turns = CONTEXT * f / (2 * math.pi)
        w = torch.minimum(torch.maximum((turns - SLOW) / (FAST - SLOW), turns * 0), turns * 0 + 1)
        f = f / s + (f - f / s) * w
    unit = torch.polar(torch.full((len(positions), R // 2), _amplitude(case), dtype=torch.float64,
                                  device="cuda"), positions.double()[:, None] * f)
    y = x.clone()
    if case["inter"]:
        z = torch.view_as_complex(x[..., :R].unflatten(-1, (R // 2, 2)).contiguous())
        y[..., :R] = torch.view_as_real(z * unit[:, None]).flatten(-2)
    else:
        z = torch.complex(x[..., :R // 2], x[..., R // 2:R]) * unit[:, None]
        y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
    return y


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "pages":
        return None                                  # whole numbers
    if op == "rope":
        return _turned(s["q"], s["positions"], case), _turned(s["k"], s["positions"], case)
    if op == "ropeq":
        x = _turned(s["q"], s["positions"], case)
        d = x.abs().amax(-1, keepdim=True) / 448
        if case["ue8m0"]:
            d = torch.exp2(torch.ceil(torch.log2(d.float().double())))
        return x / d, d[..., 0]                      # the quotients, before they are codes
    if op == "store":
        return tuple(_stored(s[w].double(), s[w + "_descale"].double().view(-1, 1, 1))
                     for w in "kv")
    e4m3 = _e4m3_table()
    level = torch.tensor(LEVELS + tuple(-x for x in LEVELS), dtype=torch.float64, device="cuda")
    B, N1, N2, ps = case["B"], case["N1"], case["N2"], case["ps"]
    G = N1 // N2
    out = torch.zeros(B, N1, D, dtype=torch.float64, device="cuda")
    lse = torch.full((N1, B), NO_KEY, dtype=torch.float64, device="cuda")

    def rows(which, b, n):
        pg = s["block_table"][b, :-(-n // ps)].long()
        c = s[which + "_pages"][pg]
        c = c.permute(2, 0, 1, 3) if case["nhd"] else c.permute(1, 0, 2, 3)
        c = c.reshape(N2, -1, D // 2)[:, :n]
        e = e4m3[s[which + "_scales"][pg].long()].permute(1, 0, 2, 3).reshape(N2, -1, D // BLOCK)
        both = torch.stack((level[(c % 16).long()], level[(c // 16).long()]), -1).flatten(-2)
        return both * e[:, :n].repeat_interleave(BLOCK, -1) * \
            s[which + "_descale"].double().view(-1, 1, 1)

    for b, n in enumerate(lengths(case)):
        if n == 0:
            continue
        q = e4m3[s["q"][b].long()] * s["q_descale"][b].double()[:, None] if case["q8"] else \
            s["q"][b].double()
        x = torch.einsum("hgd,hnd->hgn", q.view(N2, G, D), rows("k", b, n)).reshape(N1, n)
        x = x / math.sqrt(D)
        nt = -(-n // TILE)
        if case["sparse"]:
            on = torch.zeros(N1, nt, dtype=torch.bool, device="cuda")
            if case["sparse"] == "mask":
                on = s["block_mask"][b, :, :nt] != 0
            else:
                on.scatter_(1, s["sparse_indices"][b, :, :_kept(case, nt)].long(), True)
            x[~on.repeat_interleave(TILE, 1)[:, :n]] = -math.inf
        z = torch.logsumexp(x, -1)
        some = z > -math.inf
        p = torch.exp(x - z[:, None])
        p[~some] = 0
        out[b] = torch.einsum("hgn,hnd->hgd", p.view(N2, G, n), rows("v", b, n)).reshape(N1, D)
        lse[some, b] = z[some]
    return out, lse


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "rope":
        rows = case["T"] * (case["N1"] + case["N2"])
        return dict(bytes=rows * 4 * D + 4 * case["T"], flops=rows * 3 * case["R"])
    if op == "ropeq":
        rows = case["T"] * case["N1"]
        return dict(bytes=rows * (3 * D + 4) + 4 * case["T"], flops=rows * (3 * case["R"] + 2 * D))
    if op == "pages":
        # lengths in, the prefix and two lengths out; each new token's position and slot; each new
        # page off the stack, into the table, out of it and on to the stack
        lens = lengths(case)
        pages = sum(-(-n // case["ps"]) for n in lens)
        return dict(bytes=24 * case["B"] + 8 * sum(lens) + 16 * pages, flops=0)
    token4 = 2 * (D // 2 + D // BLOCK)               # bytes of a KV head's token
    if op == "store":
        rows = case["T"] * case["N2"]
        return dict(bytes=rows * 2 * (token4 + 4 * D) + 8 * case["T"], flops=rows * 6 * D)
    lens = lengths(case)
    N2, ps = case["N2"], case["ps"]
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
    nbytes = size * token4 + lists + sum(-(-n // ps) for n in lens) * 4
    nbytes += B * N1 * (D * (1 if case["q8"] else 2) + (4 if case["q8"] else 0) + 2 * D + 4)
    return dict(bytes=int(nbytes), flops=int(pairs * 4 * D))
