"""Argument checks of the rotary, page and 4-bit cache calls (no GPU: every call here returns or raises
before touching CUDA), and the host-side frequencies."""
import ctypes
import math
import os
import shutil

import numpy as np
import pytest
import torch

import block_sparse_fp8_gb300 as bsa
from block_sparse_fp8_gb300 import _build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    if _build.needs_build():
        if shutil.which(_build.nvcc()) is None and not os.path.exists(_build.nvcc()):
            pytest.skip("nvcc not available")
        _build.build()
    return bsa.lib()


# ---------------------------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------------------------

def _turns(t):
    """The frequencies in turns a position, as fractions of 2^64."""
    return [x % (1 << 64) for x in t.tolist()]


@pytest.mark.parametrize("R", [16, 64, 96, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies(L, R, base):
    """Against the formula in extended precision: a double's relative error, 2^-50."""
    for scaling, factor in ((bsa.ROPE_NONE, 1.0), (bsa.ROPE_LINEAR, 8.0), (bsa.ROPE_BASE, 4.0),
                            (bsa.ROPE_PARTS, 16.0)):
        got = _turns(bsa.rope_frequencies(R, base=base, scaling=scaling, factor=factor,
                                          context=4096))
        assert len(got) == R // 2
        for i, x in enumerate(got):
            b = np.longdouble(base)
            if scaling == bsa.ROPE_BASE:
                b = b * np.longdouble(factor) ** (np.longdouble(R) / (R - 2))
            f = b ** (np.longdouble(-2 * i) / R)
            if scaling == bsa.ROPE_LINEAR:
                f /= factor
            if scaling == bsa.ROPE_PARTS:
                t = 4096 * f / (2 * np.longdouble(math.pi))
                w = min(max((t - 1) / 31, np.longdouble(0)), np.longdouble(1))
                f = f * w + f / factor * (1 - w)
            want = float(f) / (2 * math.pi)
            assert abs(x / 2.0 ** 64 - want) <= 2.0 ** -49 * want + 2.0 ** -64, (i, scaling)


def test_frequencies_of_the_callers_own(L):
    f = [1.0, -1.0, 0.0, 2 * math.pi, 7.0, 1e-3, math.pi, 100.0]
    got = _turns(bsa.rope_frequencies(16, inv_freq=f))
    for x, w in zip(got, f):
        t = math.fmod(w / (2 * math.pi), 1.0) % 1.0
        assert min(abs(x / 2.0 ** 64 - t), 1 - abs(x / 2.0 ** 64 - t)) <= 2.0 ** -48
    with pytest.raises(ValueError):
        bsa.rope_frequencies(16, inv_freq=f[:7])


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=8), dict(rotary_dim=24), dict(rotary_dim=144),
    dict(scaling=4), dict(scaling=-1), dict(base=0.0), dict(base=float("nan")),
    dict(scaling=1, factor=0.0), dict(scaling=2, factor=float("inf")),
    dict(scaling=3, factor=2.0), dict(scaling=3, factor=2.0, context=100, slow=2.0, fast=2.0),
    dict(inv_freq=[float("nan")] * 64)])
def test_frequencies_refused(L, kw):
    with pytest.raises(bsa.BsaError):
        bsa.rope_frequencies(**dict(dict(rotary_dim=128), **kw))


@pytest.mark.parametrize("kw", [
    dict(base=1e-320), dict(base=5e-324),                           # fast ones beyond any double
    dict(scaling=1, factor=1e-320), dict(scaling=3, factor=1e-320, context=4096),
    dict(scaling=2, base=1e300, factor=1e300), dict(scaling=2, base=1e-300, factor=1e-300)])
def test_frequencies_that_overflow_are_refused(L, kw):
    """A stretched base or a frequency that no double holds."""
    with pytest.raises(bsa.BsaError):
        bsa.rope_frequencies(**dict(dict(rotary_dim=128), **kw))


# ---------------------------------------------------------------------------------------------
# rope
# ---------------------------------------------------------------------------------------------

def _rdims(**kw):
    base = dict(T=4, N1=8, N2=2, D=128, rotary_dim=64, layout=0, q_stride=1024, k_stride=256,
                q_out_stride=1024, k_out_stride=256)
    base.update(kw)
    return bsa.RopeDims(**base)


def _rope(L, dims, **kw):
    a = dict(q=FAKE, k=2 * FAKE, pos=FAKE, f=FAKE, amp=1.0, qo=3 * FAKE, ko=4 * FAKE)
    a.update(kw)
    return L.bsa_rope(ctypes.byref(dims), a["q"], a["k"], a["pos"], a["f"], a["amp"], a["qo"],
                      a["ko"], None)


def _ropeq(L, dims, **kw):
    a = dict(q=FAKE, pos=FAKE, f=FAKE, amp=1.0, rule=0, c=8 * FAKE, d=FAKE)
    a.update(kw)
    return L.bsa_rope_quantize(ctypes.byref(dims), a["q"], a["pos"], a["f"], a["amp"], a["rule"],
                               a["c"], a["d"], None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(N1=0), dict(N2=-1), dict(D=64), dict(rotary_dim=0), dict(rotary_dim=8),
    dict(rotary_dim=120), dict(rotary_dim=256), dict(layout=2), dict(q_stride=1016),
    dict(q_stride=1028), dict(k_stride=128), dict(q_out_stride=0), dict(k_out_stride=260)])
def test_rope_invalid_dims(L, bad):
    assert _rope(L, _rdims(**bad)) == INVALID
    if not any("k_" in n or "out" in n or n == "N2" for n in bad):
        assert _ropeq(L, _rdims(**dict(bad, N2=0))) == INVALID


def test_rope_pointers(L):
    d = _rdims()
    for name in ("q", "k", "pos", "f", "qo", "ko"):
        assert _rope(L, d, **{name: None}) == INVALID, name
    for name in ("q", "k", "qo", "ko"):
        assert _rope(L, d, **{name: 5 * FAKE + 8}) == INVALID, name
    assert _rope(L, d, f=FAKE + 4) == INVALID
    for amp in (float("nan"), float("inf")):
        assert _rope(L, d, amp=amp) == INVALID and _ropeq(L, _rdims(N2=0), amp=amp) == INVALID
    assert _rope(L, _rdims(N2=0)) == INVALID                        # a k that has no heads
    assert _rope(L, _rdims(q_out_stride=2048), qo=FAKE) == INVALID  # in place, at another stride
    assert _rope(L, _rdims(k_out_stride=512), ko=2 * FAKE) == INVALID
    assert _rope(L, _rdims(T=0), q=None, k=None, pos=None, f=None, qo=None, ko=None) == OK
    assert L.bsa_rope(None, *([FAKE] * 4), 1.0, FAKE, FAKE, None) == INVALID
    # memory that overlaps in part: rows of 2048 bytes, k's of 512, four of them
    far = 1 << 30
    for a in (dict(qo=FAKE + 16), dict(qo=FAKE + 2032), dict(qo=FAKE - 2032), dict(ko=2 * FAKE + 16),
              dict(qo=2 * FAKE - 64), dict(ko=FAKE + 4 * 2048 - 16), dict(qo=far, ko=far + 2032),
              dict(qo=far, ko=far), dict(ko=FAKE), dict(qo=2 * FAKE)):
        assert _rope(L, d, **a) == INVALID, a
    wide = _rdims(q_stride=4096, k_stride=4096, q_out_stride=4096, k_out_stride=4096)
    for a in (dict(k=FAKE + 2048, qo=FAKE + 2048 + 512 - 16), dict(k=FAKE + 2048, ko=FAKE + 16),
              dict(k=FAKE + 2048, qo=FAKE + 8192 - 16)):
        assert _rope(L, wide, **a) == INVALID, a
    q = _rdims(N2=0)
    assert _ropeq(L, q, c=FAKE + 16) == INVALID and _ropeq(L, q, c=FAKE + 4 * 2048 - 16) == INVALID
    for name in ("q", "pos", "f", "c", "d"):
        assert _ropeq(L, q, **{name: None}) == INVALID, name
    for name in ("q", "c"):
        assert _ropeq(L, q, **{name: 9 * FAKE + 8}) == INVALID, name
    assert _ropeq(L, q, rule=2) == INVALID
    assert _ropeq(L, d) == INVALID                                  # q alone
    assert _ropeq(L, _rdims(T=0, N2=0), q=None) == OK


# ---------------------------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------------------------

def _pdims(**kw):
    base = dict(B=3, page_size=32, num_pages=10, max_pages_per_seq=4, total=7)
    base.update(kw)
    return bsa.PagesDims(**base)


def _assign(L, dims, **kw):
    a = dict(new=FAKE, old=2 * FAKE, bt=FAKE, fp=FAKE, fc=FAKE, cu=3 * FAKE, used=4 * FAKE, pos=FAKE,
             slot=FAKE)
    a.update(kw)
    return L.bsa_assign_pages(ctypes.byref(dims), a["new"], a["old"], a["bt"], a["fp"], a["fc"],
                              a["cu"], a["used"], a["pos"], a["slot"], None, None)


def _release(L, dims, **kw):
    a = dict(lens=FAKE, keep=FAKE, bt=FAKE, fp=FAKE, fc=FAKE, out=FAKE)
    a.update(kw)
    return L.bsa_release_pages(ctypes.byref(dims), a["lens"], a["keep"], a["bt"], a["fp"], a["fc"],
                               a["out"], None, None)


def test_pages_refused(L):
    for bad in (dict(B=-1), dict(page_size=16), dict(page_size=128), dict(num_pages=-1),
                dict(max_pages_per_seq=-1), dict(total=-1), dict(num_pages=1 << 26),
                dict(page_size=64, max_pages_per_seq=1 << 25)):
        assert _assign(L, _pdims(**bad)) == INVALID, bad
        assert _release(L, _pdims(**bad)) == INVALID, bad
    for name in ("new", "old", "bt", "fp", "fc", "cu", "used", "pos", "slot"):
        assert _assign(L, _pdims(), **{name: None}) == INVALID, name
    for a in (dict(used=2 * FAKE), dict(used=FAKE + 8), dict(cu=FAKE - 12), dict(cu=2 * FAKE)):
        assert _assign(L, _pdims(), **a) == INVALID, a                # the lengths themselves
    for name in ("lens", "keep", "bt", "fp", "fc", "out"):
        assert _release(L, _pdims(), **{name: None}) == INVALID, name
    assert _assign(L, _pdims(B=0, total=0), fc=None, cu=None) == OK
    assert _release(L, _pdims(B=0), lens=None, keep=None, out=None) == OK


# ---------------------------------------------------------------------------------------------
# the 4-bit cache
# ---------------------------------------------------------------------------------------------

def _adims(**kw):
    base = dict(N2=2, D=128, page_size=64, num_pages=8, total_new=5, k_scale_kind=2,
                v_scale_kind=0, kv_layout=0, k_stride=256, v_stride=512)
    base.update(kw)
    return bsa.Fp4AppendDims(**base)


def _append(L, dims, **kw):
    a = dict(k=FAKE, v=FAKE, slot=FAKE, kd=FAKE, vd=FAKE, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE)
    a.update(kw)
    return L.bsa_fp4_append_kv(ctypes.byref(dims), a["k"], a["v"], a["slot"], a["kd"], a["vd"],
                               a["kp"], a["vp"], a["ks"], a["vs"], None, None)


def test_append_fp4_refused(L):
    for bad in (dict(N2=0), dict(D=64), dict(page_size=16), dict(num_pages=-1), dict(total_new=-1),
                dict(k_scale_kind=1), dict(v_scale_kind=1), dict(kv_layout=2), dict(k_stride=248),
                dict(v_stride=260)):
        assert _append(L, _adims(**bad)) == INVALID, bad
    for name in ("k", "v", "slot", "kd", "vd", "kp", "vp", "ks", "vs"):
        assert _append(L, _adims(), **{name: None}) == INVALID, name
    for name in ("k", "v", "kp", "vp", "ks", "vs"):
        assert _append(L, _adims(), **{name: FAKE + 8}) == INVALID, name
    assert _append(L, _adims(total_new=0), k=None, v=None) == OK


def _gather(L, dims, **kw):
    a = dict(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, kd=FAKE, vd=FAKE, cu=FAKE, bt=FAKE, ko=FAKE, vo=FAKE)
    a.update(kw)
    return L.bsa_fp4_gather_kv(ctypes.byref(dims), a["k"], a["v"], a["ks"], a["vs"], a["kd"],
                               a["vd"], a["cu"], None, a["bt"], a["ko"], a["vo"], None, None)


def test_gather_fp4_refused(L):
    def dims(**kw):
        return bsa.GatherDims(**dict(dict(B=2, N2=2, D=128, page_size=64, num_pages=8,
                                          max_pages_per_seq=4, total=10, k_scale_kind=2,
                                          v_scale_kind=2, kv_layout=0, out_type=0), **kw))

    for bad in (dict(D=64), dict(page_size=48), dict(k_scale_kind=1), dict(v_scale_kind=1),
                dict(kv_layout=3), dict(out_type=2), dict(total=-1)):
        assert _gather(L, dims(**bad)) == INVALID, bad
    for name in ("k", "v", "ks", "vs", "kd", "vd", "cu", "bt"):
        assert _gather(L, dims(), **{name: None}) == INVALID, name
    assert _gather(L, dims(), ko=None, vo=None) == INVALID
    assert _gather(L, dims(total=0)) == OK


def _decode(L, dims, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, kd=FAKE, vd=FAKE, used=FAKE, bt=FAKE,
             scale=0.088, out=FAKE, lse=FAKE, ws=None, nbytes=0)
    a.update(kw)
    return L.bsa_fp4_decode(ctypes.byref(dims), a["q"], None, a["k"], a["v"], a["ks"], a["vs"],
                            a["kd"], a["vd"], a["used"], a["bt"], None, None, None, a["scale"],
                            a["out"], a["lse"], a["ws"], a["nbytes"], None, None)


def test_decode_fp4_refused(L):
    def dims(**kw):
        return bsa.DecodeDims(**dict(dict(B=2, N1=8, N2=2, D=128, page_size=64, max_kv_len=1024,
                                          num_pages=40, max_pages_per_seq=16, k_scale_kind=2,
                                          v_scale_kind=0, kv_layout=0, q_type=0, q_stride=1024,
                                          sparse=0), **kw))

    for bad in (dict(D=64), dict(page_size=16), dict(N1=9), dict(N1=34, q_stride=34 * 128),
                dict(k_scale_kind=1), dict(v_scale_kind=1), dict(kv_layout=2), dict(q_stride=1023)):
        assert _decode(L, dims(**bad)) == INVALID, bad
        assert bsa.decode_fp4_workspace_size(dims(**bad)) == 0
    assert bsa.decode_workspace_size(dims()) == 0              # per head: the 4-bit cache's kind
    for name in ("q", "k", "v", "ks", "vs", "kd", "vd", "used", "bt", "out"):
        assert _decode(L, dims(), **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "ks", "vs", "out"):
        assert _decode(L, dims(), **{name: FAKE + 8}) == INVALID, name
    assert _decode(L, dims(), scale=float("nan")) == INVALID
    assert _decode(L, dims()) == WORKSPACE
    assert _decode(L, dims(max_kv_len=4097 * 128, max_pages_per_seq=4097 * 2)) == UNSUPPORTED
    assert _decode(L, dims(B=0), q=None, used=None, out=None) == OK


# ---------------------------------------------------------------------------------------------
# the bindings
# ---------------------------------------------------------------------------------------------

def _cpu():
    bf16, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    x = torch.zeros(4, 2, 128, dtype=bf16)
    return dict(x=x, pos=torch.zeros(4, dtype=i32), f=torch.zeros(64, dtype=torch.int64),
                p=torch.zeros(6, 2, 32, 64, dtype=u8), s=torch.zeros(6, 2, 32, 8, dtype=u8),
                g=torch.ones(2), i4=torch.zeros(4, dtype=i32), bt=torch.zeros(4, 3, dtype=i32),
                fp=torch.zeros(6, dtype=i32), fc=torch.zeros(1, dtype=i32))


def test_bindings_refuse_shapes_and_types(L):
    c = _cpu()
    x, pos, f, p, s, g, i4, bt, fp, fc = (c[n] for n in ("x", "pos", "f", "p", "s", "g", "i4", "bt",
                                                         "fp", "fc"))
    refused = [
        lambda: bsa.rope(x, pos[:3], f), lambda: bsa.rope(x.float(), pos, f),
        lambda: bsa.rope(x, pos.long(), f), lambda: bsa.rope(x, pos, f.int()),
        lambda: bsa.rope(x[..., :64], pos, f), lambda: bsa.rope(x.transpose(0, 1), pos[:2], f),
        lambda: bsa.rope(x, pos, f, k=x[:3]), lambda: bsa.rope(x, pos, f, k_out=x),
        lambda: bsa.rope(x, pos, f, out=x[:, :1]), lambda: bsa.rope(x, pos, f, k=x, k_out=x[:, :1]),
        lambda: bsa.rope_quantize(x, pos, f, codes=x), lambda: bsa.rope_quantize(x, pos, f, descale=g),
        lambda: bsa.assign_pages(i4, i4[:3], bt, fp, fc, 32, 5),
        lambda: bsa.assign_pages(i4, i4, bt[:3], fp, fc, 32, 5),
        lambda: bsa.assign_pages(i4, i4, bt, fp, fp, 32, 5),
        lambda: bsa.assign_pages(i4, i4, bt, fp, fc, 32, 5, slot_map=i4),
        lambda: bsa.release_pages(i4, i4[:3], bt, fp, fc, 32),
        lambda: bsa.release_pages(i4, i4, bt, fp, fc, 32, out=fp),
        lambda: bsa.append_kv_fp4(x, x, i4[:3], p, p, s, s, g, g),
        lambda: bsa.append_kv_fp4(x[:, :1], x, i4, p, p, s, s, g, g),
        lambda: bsa.append_kv_fp4(x, x, i4, p[..., :32], p, s, s, g, g),
        lambda: bsa.append_kv_fp4(x, x, i4, p, p, s[..., :4], s, g, g),
        lambda: bsa.append_kv_fp4(x, x, i4, p, p, s, None, g, g),
        lambda: bsa.append_kv_fp4(x, x, i4, p, p, s, s, g, torch.ones(3)),
        lambda: bsa.gather_kv_fp4(p, p, s, None, g, g, i4[:3], bt[:2], 5),
        lambda: bsa.gather_kv_fp4(None, None, s, s, g, g, i4[:3], bt[:2], 5),
        lambda: bsa.decode_fp4(x, p, p, s, s[..., :4], g, g, i4, bt, 90),
        lambda: bsa.decode_fp4(x, p, p, None, None, g, g, i4, bt, 90),
        lambda: bsa.decode_fp4(x, torch.zeros(6, 2, 32, 128, dtype=torch.uint8), p, s, s, g, g, i4,
                               bt, 90),
        # all in order, but not on a GPU
        lambda: bsa.rope(x, pos, f, k=x), lambda: bsa.rope_quantize(x, pos, f),
        lambda: bsa.assign_pages(i4, i4.clone(), bt, fp, fc, 32, 5),
        lambda: bsa.release_pages(i4, i4, bt, fp, fc, 32),
        lambda: bsa.append_kv_fp4(x, x, i4, p, p, s, s, g, g),
        lambda: bsa.gather_kv_fp4(p, p, s, s, g, g, i4[:3], bt[:2], 5),
        lambda: bsa.decode_fp4(x, p, p, s, s, g, g, i4, bt, 90),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")


class _Library:
    """Stands in for the compiled library: every call succeeds, every workspace has 512 bytes."""

    def __getattr__(self, name):
        return lambda *args: 512 if name.endswith("_size") else 0


class _Stream:
    cuda_stream = 0
    device = torch.device("cuda", 0)


@pytest.mark.parametrize("name,count", [("rope", 2), ("rope_quantize", 2), ("assign_pages", 4),
                                        ("release_pages", 1), ("gather_kv_fp4", 2),
                                        ("decode_fp4", 2)])
def test_tensors_come_from_the_stream_of_the_call(name, count, monkeypatch):
    """Whatever a call on a named stream makes for itself is allocated with that stream current."""
    c = _cpu()
    x, i4 = c["x"], c["i4"]
    call = {
        "rope": lambda **k: bsa.rope(x, c["pos"], c["f"], k=x, **k),
        "rope_quantize": lambda **k: bsa.rope_quantize(x, c["pos"], c["f"], **k),
        "assign_pages": lambda **k: bsa.assign_pages(i4, i4, c["bt"], c["fp"], c["fc"], 32, 5, **k),
        "release_pages": lambda **k: bsa.release_pages(i4, i4, c["bt"], c["fp"], c["fc"], 32, **k),
        "gather_kv_fp4": lambda **k: bsa.gather_kv_fp4(c["p"], c["p"], c["s"], c["s"], c["g"], c["g"],
                                                       i4[:3], c["bt"][:2], 5, **k),
        "decode_fp4": lambda **k: bsa.decode_fp4(x, c["p"], c["p"], c["s"], c["s"], c["g"], c["g"], i4,
                                                 c["bt"], 90, **k),
    }[name]
    state, seen, empty = [None], [], torch.empty

    class on:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            self.before, state[0] = state[0], self.stream

        def __exit__(self, *_):
            state[0] = self.before

    def made(*args, **kw):
        seen.append(state[0])
        return empty(*args, **kw)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", made)
    monkeypatch.setattr(bsa, "lib", lambda: _Library())
    side = _Stream()
    with pytest.raises(ValueError):       # for their CPU tensors, after the outputs were made
        call(stream=side)
    assert seen == [side] * count


def test_release_refuses_lengths_that_overlap_in_part(L):
    """lens_out may be either of the lengths read, not lie across them: those of the first 1024 sequences
    would be written before the others' are read."""
    far = 64 * FAKE
    for B in (3, 2000):
        d = _pdims(B=B)
        for name in ("lens", "keep"):
            other = dict(lens=far, keep=2 * far)
            for off in (4, -4, 4 * B - 4, 4 - 4 * B):
                a = dict(other, out=other[name] + off)
                assert _release(L, d, **a) == INVALID, (B, name, off)
            # itself, or beside it: refused for nothing but the missing GPU
            for off in (0, 4 * B, -4 * B):
                if not torch.cuda.is_available():
                    assert _release(L, d, **dict(other, out=other[name] + off)) not in (OK, INVALID)


# ---------------------------------------------------------------------------------------------
# the e4m3 cache behind assign_pages
# ---------------------------------------------------------------------------------------------

def test_append_slots_refused(L):
    def call(dims, **kw):
        a = dict(k=FAKE, v=FAKE, slot=FAKE, ks=None, vs=FAKE, kp=FAKE, vp=FAKE, kd=FAKE)
        a.update(kw)
        return L.bsa_fp8_append_kv_slots(ctypes.byref(dims), a["k"], a["v"], a["slot"], a["ks"],
                                         a["vs"], a["kp"], a["vp"], a["kd"], None, None)

    def dims(**kw):
        return bsa.AppendDims(**dict(dict(B=0, N2=2, D=128, page_size=64, num_pages=4,
                                          max_pages_per_seq=0, total_new=8, k_scale_kind=1,
                                          v_scale_kind=2, kv_layout=0, k_descale_rule=0), **kw))

    for bad in (dict(N2=0), dict(D=64), dict(page_size=16), dict(num_pages=-1), dict(total_new=-1),
                dict(k_scale_kind=2), dict(v_scale_kind=1), dict(kv_layout=2), dict(k_descale_rule=2)):
        assert call(dims(**bad)) == INVALID, bad
    for name in ("k", "v", "slot", "vs", "kp", "vp", "kd"):
        assert call(dims(), **{name: None}) == INVALID, name
    for name in ("k", "v", "kp", "vp"):
        assert call(dims(), **{name: FAKE + 8}) == INVALID, name
    assert call(dims(k_scale_kind=0), kd=None) == INVALID           # a descale per tensor is given
    assert call(dims(total_new=0), k=None, slot=None) == OK


def test_append_slots_binding_refuses(L):
    x, i4 = torch.zeros(4, 2, 128, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    p, kd, vs = torch.zeros(6, 2, 32, 128, dtype=torch.uint8), torch.zeros(6, 2, 32), torch.ones(2)
    none = (None, None, None)
    wide = torch.zeros(4, 6, 128, dtype=torch.bfloat16)
    for call in (lambda: bsa.append_kv(x, x, i4, i4, i4[None], p, p, kd, v_scale=vs, slot_map=i4),
                 lambda: bsa.append_kv(x, x, None, None, i4[None], p, p, kd, v_scale=vs, slot_map=i4),
                 lambda: bsa.append_kv(x, x, *none, p, p, kd, v_scale=vs, slot_map=i4[:3]),
                 lambda: bsa.append_kv(x, x, *none, p, p, kd, v_scale=vs, slot_map=i4.long()),
                 lambda: bsa.append_kv(wide[:, :2], x, *none, p, p, kd, v_scale=vs, slot_map=i4),
                 lambda: bsa.append_kv(x, wide[:, 4:], *none, p, p, kd, v_scale=vs, slot_map=i4),
                 lambda: bsa.append_kv(x, x[:3], *none, p, p, kd, v_scale=vs, slot_map=i4),
                 lambda: bsa.append_kv(x, x, *none, p, p[:5], kd, v_scale=vs, slot_map=i4),
                 lambda: bsa.append_kv(x, x, *none, p, p, kd, v_scale=vs, slot_map=i4)):  # no GPU
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------------------------------------
# packed queries
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fp4", [False, True])
def test_decode_rows_refused(L, fp4):
    def dims(**kw):
        return bsa.DecodeDims(**dict(dict(B=2, N1=8, N2=2, D=128, page_size=64, max_kv_len=1024,
                                          num_pages=40, max_pages_per_seq=16,
                                          k_scale_kind=2 if fp4 else 1, v_scale_kind=0, kv_layout=0,
                                          q_type=0, q_stride=1024, sparse=0), **kw))

    def call(d, **kw):
        a = dict(T=3, cu=FAKE, q=FAKE, k=FAKE, v=FAKE, sc=FAKE, kd=FAKE, vd=FAKE, used=FAKE, bt=FAKE,
                 out=FAKE, lse=FAKE)
        a.update(kw)
        fn = L.bsa_fp4_decode_rows if fp4 else L.bsa_fp8_decode_rows
        return fn(ctypes.byref(d), a["T"], a["cu"], a["q"], None, a["k"], a["v"],
                  *([a["sc"]] * 2 if fp4 else []), a["kd"], a["vd"], a["used"], a["bt"], None, None,
                  None, 0.088, a["out"], a["lse"], None, 0, None, None)

    assert call(dims()) == WORKSPACE
    assert call(dims(), T=-1) == INVALID
    for name in ("cu", "q", "k", "v", "kd", "vd", "used", "bt", "out"):
        assert call(dims(), **{name: None}) == INVALID, name
    assert call(dims(N1=9)) == INVALID and call(dims(B=-1)) == INVALID
    assert call(dims(), T=0, cu=None, q=None, out=None) == OK
    # no sequences: the rows are written all the same
    assert call(dims(B=0), k=None, v=None, used=None, bt=None) == WORKSPACE
    assert call(dims(B=0), out=None) == INVALID and call(dims(B=0), cu=None) == INVALID


def test_decode_rows_binding_refuses(L):
    x, i4 = torch.zeros(3, 8, 128, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    p4, s4 = torch.zeros(6, 2, 32, 64, dtype=torch.uint8), torch.zeros(6, 2, 32, 8, dtype=torch.uint8)
    p8, kd, g = torch.zeros(6, 2, 32, 128, dtype=torch.uint8), torch.zeros(6, 2, 32), torch.ones(2)
    bt, cu = torch.zeros(4, 3, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    good = dict(q=x, seqused_kv=i4, block_table=bt, max_kv_len=90, cu_seqlens_q=cu)
    for bad, match in ((dict(cu_seqlens_q=cu[:3]), "shape"), (dict(cu_seqlens_q=cu.long()), "dtype"),
                       (dict(cu_seqlens_q=cu[:0]), "shape"), (dict(cu_seqlens_q=cu[None]), "shape"),
                       (dict(seqused_kv=i4[:3]), "shape"), (dict(block_table=bt[:3]), "shape"),
                       (dict(out=torch.zeros(4, 8, 128, dtype=torch.bfloat16)), "shape"),
                       (dict(lse=torch.zeros(8, 4)), "shape"),
                       (dict(block_mask=torch.zeros(3, 8, 1, dtype=torch.uint8)), "shape"),
                       ({}, "CUDA")):
        a = dict(good, **bad)
        with pytest.raises(ValueError, match=match):
            bsa.decode(k_pages=p8, v_pages=p8, k_descale=kd, v_descale=g, **a)
        with pytest.raises(ValueError, match=match):
            bsa.decode_fp4(k_pages=p4, v_pages=p4, k_scales=s4, v_scales=s4, k_descale=g, v_descale=g, **a)
