"""Argument checks of decode, gather_kv and merge_states (no GPU: every call here returns or
raises before touching CUDA)."""
import ctypes
import os
import shutil

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


def _ddims(**kw):
    base = dict(B=2, N1=8, N2=2, D=128, page_size=64, max_kv_len=1024, num_pages=40,
                max_pages_per_seq=16, k_scale_kind=1, v_scale_kind=2, kv_layout=0, q_type=0,
                q_stride=1024, sparse=0)
    base.update(kw)
    return bsa.DecodeDims(**base)


def _decode(L, dims, **kw):
    a = dict(q=FAKE, qd=None, k=FAKE, v=FAKE, kd=FAKE, vd=FAKE, used=FAKE, bt=FAKE, mask=None,
             idx=None, sl=None, scale=0.088, out=FAKE, lse=FAKE, ws=None, nbytes=0)
    a.update(kw)
    return L.bsa_fp8_decode(ctypes.byref(dims), a["q"], a["qd"], a["k"], a["v"], a["kd"], a["vd"],
                            a["used"], a["bt"], a["mask"], a["idx"], a["sl"], a["scale"],
                            a["out"], a["lse"], a["ws"], a["nbytes"], None, None)


@pytest.mark.parametrize("bad", [
    dict(D=64), dict(page_size=16), dict(page_size=128), dict(B=-1), dict(N1=0), dict(N2=0),
    dict(N1=9), dict(N1=34, q_stride=34 * 128), dict(max_kv_len=-1), dict(max_kv_len=1025),
    dict(num_pages=-1), dict(max_pages_per_seq=-1), dict(k_scale_kind=2), dict(v_scale_kind=1),
    dict(kv_layout=2), dict(q_type=2), dict(q_stride=1023), dict(q_stride=1028),
    dict(q_type=1, q_stride=1032), dict(sparse=2), dict(num_pages=0)])
def test_decode_invalid_dims(L, bad):
    kw = dict(qd=FAKE) if bad.get("q_type") == 1 else {}
    assert _decode(L, _ddims(**bad), **kw) == INVALID
    if bad != dict(num_pages=0):
        assert bsa.decode_workspace_size(_ddims(**bad)) == 0


def test_decode_unsupported_sizes(L):
    big = dict(max_kv_len=4097 * 128, max_pages_per_seq=4097 * 2)
    assert _decode(L, _ddims(**big)) == UNSUPPORTED
    assert _decode(L, _ddims(B=1 << 29, N1=16, q_stride=2048)) == UNSUPPORTED
    assert _decode(L, _ddims(B=1 << 20, max_kv_len=4096 * 128,
                             max_pages_per_seq=4096 * 2)) == UNSUPPORTED


def test_decode_pointers_and_scalars(L):
    d = _ddims()
    for name in ("q", "k", "v", "kd", "vd", "used", "bt", "out"):
        assert _decode(L, d, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "kd", "out"):
        assert _decode(L, d, **{name: FAKE + 8}) == INVALID, name
    assert _decode(L, d, lse=FAKE + 2) == INVALID
    assert _decode(L, d, scale=float("nan")) == INVALID
    assert _decode(L, d, scale=float("inf")) == INVALID
    assert _decode(L, d, qd=FAKE) == INVALID                       # bf16 queries have none
    assert _decode(L, _ddims(q_type=1)) == INVALID                 # e4m3 queries need one
    s = _ddims(sparse=1)
    assert _decode(L, s) == INVALID                                # says sparse, gives nothing
    assert _decode(L, d, mask=FAKE) == INVALID                     # gives a mask, says dense
    assert _decode(L, s, mask=FAKE, idx=FAKE, sl=FAKE) == INVALID  # both
    assert _decode(L, s, idx=FAKE) == INVALID                      # no lengths
    assert _decode(L, d) == WORKSPACE
    assert _decode(L, d, ws=FAKE + 16, nbytes=1 << 40) == WORKSPACE
    assert _decode(L, _ddims(B=0), q=None, used=None, out=None) == OK
    assert L.bsa_fp8_decode(None, *([None] * 11), 0.1, None, None, None, 0, None, None) == INVALID


def _gdims(**kw):
    base = dict(B=2, N2=2, D=128, page_size=64, num_pages=8, max_pages_per_seq=4, total=10,
                k_scale_kind=1, v_scale_kind=2, kv_layout=0, out_type=0)
    base.update(kw)
    return bsa.GatherDims(**base)


def _gather(L, dims, **kw):
    a = dict(k=FAKE, v=FAKE, kd=FAKE, vd=FAKE, cu=FAKE, cs=None, bt=FAKE, ko=FAKE, vo=FAKE)
    a.update(kw)
    return L.bsa_fp8_gather_kv(ctypes.byref(dims), a["k"], a["v"], a["kd"], a["vd"], a["cu"],
                               a["cs"], a["bt"], a["ko"], a["vo"], None, None)


def test_gather_checks(L):
    for bad in (dict(D=64), dict(page_size=48), dict(B=-1), dict(N2=0), dict(num_pages=-1),
                dict(max_pages_per_seq=-1), dict(total=-1), dict(k_scale_kind=2),
                dict(v_scale_kind=1), dict(kv_layout=3), dict(out_type=2)):
        assert _gather(L, _gdims(**bad)) == INVALID, bad
    d = _gdims()
    for name in ("k", "v", "kd", "vd", "cu", "bt"):
        assert _gather(L, d, **{name: None}) == INVALID, name
    for name in ("k", "v", "ko", "vo"):
        assert _gather(L, d, **{name: FAKE + 8}) == INVALID, name
    assert _gather(L, d, ko=None, vo=None) == INVALID
    assert _gather(L, _gdims(total=0), ko=None, vo=None) == OK
    assert _gather(L, _gdims(B=0)) == OK
    assert L.bsa_fp8_gather_kv(None, *([FAKE] * 9), None, None) == INVALID


def _merge(L, count=2, outs=(FAKE, FAKE), lses=(FAKE, FAKE), T=4, N1=8, out=FAKE, lse=FAKE):
    po = (ctypes.c_void_p * len(outs))(*outs)
    pl = (ctypes.c_void_p * len(lses))(*lses)
    return L.bsa_fp8_merge_states(count, po, pl, T, N1, out, lse, None)


def test_merge_checks(L):
    for kw in (dict(count=0), dict(count=9), dict(T=-1), dict(N1=0), dict(T=1 << 20, N1=1 << 11),
               dict(outs=(FAKE, None)), dict(lses=(None, FAKE)), dict(outs=(FAKE, FAKE + 8)),
               dict(lses=(FAKE + 2, FAKE)), dict(out=None), dict(out=FAKE + 8),
               dict(lse=FAKE + 1)):
        assert _merge(L, **kw) == INVALID, kw
    assert _merge(L, T=0) == OK
    assert L.bsa_fp8_merge_states(2, None, None, 4, 8, FAKE, None, None) == INVALID


# ------------------------------------------------------------------- the binding's own checks

def _decode_args():
    return dict(q=torch.zeros(2, 8, 128, dtype=torch.bfloat16),
                k_pages=torch.zeros(6, 2, 32, 128, dtype=torch.uint8),
                v_pages=torch.zeros(6, 2, 32, 128, dtype=torch.uint8),
                k_descale=torch.zeros(6, 2, 32), v_descale=torch.zeros(2),
                seqused_kv=torch.zeros(2, dtype=torch.int32),
                block_table=torch.zeros(2, 3, dtype=torch.int32), max_kv_len=90)


@pytest.mark.parametrize("name,value,match", [
    ("q", torch.zeros(2, 8, 128), "dtype"), ("q", torch.zeros(2, 1024), "shape"),
    ("q", torch.zeros(2, 8, 256, dtype=torch.bfloat16)[:, :, ::2], "contiguous"),
    ("q", torch.zeros(8, 2, 128, dtype=torch.bfloat16).transpose(0, 1), "contiguous"),
    ("v_pages", torch.zeros(6, 2, 64, 128, dtype=torch.uint8), "shape"),
    ("k_pages", torch.zeros(6, 32, 2, 128, dtype=torch.uint8).transpose(1, 2), "contiguous"),
    ("k_pages", torch.zeros(6, 2, 32, 128, dtype=torch.float16), "dtype"),
    ("k_pages", torch.zeros(6, 2, 32, 64, dtype=torch.uint8), "head dim"),
    ("k_pages", torch.zeros(6, 2, 32 * 128, dtype=torch.uint8), "shape"),
    ("k_descale", torch.zeros(6, 2, 31), "shape"), ("k_descale", torch.zeros(2), "shape"),
    ("v_descale", torch.zeros(3), "shape"), ("v_descale", torch.zeros(2).double(), "dtype"),
    ("seqused_kv", torch.zeros(2, dtype=torch.int64), "dtype"),
    ("seqused_kv", torch.zeros(3, dtype=torch.int32), "shape"),
    ("block_table", torch.zeros(3, 3, dtype=torch.int32), "shape"),
    ("block_table", torch.zeros(6, dtype=torch.int32), "shape"),
    ("block_mask", torch.zeros(2, 8, 2, dtype=torch.uint8), "shape"),
    ("sparse_indices", torch.zeros(2, 8, 2, dtype=torch.int32), "shape"),
    ("sparse_seq_len", torch.zeros(2, 8, dtype=torch.int64), None),
    ("q_descale", torch.zeros(8, 2), "shape"),
    ("out", torch.zeros(2, 8, 128), "dtype"), ("lse", torch.zeros(2, 8), "shape"),
    ("dev_status", torch.zeros(1, dtype=torch.int64), "int32"),
    ("workspace", torch.zeros(64, 2, dtype=torch.uint8)[:, 0], "contiguous")])
def test_decode_binding_refuses(name, value, match):
    a = _decode_args()
    a[name] = value
    with pytest.raises(ValueError, match=match):
        bsa.decode(**a)


def test_binding_refuses_cpu_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        bsa.decode(**_decode_args())
    o, l = torch.zeros(3, 4, 128, dtype=torch.bfloat16), torch.zeros(4, 3)
    with pytest.raises(ValueError, match="CUDA"):
        bsa.merge_states([o, o], [l, l])
    a = _decode_args()
    with pytest.raises(ValueError, match="CUDA"):
        bsa.gather_kv(a["k_pages"], a["v_pages"], a["k_descale"], a["v_descale"],
                      torch.zeros(3, dtype=torch.int32), a["block_table"], 4)


def test_gather_and_merge_bindings_refuse():
    a = _decode_args()
    cu = torch.zeros(3, dtype=torch.int32)
    args = (a["k_pages"], a["v_pages"], a["k_descale"], a["v_descale"], cu, a["block_table"], 4)

    def refused(match, *pos, **kw):
        with pytest.raises(ValueError, match=match):
            bsa.gather_kv(*(pos or args), **kw)

    refused("both None", None, None, None, None, cu, a["block_table"], 4)
    refused("out_dtype", out_dtype=torch.float16)
    refused("dtype", k_out=torch.zeros(4, 2, 128, dtype=torch.bfloat16),
            v_out=torch.zeros(4, 2, 128))
    refused("shape", k_out=torch.zeros(5, 2, 128))
    refused("shape", *args[:4], cu[:2], *args[5:])
    refused("cache_starts", cache_starts=torch.zeros(3, dtype=torch.int32))
    refused("without", None, *args[1:], k_out=torch.zeros(4, 2, 128))
    o, l = torch.zeros(3, 4, 128, dtype=torch.bfloat16), torch.zeros(4, 3)
    for outs, lses, kw in (([], [], {}), ([o] * 9, [l] * 9, {}), ([o, o], [l], {}),
                           ([o, o[:2]], [l, l], {}), ([o, o.float()], [l, l], {}),
                           ([o, o], [l, l.t()], {}), ([o], [l], dict(out=o.float())),
                           ([o[..., :64]], [l], {}), ([o], [l], dict(lse=l.double()))):
        with pytest.raises(ValueError):
            bsa.merge_states(outs, lses, **kw)
