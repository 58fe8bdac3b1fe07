"""Block-sparse FP8 attention prefill over a paged KV cache on GB300 (sm_103a).

A thin ctypes binding over the C ABI in include/bsa_fp8.h: it marshals PyTorch CUDA tensors
(device pointers) and the current stream into ``bsa_fp8_prefill`` / ``bsa_fp8_compact_tiles``
and the quantise step ``bsa_fp8_quantize_rows`` / ``bsa_fp8_append_kv``; ``prefill_host``
marshals CPU tensors into ``bsa_fp8_prefill_host``, which copies them in and the results out.
``decode`` / ``gather_kv`` / ``merge_states`` serve from the same cache: the next token's
attention, the cache read back, and the join of attention results over parts of a cache.
Around them: ``rope`` / ``rope_quantize`` (rotary positions), ``assign_pages`` / ``release_pages``
(block tables and slot maps from the requests' lengths), and a cache held in 4 bits:
``append_kv_fp4`` / ``gather_kv_fp4`` / ``decode_fp4``.
Every step of the computation runs in the library's CUDA kernels; there is no CPU path.
Every call takes ``stream=`` (default: the current one).  The caller sees to it that the inputs are
ready there; outputs and workspaces that the call makes itself come from that stream's memory.
The library must have been built (``block_sparse_fp8_gb300._build.build()``); importing the
binding on a machine without it raises immediately.
"""
from __future__ import annotations

import ctypes
import math
import os

from . import _build

__all__ = ["Dims", "AppendDims", "Tensors", "TENSOR_NAMES", "Q_TND", "Q_NTD", "KV_HND",
           "KV_NHD", "prefill", "prefill_host", "compact_tiles", "quantize_rows", "append_kv",
           "workspace_size", "status_string", "set_wait_limit_ns", "lib",
           "SCALE_PER_TENSOR", "SCALE_PER_TOKEN_HEAD", "SCALE_PER_HEAD", "BsaError",
           "DESCALE_AMAX", "DESCALE_UE8M0", "DecodeDims", "GatherDims", "make_decode_dims",
           "decode", "decode_workspace_size", "gather_kv", "merge_states", "QTYPE_BF16",
           "QTYPE_E4M3", "OUT_BF16", "OUT_FP32", "MAX_MERGE",
           "rope", "rope_quantize", "rope_frequencies", "ROPE_HALF", "ROPE_INTERLEAVED", "ROPE_NONE",
           "ROPE_LINEAR", "ROPE_BASE", "ROPE_PARTS", "RopeDims", "assign_pages", "release_pages",
           "PagesDims", "append_kv_fp4", "gather_kv_fp4", "decode_fp4",
           "decode_fp4_workspace_size", "Fp4AppendDims",
           "DEV_BAD_INDEX", "DEV_BAD_PAGE", "DEV_BAD_SEQLEN", "DEV_TIMEOUT", "DEV_NO_PAGES"]

SCALE_PER_TENSOR = 0
SCALE_PER_TOKEN_HEAD = 1
SCALE_PER_HEAD = 2

DEV_BAD_INDEX = 1
DEV_BAD_PAGE = 2
DEV_BAD_SEQLEN = 4
DEV_TIMEOUT = 8
DEV_NO_PAGES = 16

EXPORTED = ("bsa_fp8_prefill", "bsa_fp8_prefill_workspace_size", "bsa_fp8_compact_tiles",
            "bsa_fp8_prefill_noalloc", "bsa_fp8_prefill_host", "bsa_fp8_quantize_rows",
            "bsa_fp8_quantize_rows_ue8m0", "bsa_fp8_append_kv", "bsa_fp8_append_kv_slots",
            "bsa_fp8_set_wait_limit_ns",
            "bsa_fp8_decode", "bsa_fp8_decode_rows", "bsa_fp8_decode_workspace_size", "bsa_fp8_gather_kv",
            "bsa_fp8_merge_states", "bsa_rope_frequencies", "bsa_rope", "bsa_rope_quantize",
            "bsa_assign_pages", "bsa_release_pages", "bsa_fp4_append_kv", "bsa_fp4_gather_kv",
            "bsa_fp4_decode", "bsa_fp4_decode_rows", "bsa_fp4_decode_workspace_size", "bsa_status_string")

# descale rules of the quantise step
DESCALE_AMAX = 0    # amax / 448
DESCALE_UE8M0 = 1   # amax / 448 rounded up to a power of two


class BsaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "B", "N1", "N2", "D", "page_size", "max_q_len", "max_kv_len", "num_pages",
        "max_pages_per_seq", "total_q", "k_scale_kind", "v_scale_kind", "causal", "q_layout",
        "kv_layout", "tiles_per_step")]


# the tensors of one call, in bsa_fp8_tensors_t's order (prefill's argument names; out, lse)
TENSOR_NAMES = ("q", "k_pages", "v_pages", "q_descale", "k_descale", "v_descale",
                "cu_seqlens_q", "seqused_kv", "block_table", "block_mask", "sparse_indices",
                "sparse_seq_len", "out", "lse")


class Tensors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in TENSOR_NAMES]


Q_TND, Q_NTD = 0, 1
KV_HND, KV_NHD = 0, 1


class AppendDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "B", "N2", "D", "page_size", "num_pages", "max_pages_per_seq", "total_new",
        "k_scale_kind", "v_scale_kind", "kv_layout", "k_descale_rule")]


# decode's query types, gather_kv's output types, most parts of one merge_states call
QTYPE_BF16, QTYPE_E4M3 = 0, 1
OUT_BF16, OUT_FP32 = 0, 1
MAX_MERGE = 8


class DecodeDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "B", "N1", "N2", "D", "page_size", "max_kv_len", "num_pages", "max_pages_per_seq",
        "k_scale_kind", "v_scale_kind", "kv_layout", "q_type", "q_stride", "sparse")]


class GatherDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "B", "N2", "D", "page_size", "num_pages", "max_pages_per_seq", "total", "k_scale_kind",
        "v_scale_kind", "kv_layout", "out_type")]


# pairs of a rotated head, and how frequencies are stretched
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_NONE, ROPE_LINEAR, ROPE_BASE, ROPE_PARTS = 0, 1, 2, 3


class RopeDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("T", "N1", "N2", "D", "rotary_dim", "layout")] + [
        (n, ctypes.c_longlong) for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")]


class PagesDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "B", "page_size", "num_pages", "max_pages_per_seq", "total")]


class Fp4AppendDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "N2", "D", "page_size", "num_pages", "total_new", "k_scale_kind", "v_scale_kind",
        "kv_layout")] + [(n, ctypes.c_longlong) for n in ("k_stride", "v_stride")]


_lib = None


def lib():
    """The loaded libbsa_fp8.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.LIB):
            raise ImportError(
                f"{_build.LIB} is missing: build it with block_sparse_fp8_gb300._build.build()")
        L = ctypes.CDLL(_build.LIB)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.bsa_fp8_prefill.restype = i32
        L.bsa_fp8_prefill.argtypes = [ctypes.POINTER(Dims)] + [vp] * 12 + [f32, f32, vp, vp, vp,
                                                                           sz, vp, vp]
        L.bsa_fp8_prefill_workspace_size.restype = sz
        L.bsa_fp8_prefill_workspace_size.argtypes = [ctypes.POINTER(Dims)]
        L.bsa_fp8_prefill_noalloc.restype = i32
        L.bsa_fp8_prefill_noalloc.argtypes = [ctypes.POINTER(Dims)] + [vp] * 12 + [f32, f32, vp,
                                                                                  vp, vp, vp]
        L.bsa_fp8_prefill_host.restype = i32
        L.bsa_fp8_prefill_host.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(Tensors),
                                           ctypes.POINTER(Tensors), f32, f32, vp, sz, vp, vp]
        L.bsa_fp8_compact_tiles.restype = i32
        L.bsa_fp8_compact_tiles.argtypes = [ctypes.POINTER(Dims)] + [vp] * 9
        L.bsa_fp8_quantize_rows.restype = i32
        L.bsa_fp8_quantize_rows.argtypes = [vp, ctypes.c_longlong, vp, vp, vp]
        L.bsa_fp8_quantize_rows_ue8m0.restype = i32
        L.bsa_fp8_quantize_rows_ue8m0.argtypes = [vp, ctypes.c_longlong, vp, vp, vp]
        L.bsa_fp8_append_kv.restype = i32
        L.bsa_fp8_append_kv.argtypes = [ctypes.POINTER(AppendDims)] + [vp] * 12
        L.bsa_fp8_append_kv_slots.restype = i32
        L.bsa_fp8_append_kv_slots.argtypes = [ctypes.POINTER(AppendDims)] + [vp] * 10
        L.bsa_fp8_set_wait_limit_ns.restype = i32
        L.bsa_fp8_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
        L.bsa_fp8_decode.restype = i32
        L.bsa_fp8_decode.argtypes = [ctypes.POINTER(DecodeDims)] + [vp] * 11 + [f32, vp, vp, vp,
                                                                                sz, vp, vp]
        L.bsa_fp8_decode_workspace_size.restype = sz
        L.bsa_fp8_decode_workspace_size.argtypes = [ctypes.POINTER(DecodeDims)]
        L.bsa_fp8_gather_kv.restype = i32
        L.bsa_fp8_gather_kv.argtypes = [ctypes.POINTER(GatherDims)] + [vp] * 11
        L.bsa_fp8_merge_states.restype = i32
        L.bsa_fp8_merge_states.argtypes = [i32, vp, vp, i32, i32, vp, vp, vp]
        f64 = ctypes.c_double
        L.bsa_rope_frequencies.restype = i32
        L.bsa_rope_frequencies.argtypes = [i32, i32, f64, f64, f64, f64, f64, vp, vp]
        L.bsa_rope.restype = i32
        L.bsa_rope.argtypes = [ctypes.POINTER(RopeDims)] + [vp] * 4 + [f32] + [vp] * 3
        L.bsa_rope_quantize.restype = i32
        L.bsa_rope_quantize.argtypes = [ctypes.POINTER(RopeDims)] + [vp] * 3 + [f32, i32] + [vp] * 3
        L.bsa_assign_pages.restype = i32
        L.bsa_assign_pages.argtypes = [ctypes.POINTER(PagesDims)] + [vp] * 11
        L.bsa_release_pages.restype = i32
        L.bsa_release_pages.argtypes = [ctypes.POINTER(PagesDims)] + [vp] * 8
        L.bsa_fp4_append_kv.restype = i32
        L.bsa_fp4_append_kv.argtypes = [ctypes.POINTER(Fp4AppendDims)] + [vp] * 11
        L.bsa_fp4_gather_kv.restype = i32
        L.bsa_fp4_gather_kv.argtypes = [ctypes.POINTER(GatherDims)] + [vp] * 13
        L.bsa_fp4_decode.restype = i32
        L.bsa_fp4_decode.argtypes = [ctypes.POINTER(DecodeDims)] + [vp] * 13 + [f32, vp, vp, vp,
                                                                                sz, vp, vp]
        for rows, fn in ((L.bsa_fp8_decode_rows, L.bsa_fp8_decode),
                         (L.bsa_fp4_decode_rows, L.bsa_fp4_decode)):
            rows.restype = i32
            rows.argtypes = [fn.argtypes[0], i32, vp] + fn.argtypes[1:]
        L.bsa_fp4_decode_workspace_size.restype = sz
        L.bsa_fp4_decode_workspace_size.argtypes = [ctypes.POINTER(DecodeDims)]
        L.bsa_status_string.restype = ctypes.c_char_p
        L.bsa_status_string.argtypes = [i32]
        _lib = L
    return _lib


def set_wait_limit_ns(ns: int) -> None:
    """Limit of every bounded wait inside the prefill and decode kernels for later launches (0:
    the default, 2 s).  A wait that runs out sets DEV_TIMEOUT in the device status word."""
    lib().bsa_fp8_set_wait_limit_ns(int(ns))


def status_string(status: int) -> str:
    return lib().bsa_status_string(status).decode()


def _p(t):
    return None if t is None else t.data_ptr()


def _stream_handle(stream):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _empty(shape, dtype, device, stream, result=True):
    """A tensor that a call makes for itself, from the memory of the stream that the call runs on
    (None: the current one): memory that was freed may still be in use by work queued before, and
    the allocator orders such reuse within one stream only.  A result may be read on the
    current stream, once that has waited for `stream`, and dropped there: its memory is kept from
    `stream` until the current one is through with it."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if result and t.is_cuda:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def make_dims(q, k_pages, block_table, cu_seqlens_q, max_q_len, max_kv_len, k_scale_kind,
              v_scale_kind, causal=True, q_layout=Q_TND, kv_layout=KV_HND,
              tiles_per_step=1) -> Dims:
    if q_layout == Q_NTD:
        N1, T, D = q.shape
    else:
        T, N1, D = q.shape
    if kv_layout == KV_NHD:
        P, ps, N2, D2 = k_pages.shape
    else:
        P, N2, ps, D2 = k_pages.shape
    return Dims(B=cu_seqlens_q.shape[0] - 1, N1=N1, N2=N2, D=D, page_size=ps,
                max_q_len=int(max_q_len), max_kv_len=int(max_kv_len), num_pages=P,
                max_pages_per_seq=block_table.shape[1], total_q=T,
                k_scale_kind=int(k_scale_kind), v_scale_kind=int(v_scale_kind),
                causal=int(bool(causal)), q_layout=int(q_layout), kv_layout=int(kv_layout),
                tiles_per_step=int(tiles_per_step))


def workspace_size(dims: Dims) -> int:
    return int(lib().bsa_fp8_prefill_workspace_size(ctypes.byref(dims)))


def prefill(q, k_pages, v_pages, q_descale, k_descale, v_descale, cu_seqlens_q, seqused_kv,
            block_table, max_q_len: int, max_kv_len: int, block_mask=None, sparse_indices=None,
            sparse_seq_len=None, softmax_scale: float | None = None, p_scale: float = 256.0,
            causal: bool = True, out=None, lse=None, return_lse: bool = True, dev_status=None,
            workspace=None, stream=None, k_scale_kind: int | None = None,
            v_scale_kind: int | None = None, q_layout: int = Q_TND, kv_layout: int = KV_HND,
            tiles_per_step: int = 1):
    """Block-sparse FP8 prefill.  Tensors are CUDA tensors in the C ABI's layouts:
    q uint8/float8_e4m3fn [T, N1, 128] (q_layout Q_TND) or [N1, T, 128] (Q_NTD, with q_descale
    [N1, T]); k_pages, v_pages [P, N2, page, 128] (KV_HND) or [P, page, N2, 128] (KV_NHD);
    q_descale f32 [T, N1]; k_descale f32 [1] or [P, N2, page]; v_descale f32 [1] or [N2];
    cu_seqlens_q i32
    [B+1]; seqused_kv i32 [B] or None; block_table i32 [B, L]; block_mask u8 [B, N1, Qb, Kb]
    or sparse_indices i32 [B, N1, Qb, Kb] + sparse_seq_len i32 [B, N1, Qb].
    max_q_len / max_kv_len are host integers (upper bounds of the per-sequence lengths).
    The scale kinds default to what the descale shapes imply (K [P, N2, page] = per token and
    head; V [N2] = per head, which for N2 = 1 is the same as per tensor).
    tiles_per_step = 2 runs the online softmax over 256-wide macro blocks (two list tiles
    per step).  Returns (out bf16 [T, N1, 128], lse f32 [N1, T] or None)."""
    import torch

    n2 = k_pages.shape[2] if kv_layout == KV_NHD else k_pages.shape[1]
    k_kind = k_scale_kind if k_scale_kind is not None else (
        SCALE_PER_TOKEN_HEAD if k_descale.dim() == 3 else SCALE_PER_TENSOR)
    v_kind = v_scale_kind if v_scale_kind is not None else (
        SCALE_PER_HEAD if v_descale.numel() == n2 else SCALE_PER_TENSOR)
    dims = make_dims(q, k_pages, block_table, cu_seqlens_q, max_q_len, max_kv_len, k_kind,
                     v_kind, causal, q_layout, kv_layout, tiles_per_step)
    T, N1, D = dims.total_q, dims.N1, dims.D
    if out is None:
        out = _empty((T, N1, D), torch.bfloat16, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((N1, T), torch.float32, q.device, stream)
    ws_bytes = workspace_size(dims)
    if ws_bytes and workspace is None:
        workspace = _empty(ws_bytes, torch.uint8, q.device, stream, result=False)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    st = lib().bsa_fp8_prefill(
        ctypes.byref(dims), _p(q), _p(k_pages), _p(v_pages), _p(q_descale), _p(k_descale),
        _p(v_descale), _p(cu_seqlens_q), _p(seqused_kv), _p(block_table), _p(block_mask),
        _p(sparse_indices), _p(sparse_seq_len), float(softmax_scale), float(p_scale), _p(out),
        _p(lse), _p(workspace), ws_bytes, _p(dev_status), _stream_handle(stream))
    if st != 0:
        raise BsaError(st, "bsa_fp8_prefill")
    return out, lse


def prefill_host(host: dict, dev: dict, max_q_len: int, max_kv_len: int,
                 softmax_scale: float | None = None, p_scale: float = 256.0, causal: bool = True,
                 workspace=None, dev_status=None, stream=None, k_scale_kind: int | None = None,
                 v_scale_kind: int | None = None, q_layout: int = Q_TND,
                 kv_layout: int = KV_HND, tiles_per_step: int = 1) -> None:
    """The prefill on host tensors (bsa_fp8_prefill_host).  `host` maps the names in
    TENSOR_NAMES to CPU tensors (page-locked ones make the copies asynchronous; absent or None
    = not given); "out" and "lse" receive the results once `stream` has been synchronised.
    `dev` maps the same names to CUDA tensors of the same shapes, which the call fills and
    computes on.  Scale kinds default as in prefill()."""
    import torch

    k_descale, v_descale = host["k_descale"], host["v_descale"]
    k_pages = host["k_pages"]
    n2 = k_pages.shape[2] if kv_layout == KV_NHD else k_pages.shape[1]
    k_kind = k_scale_kind if k_scale_kind is not None else (
        SCALE_PER_TOKEN_HEAD if k_descale.dim() == 3 else SCALE_PER_TENSOR)
    v_kind = v_scale_kind if v_scale_kind is not None else (
        SCALE_PER_HEAD if v_descale.numel() == n2 else SCALE_PER_TENSOR)
    dims = make_dims(host["q"], k_pages, host["block_table"], host["cu_seqlens_q"], max_q_len,
                     max_kv_len, k_kind, v_kind, causal, q_layout, kv_layout, tiles_per_step)
    ws_bytes = workspace_size(dims)
    if ws_bytes and workspace is None:
        workspace = _empty(ws_bytes, torch.uint8, dev["q"].device, stream, result=False)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(dims.D)
    th = Tensors(*(_p(host.get(n)) for n in TENSOR_NAMES))
    td = Tensors(*(_p(dev.get(n)) for n in TENSOR_NAMES))
    st = lib().bsa_fp8_prefill_host(ctypes.byref(dims), ctypes.byref(th), ctypes.byref(td),
                                    float(softmax_scale), float(p_scale), _p(workspace),
                                    ws_bytes, _p(dev_status), _stream_handle(stream))
    if st != 0:
        raise BsaError(st, "bsa_fp8_prefill_host")


def compact_tiles(cu_seqlens_q, seqused_kv, dims: Dims, block_mask=None, sparse_indices=None,
                  sparse_seq_len=None, dev_status=None, stream=None):
    """Active-tile lists [B, N1, Qb, Kb] (-1 past the count) and counts [B, N1, Qb]."""
    import torch

    Qb = -(-dims.max_q_len // 128)
    Kb = -(-dims.max_kv_len // 128)
    dev = cu_seqlens_q.device
    lists = _empty((dims.B, dims.N1, Qb, Kb), torch.int32, dev, stream)
    counts = _empty((dims.B, dims.N1, Qb), torch.int32, dev, stream)
    st = lib().bsa_fp8_compact_tiles(ctypes.byref(dims), _p(cu_seqlens_q), _p(seqused_kv),
                                     _p(block_mask), _p(sparse_indices), _p(sparse_seq_len),
                                     _p(lists), _p(counts), _p(dev_status),
                                     _stream_handle(stream))
    if st != 0:
        raise BsaError(st, "bsa_fp8_compact_tiles")
    return lists, counts


def quantize_rows(x, codes=None, descale=None, stream=None, rule: int = DESCALE_AMAX):
    """bf16 tensor [..., 128] -> (e4m3 codes uint8 [..., 128], fp32 descale [...]): per row
    descale = amax / 448 (1 for a zero row), rounded up to a power of two under
    DESCALE_UE8M0; code = e4m3(x / descale)."""
    import torch

    if x.dtype != torch.bfloat16 or x.shape[-1] != 128 or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 tensor [..., 128]")
    if codes is None:
        codes = _empty(x.shape, torch.uint8, x.device, stream)
    if descale is None:
        descale = _empty(x.shape[:-1], torch.float32, x.device, stream)
    fn = lib().bsa_fp8_quantize_rows_ue8m0 if rule == DESCALE_UE8M0 else lib().bsa_fp8_quantize_rows
    st = fn(_p(x), x.numel() // 128, _p(codes), _p(descale), _stream_handle(stream))
    if st != 0:
        raise BsaError(st, "bsa_fp8_quantize_rows")
    return codes, descale


def append_kv(k_new, v_new, cu_seqlens_new, cache_seqlens, block_table, k_pages, v_pages,
              k_descale=None, k_scale=None, v_scale=None, k_scale_kind=SCALE_PER_TOKEN_HEAD,
              v_scale_kind=SCALE_PER_HEAD, dev_status=None, stream=None, kv_layout=KV_HND,
              k_descale_rule: int = DESCALE_AMAX, slot_map=None):
    """Writes bf16 K/V tokens [T_new, N2, 128] into the paged cache (k_pages / v_pages
    [P, N2, page_size, 128] (KV_HND) or [P, page_size, N2, 128] (KV_NHD) uint8 e4m3,
    k_descale [P, N2, page_size] for per-token K, computed under k_descale_rule) at positions
    cache_seqlens[b] + i through block_table [B, L]; in place; rows from cu_seqlens_new[B] on are
    skipped.  Behind assign_pages() give its
    slot_map i32 [T_new] (page * page_size + slot; negative: skipped) and None for cu_seqlens_new,
    cache_seqlens and block_table: rows that got no place are then skipped, where the table may still
    name pages that were given back and belong to another sequence by now."""
    if slot_map is not None:
        if cu_seqlens_new is not None or cache_seqlens is not None or block_table is not None:
            raise ValueError("slot_map takes the place of cu_seqlens_new, cache_seqlens and block_table")
    if kv_layout == KV_NHD:
        P, ps, N2, D = k_pages.shape
    else:
        P, N2, ps, D = k_pages.shape
    named = slot_map is not None
    if named:
        _, bf16, _, i32, codes = _torch_names()
        T, dev = k_new.shape[0], k_pages.get_device()
        _check_all(dev, ("k_new", k_new, bf16, (T, N2, D)), ("v_new", v_new, bf16, (T, N2, D)),
                   ("slot_map", slot_map, i32, (T,)))
        _check_codes("k_pages", k_pages, k_pages.shape, dev, codes)
        _check_codes("v_pages", v_pages, k_pages.shape, dev, codes)
    dims = AppendDims(B=0 if named else cu_seqlens_new.numel() - 1, N2=N2, D=D, page_size=ps,
                      num_pages=P, max_pages_per_seq=0 if named else block_table.shape[1],
                      total_new=k_new.shape[0],
                      k_scale_kind=k_scale_kind, v_scale_kind=v_scale_kind,
                      kv_layout=int(kv_layout), k_descale_rule=int(k_descale_rule))
    if named:
        _call(lib().bsa_fp8_append_kv_slots,
              (ctypes.byref(dims), _p(k_new), _p(v_new), _p(slot_map), _p(k_scale), _p(v_scale),
               _p(k_pages), _p(v_pages), _p(k_descale), _p(dev_status)), dev, stream,
              "bsa_fp8_append_kv_slots")
        return k_pages, v_pages, k_descale
    st = lib().bsa_fp8_append_kv(ctypes.byref(dims), _p(k_new), _p(v_new), _p(cu_seqlens_new),
                                 _p(cache_seqlens), _p(block_table), _p(k_scale), _p(v_scale),
                                 _p(k_pages), _p(v_pages), _p(k_descale), _p(dev_status),
                                 _stream_handle(stream))
    if st != 0:
        raise BsaError(st, "bsa_fp8_append_kv")
    return k_pages, v_pages, k_descale


# ---------------------------------------------------------------------------------------------
# serving: decode, gather_kv, merge_states
# ---------------------------------------------------------------------------------------------

# A serving loop makes these calls once a layer and token, so their checks are kept to a few plain
# comparisons a tensor (a refusal works out its message afterwards), and the names they need are
# looked up once.

_names = None


def _torch_names():
    """(torch, bf16, fp32, int32, the dtypes of e4m3 codes)."""
    global _names
    if _names is None:
        import torch

        _names = (torch, torch.bfloat16, torch.float32, torch.int32,
                  (torch.uint8, torch.float8_e4m3fn))
    return _names


def _check(name, t, dtype, shape, dev):
    """Raises ValueError unless `t` is a contiguous tensor of `dtype` (or of one of a tuple of them)
    and of `shape` on the CUDA device of index `dev` (-1: no CUDA device, which _call refuses)."""
    if (t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
        return
    dtypes = dtype if type(dtype) is tuple else (dtype,)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, q or the cache on another device")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _call(fn, args, dev, stream, what):
    """fn(*args, stream handle) with device `dev` current; raises BsaError on a status but 0."""
    torch = _torch_names()[0]
    if dev < 0:
        raise ValueError(f"{what}: tensors must be on a CUDA device")
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"{what}: the stream is on {stream.device}, the tensors on cuda:{dev}")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st != 0:
        raise BsaError(st, what)


def _check_status(dev_status, dev):
    if (dev_status.dtype is not _torch_names()[3] or dev_status.numel() < 1
            or dev_status.get_device() != dev):
        raise ValueError("dev_status must be an int32 tensor on the device of the others")


def _check_all(dev, *items):
    """_check() of several (name, tensor, dtype, shape); a call less for each that is in order."""
    for name, t, dtype, shape in items:
        if not (t.dtype is dtype and t.shape == shape and t.get_device() == dev
                and t.is_contiguous()):
            _check(name, t, dtype, shape, dev)


def _check_codes(name, t, shape, dev, codes):
    """_check() of a tensor that holds e4m3 codes as bytes or as such."""
    if (t.dtype in codes and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
        return
    _check(name, t, t.dtype if t.dtype in codes else codes, shape, dev)


def _check_fp4(k_pages, v_pages, k_scales, v_scales, pool, scales, dev):
    """The pages and block scales of a 4-bit cache; a side whose pages are None is not looked at."""
    codes = _torch_names()[4]
    for name, t, sc in (("k", k_pages, k_scales), ("v", v_pages, v_scales)):
        if t is None:
            continue
        if sc is None:
            raise ValueError(f"{name}_pages given without {name}_scales")
        if not (t.dtype is codes[0] and t.shape == pool and t.get_device() == dev
                and t.is_contiguous()):
            _check(name + "_pages", t, codes[0], pool, dev)
        if not (sc.dtype in codes and sc.shape == scales and sc.get_device() == dev
                and sc.is_contiguous()):
            _check_codes(name + "_scales", sc, scales, dev, codes)


def _pool(pages, kv_layout):
    """(pages, KV heads, page size, head dim) of a page pool."""
    shape = pages.shape
    if len(shape) != 4:
        raise ValueError(f"pages have shape {tuple(shape)}, expected four dimensions")
    P, a, b, D = shape
    return (P, b, a, D) if kv_layout == KV_NHD else (P, a, b, D)


def make_decode_dims(q, k_pages, block_table, max_kv_len, k_scale_kind, v_scale_kind,
                     kv_layout=KV_HND, sparse=False) -> DecodeDims:
    T, N1, D = q.shape
    P, N2, ps, _ = _pool(k_pages, kv_layout)
    # in the order of DecodeDims' fields
    return DecodeDims(block_table.shape[0], N1, N2, D, ps, max_kv_len, P, block_table.shape[1],
                      k_scale_kind, v_scale_kind, kv_layout,
                      QTYPE_E4M3 if q.element_size() == 1 else QTYPE_BF16,
                      q.stride(0) if T > 1 else N1 * D, 1 if sparse else 0)


def decode_workspace_size(dims: DecodeDims) -> int:
    """Bytes of workspace decode() needs for `dims` on the current device."""
    return int(lib().bsa_fp8_decode_workspace_size(ctypes.byref(dims)))


def _decode(what, size, fp4, cu_seqlens_q, q, k_pages, v_pages, k_scales, v_scales, k_descale,
            v_descale, seqused_kv, block_table, max_kv_len, q_descale, block_mask, sparse_indices,
            sparse_seq_len, softmax_scale, out, lse, return_lse, dev_status, workspace, stream,
            k_scale_kind, v_scale_kind, kv_layout):
    """decode() and decode_fp4(), which gives block scales."""
    torch, bf16, f32, i32, codes = _torch_names()
    dev = q.get_device()
    shape = q.shape
    if len(shape) != 3:
        raise ValueError(f"q has shape {tuple(shape)}, expected [B, N1, 128]")
    T, N1, D = shape
    B, packed = T, ()
    if cu_seqlens_q is not None:
        if cu_seqlens_q.dim() != 1 or cu_seqlens_q.shape[0] < 1:
            raise ValueError(f"cu_seqlens_q has shape {tuple(cu_seqlens_q.shape)}, expected [B + 1]")
        B = cu_seqlens_q.shape[0] - 1
        _check("cu_seqlens_q", cu_seqlens_q, i32, (B + 1,), dev)
        what, packed = what + "_rows", (T, cu_seqlens_q.data_ptr())
    is_bf16 = q.dtype is bf16
    if not is_bf16 and q.dtype not in codes:
        raise ValueError(f"q has dtype {q.dtype}, expected bf16 or e4m3 codes")
    q_stride = N1 * D
    if not q.is_contiguous():
        if q.stride(2) != 1 or (N1 > 1 and q.stride(1) != D):
            raise ValueError("q must be contiguous within a sequence's row")
        if T > 1:
            q_stride = q.stride(0)
            if q_stride >= 1 << 31:
                raise ValueError(f"q's rows lie {q_stride} elements apart: 2^31 - 1 at most")
    P, N2, ps, pool_d = _pool(k_pages, kv_layout)
    if pool_d != (D // 2 if fp4 else D):
        raise ValueError(f"k_pages has shape {tuple(k_pages.shape)}, q a head dim of {D}")
    table = block_table.shape
    if len(table) != 2:
        raise ValueError(f"block_table has shape {tuple(table)}, expected [B, L]")
    if k_scale_kind is not None:
        k_kind = k_scale_kind
    elif fp4:
        k_kind = SCALE_PER_HEAD if k_descale.numel() == N2 else SCALE_PER_TENSOR
    else:
        k_kind = SCALE_PER_TOKEN_HEAD if k_descale.dim() == 3 else SCALE_PER_TENSOR
    v_kind = v_scale_kind if v_scale_kind is not None else (
        SCALE_PER_HEAD if v_descale.numel() == N2 else SCALE_PER_TENSOR)
    pool = k_pages.shape
    if fp4:
        _check_fp4(k_pages, v_pages, k_scales, v_scales, pool, (P, N2, ps, 8), dev)
    else:
        _check_codes("k_pages", k_pages, pool, dev, codes)
        _check_codes("v_pages", v_pages, pool, dev, codes)
    _check("k_descale", k_descale, f32,
           (P, N2, ps) if k_kind == SCALE_PER_TOKEN_HEAD else
           (N2,) if k_kind == SCALE_PER_HEAD else (1,), dev)
    _check("v_descale", v_descale, f32, (N2,) if v_kind == SCALE_PER_HEAD else (1,), dev)
    _check("seqused_kv", seqused_kv, i32, (B,), dev)
    L = table[1]
    _check("block_table", block_table, i32, (B, L), dev)
    if q_descale is not None:
        _check("q_descale", q_descale, f32, (T, N1), dev)
    sparse = block_mask is not None or sparse_indices is not None
    if sparse:
        Kb = -(-int(max_kv_len) // 128)
        if block_mask is not None:
            _check("block_mask", block_mask,
                   torch.bool if block_mask.dtype is torch.bool else torch.uint8, (B, N1, Kb), dev)
        if sparse_indices is not None:
            _check("sparse_indices", sparse_indices, i32, (B, N1, Kb), dev)
        if sparse_seq_len is not None:
            _check("sparse_seq_len", sparse_seq_len, i32, (B, N1), dev)
    if out is None:
        out = _empty((T, N1, D), bf16, q.device, stream)
    else:
        _check("out", out, bf16, shape, dev)
    if lse is not None:
        _check("lse", lse, f32, (N1, T), dev)
    elif return_lse:
        lse = _empty((N1, T), f32, q.device, stream)
    if dev_status is not None:
        _check_status(dev_status, dev)
    # in the order of DecodeDims' fields, as make_decode_dims
    dims = DecodeDims(B, N1, N2, D, ps, int(max_kv_len), P, L, k_kind, v_kind, kv_layout,
                      QTYPE_BF16 if is_bf16 else QTYPE_E4M3, q_stride, sparse)
    if workspace is None:
        if dev < 0:
            raise ValueError("decode: tensors must be on a CUDA device")
        with torch.cuda.device(dev):
            nbytes = size(dims)
        workspace = _empty(nbytes, torch.uint8, q.device, stream, result=False)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on q's device")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    scales = (k_scales.data_ptr(), v_scales.data_ptr()) if fp4 else ()
    _call(getattr(lib(), what),
          (ctypes.byref(dims), *packed, q.data_ptr(), _p(q_descale), k_pages.data_ptr(),
           v_pages.data_ptr(), *scales, k_descale.data_ptr(), v_descale.data_ptr(), seqused_kv.data_ptr(),
           block_table.data_ptr(), _p(block_mask), _p(sparse_indices), _p(sparse_seq_len),
           float(softmax_scale), out.data_ptr(), _p(lse), workspace.data_ptr(), workspace.nbytes,
           _p(dev_status)), dev, stream, what)
    return out, lse


def decode(q, k_pages, v_pages, k_descale, v_descale, seqused_kv, block_table, max_kv_len: int,
           q_descale=None, block_mask=None, sparse_indices=None, sparse_seq_len=None,
           softmax_scale: float | None = None, out=None, lse=None, return_lse: bool = True,
           dev_status=None, workspace=None, stream=None, k_scale_kind: int | None = None,
           v_scale_kind: int | None = None, kv_layout: int = KV_HND, cu_seqlens_q=None):
    """Attention of one new token per sequence over the paged cache (whose seqused_kv counts the
    new token, appended beforehand).  q bf16 [B, N1, 128], or uint8/float8_e4m3fn with q_descale
    f32 [B, N1]; its rows may lie further apart than N1 * 128 (a slice of a wider projection).
    Pages, descales, block_table and scale kinds as in prefill(); seqused_kv i32 [B];
    block_mask u8 [B, N1, Kb] or sparse_indices i32 [B, N1, Kb] + sparse_seq_len i32 [B, N1]
    select 128-token tiles for each query head, Kb = ceil(max_kv_len / 128).
    Returns (out bf16 [B, N1, 128], lse f32 [N1, B] or None); a sequence without tokens, or a head
    without an enabled tile, gives 0 and -FLT_MAX.  `out` may be q itself.  `workspace`
    (decode_workspace_size bytes) must not be shared by calls in flight at once.
    With cu_seqlens_q i32 [B + 1], as assign_pages() gives it, q, q_descale, out and lse have a row
    for each sequence that has a new token, [T, N1, 128] and so on, row cu_seqlens_q[b] being
    sequence b's, and a sequence without one takes no part; rows behind the last sequence's get 0
    and -FLT_MAX, and so do those of a sequence with several (DEV_BAD_SEQLEN)."""
    return _decode("bsa_fp8_decode", decode_workspace_size, False, cu_seqlens_q, q, k_pages, v_pages,
                   None, None, k_descale, v_descale, seqused_kv, block_table, max_kv_len, q_descale,
                   block_mask, sparse_indices, sparse_seq_len, softmax_scale, out, lse, return_lse,
                   dev_status, workspace, stream, k_scale_kind, v_scale_kind, kv_layout)


def _gather_rows(name, t, dtype, shape, pages, stream):
    if t is None:
        return _empty(shape, dtype, pages.device, stream)
    _check(name, t, dtype, shape, pages.get_device())
    return t


def _gather(fn, what, fp4, k_pages, v_pages, k_scales, v_scales, k_descale, v_descale, cu_seqlens,
            block_table, total, cache_starts, k_out, v_out, out_dtype, dev_status, stream,
            k_scale_kind, v_scale_kind, kv_layout):
    """gather_kv() and gather_kv_fp4()."""
    torch, _, f32, i32, codes = _torch_names()
    pages = k_pages if k_pages is not None else v_pages
    if pages is None:
        raise ValueError("k_pages and v_pages are both None")
    dev = pages.get_device()
    P, N2, ps, D = _pool(pages, kv_layout)
    if fp4:
        D *= 2
        _check_fp4(k_pages, v_pages, k_scales, v_scales, pages.shape, (P, N2, ps, D // 16), dev)
    given = k_out if k_out is not None else v_out
    if out_dtype is None:
        out_dtype = given.dtype if given is not None else torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"out_dtype {out_dtype}: bf16 or float32")
    if block_table.dim() != 2:
        raise ValueError(f"block_table has shape {tuple(block_table.shape)}, expected [B, L]")
    B, L = block_table.shape
    _check("block_table", block_table, i32, (B, L), dev)
    _check("cu_seqlens", cu_seqlens, i32, (B + 1,), dev)
    if cache_starts is not None:
        _check("cache_starts", cache_starts, i32, (B,), dev)
    if dev_status is not None:
        _check_status(dev_status, dev)
    total = int(total)
    k_kind = v_kind = SCALE_PER_TENSOR
    shape = (total, N2, D)
    if k_pages is not None:
        if k_scale_kind is not None:
            k_kind = k_scale_kind
        elif fp4:
            k_kind = SCALE_PER_HEAD if k_descale.numel() == N2 else SCALE_PER_TENSOR
        else:
            k_kind = SCALE_PER_TOKEN_HEAD if k_descale.dim() == 3 else SCALE_PER_TENSOR
        if not fp4:
            _check_codes("k_pages", k_pages, pages.shape, dev, codes)
        _check("k_descale", k_descale, f32,
               (P, N2, ps) if k_kind == SCALE_PER_TOKEN_HEAD else
               (N2,) if k_kind == SCALE_PER_HEAD else (1,), dev)
        k_out = _gather_rows("k_out", k_out, out_dtype, shape, pages, stream)
    elif k_out is not None:
        raise ValueError("k_out given without k_pages")
    if v_pages is not None:
        v_kind = v_scale_kind if v_scale_kind is not None else (
            SCALE_PER_HEAD if v_descale.numel() == N2 else SCALE_PER_TENSOR)
        if not fp4:
            _check_codes("v_pages", v_pages, pages.shape, dev, codes)
        _check("v_descale", v_descale, f32, (N2,) if v_kind == SCALE_PER_HEAD else (1,), dev)
        v_out = _gather_rows("v_out", v_out, out_dtype, shape, pages, stream)
    elif v_out is not None:
        raise ValueError("v_out given without v_pages")
    # in the order of GatherDims' fields
    dims = GatherDims(B, N2, D, ps, P, L, total, k_kind, v_kind, kv_layout,
                      OUT_FP32 if out_dtype is torch.float32 else OUT_BF16)
    scales = (_p(k_scales), _p(v_scales)) if fp4 else ()
    _call(fn,
          (ctypes.byref(dims), _p(k_pages), _p(v_pages), *scales, _p(k_descale), _p(v_descale),
           cu_seqlens.data_ptr(), _p(cache_starts), block_table.data_ptr(), _p(k_out), _p(v_out),
           _p(dev_status)), dev, stream, what)
    return k_out, v_out


def gather_kv(k_pages, v_pages, k_descale, v_descale, cu_seqlens, block_table, total: int,
              cache_starts=None, k_out=None, v_out=None, out_dtype=None, dev_status=None,
              stream=None, k_scale_kind: int | None = None, v_scale_kind: int | None = None,
              kv_layout: int = KV_HND):
    """Reads tokens back from the paged cache: row cu_seqlens[b] + i of the returned k, v
    [total, N2, 128] is the token at position cache_starts[b] + i (0 + i without it) of sequence
    b, code * descale.  out_dtype bf16 (default) or float32, or that of k_out / v_out when given;
    rows from cu_seqlens[B] on are left as they were.  k_pages = None or v_pages = None leaves
    that side out (returned as None)."""
    return _gather(lib().bsa_fp8_gather_kv, "bsa_fp8_gather_kv", False, k_pages, v_pages, None, None,
                   k_descale, v_descale, cu_seqlens, block_table, total, cache_starts, k_out, v_out,
                   out_dtype, dev_status, stream, k_scale_kind, v_scale_kind, kv_layout)


def merge_states(outs, lses, out=None, lse=None, return_lse: bool = True, stream=None):
    """Joins attention results over disjoint sets of keys: outs are 1 to MAX_MERGE bf16 tensors
    [T, N1, 128] and lses their fp32 LSEs [N1, T], as prefill() and decode() return them (for
    decode T = B).  Returns (out, lse) over the union of the keys.  `out` may be one of `outs`
    and `lse` one of `lses`; memory that overlaps in part is refused."""
    torch, bf16, f32, _, _ = _torch_names()
    n = len(outs)
    if n < 1 or n > MAX_MERGE or len(lses) != n:
        raise ValueError(f"{n} outs and {len(lses)} lses: 1 to {MAX_MERGE} of each")
    first = outs[0]
    dev = first.get_device()
    if first.dim() != 3 or first.shape[2] != 128:
        raise ValueError(f"outs[0] has shape {tuple(first.shape)}, expected [T, N1, 128]")
    shape = first.shape
    T, N1, _ = shape
    for o in outs:
        _check("outs", o, bf16, shape, dev)
    for x in lses:
        _check("lses", x, f32, (N1, T), dev)
    if out is None:
        out = _empty(shape, bf16, first.device, stream)
    else:
        _check("out", out, bf16, shape, dev)
    if lse is not None:
        _check("lse", lse, f32, (N1, T), dev)
    elif return_lse:
        lse = _empty((N1, T), f32, first.device, stream)
    ptrs = ctypes.c_void_p * n
    _call(lib().bsa_fp8_merge_states,
          (n, ptrs(*[o.data_ptr() for o in outs]), ptrs(*[x.data_ptr() for x in lses]), T, N1,
           out.data_ptr(), _p(lse)), dev, stream, "bsa_fp8_merge_states")
    return out, lse


# ---------------------------------------------------------------------------------------------
# around attention: rotary positions, pages, the 4-bit cache
# ---------------------------------------------------------------------------------------------

def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: int = ROPE_NONE,
                     factor: float = 1.0, context: float = 0.0, slow: float = 1.0,
                     fast: float = 32.0, inv_freq=None, device=None):
    """The frequencies rope() takes: an int64 tensor [rotary_dim / 2] of turns per position times
    2^64, modulo 2^64.  f_i = base^(-2i / rotary_dim) radians a position, stretched by `factor`:
    ROPE_LINEAR f_i / factor; ROPE_BASE base * factor^(R / (R - 2)); ROPE_PARTS f_i where a dimension
    turns more than `fast` times within `context` positions, f_i / factor where fewer than `slow`
    times, a blend, linear in the number of turns, between (a model whose blend is linear in the number
    of the dimension needs inv_freq).  inv_freq (rotary_dim / 2 numbers, radians a position) gives frequencies
    of the caller's own instead.  Made on the host, once for a model."""
    import torch

    n = int(rotary_dim) // 2
    out = (ctypes.c_uint64 * max(n, 1))()
    own = None
    if inv_freq is not None:
        values = [float(x) for x in inv_freq]
        if len(values) != n:
            raise ValueError(f"{len(values)} frequencies, expected {n}")
        own = (ctypes.c_double * n)(*values)
    st = lib().bsa_rope_frequencies(int(rotary_dim), int(scaling), base, factor, context, slow, fast,
                                    own, out)
    if st != 0:
        raise BsaError(st, "bsa_rope_frequencies")
    signed = [x - (1 << 64) if x >> 63 else x for x in out]
    return torch.tensor(signed, dtype=torch.int64, device=device)


def _rows(name, t, T, dev):
    """The stride from token to token of a bf16 tensor [T, heads, 128] whose tokens are each in one
    piece."""
    shape, stride = t.shape, t.stride()
    if (t.dtype is _torch_names()[1] and len(shape) == 3 and shape[2] == 128 and shape[0] == T
            and stride[2] == 1 and (stride[1] == 128 or shape[1] == 1) and t.get_device() == dev):
        return stride[0] if T > 1 else shape[1] * 128
    if t.dtype is not _torch_names()[1]:
        raise ValueError(f"{name} has dtype {t.dtype}, expected bf16")
    if len(shape) != 3 or shape[2] != 128 or shape[0] != T:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [{T}, heads, 128]")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the others on another device")
    raise ValueError(f"{name} must be contiguous within a token")


def _rope_common(q, positions, freqs):
    torch, _, _, i32, _ = _torch_names()
    if q.dim() != 3:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [T, N1, 128]")
    T, dev, n = q.shape[0], q.get_device(), freqs.shape
    if len(n) != 1:
        raise ValueError(f"freqs has shape {tuple(n)}, expected [rotary_dim / 2]")
    _check_all(dev, ("positions", positions, i32, (T,)), ("freqs", freqs, torch.int64, n))
    return T, dev, _rows("q", q, T, dev)


def rope(q, positions, freqs, k=None, layout: int = ROPE_HALF, amplitude: float = 1.0, out=None,
         k_out=None, stream=None):
    """Rotary positions of q bf16 [T, N1, 128] and, in the same launch, k bf16 [T, N2, 128]: pairs of
    the first 2 * len(freqs) values of every head (value i with i + len(freqs) under ROPE_HALF, 2i
    with 2i + 1 under ROPE_INTERLEAVED) turned by position * frequency and multiplied by `amplitude`,
    the rest of the head copied.  positions i32 [T]; freqs from rope_frequencies().  Tokens may lie
    further apart than their heads fill (slices of a wider projection).  out / k_out may be q / k
    themselves.  Returns (out, k_out), k_out None without k."""
    bf16 = _torch_names()[1]
    T, dev, q_stride = _rope_common(q, positions, freqs)
    N1, N2 = q.shape[1], 0
    k_stride = k_out_stride = 0
    if out is None:
        out = _empty(q.shape, bf16, q.device, stream)
    q_out_stride = _rows("out", out, T, dev)
    if out.shape != q.shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(q.shape)}")
    if k is not None:
        k_stride = _rows("k", k, T, dev)
        N2 = k.shape[1]
        if k_out is None:
            k_out = _empty(k.shape, bf16, k.device, stream)
        k_out_stride = _rows("k_out", k_out, T, dev)
        if k_out.shape != k.shape:
            raise ValueError(f"k_out has shape {tuple(k_out.shape)}, expected {tuple(k.shape)}")
    elif k_out is not None:
        raise ValueError("k_out given without k")
    # in the order of RopeDims' fields
    dims = RopeDims(T, N1, N2, 128, 2 * freqs.shape[0], layout, q_stride, k_stride, q_out_stride,
                    k_out_stride)
    _call(lib().bsa_rope,
          (ctypes.byref(dims), q.data_ptr(), _p(k), positions.data_ptr(), freqs.data_ptr(),
           amplitude, out.data_ptr(), _p(k_out)), dev, stream, "bsa_rope")
    return out, k_out


def rope_quantize(q, positions, freqs, layout: int = ROPE_HALF, amplitude: float = 1.0, codes=None,
                  descale=None, rule: int = DESCALE_AMAX, stream=None):
    """rope() of q alone and quantize_rows() of the result in one, without rounding to bf16 in
    between: (e4m3 codes uint8 [T, N1, 128], fp32 descale [T, N1]), as prefill() and decode() take
    queries."""
    torch, _, f32, _, kinds = _torch_names()
    T, dev, q_stride = _rope_common(q, positions, freqs)
    N1 = q.shape[1]
    if codes is None:
        codes = _empty(q.shape, torch.uint8, q.device, stream)
    else:
        _check("codes", codes, codes.dtype if codes.dtype in kinds else kinds, q.shape, dev)
    if descale is None:
        descale = _empty((T, N1), f32, q.device, stream)
    else:
        _check("descale", descale, f32, (T, N1), dev)
    dims = RopeDims(T, N1, 0, 128, 2 * freqs.shape[0], layout, q_stride, 0, 0, 0)
    _call(lib().bsa_rope_quantize,
          (ctypes.byref(dims), q.data_ptr(), positions.data_ptr(), freqs.data_ptr(), amplitude,
           int(rule), codes.data_ptr(), descale.data_ptr()), dev, stream, "bsa_rope_quantize")
    return codes, descale


def _check_pages(block_table, free_pages, free_count, B, dev):
    i32 = _torch_names()[3]
    if block_table.dim() != 2:
        raise ValueError(f"block_table has shape {tuple(block_table.shape)}, expected [B, L]")
    if free_pages.dim() != 1:
        raise ValueError(f"free_pages has shape {tuple(free_pages.shape)}, expected [num_pages]")
    L = block_table.shape[1]
    _check_all(dev, ("block_table", block_table, i32, (B, L)),
               ("free_pages", free_pages, i32, free_pages.shape),
               ("free_count", free_count, i32, (1,)))
    return L


def assign_pages(new_lens, cache_seqlens, block_table, free_pages, free_count, page_size: int,
                 total: int, cu_seqlens=None, seqused_kv=None, positions=None, slot_map=None,
                 dev_status=None, stream=None):
    """Gives every sequence the pages for its new_lens i32 [B] tokens behind the cache_seqlens i32
    [B] that it holds, and says where those tokens go.  block_table i32 [B, L] gets the new pages;
    free_pages i32 [num_pages] is a stack whose first free_count i32 [1] entries are free: pages are
    taken from its top in the sequences' order.  Returns (cu_seqlens i32 [B + 1], seqused_kv i32
    [B], positions i32 [total], slot_map i32 [total]): the new tokens' first rows, the lengths
    afterwards, and each new token's position in its sequence and its slot (page * page_size +
    slot), as prefill(), both decodes (cu_seqlens_q), rope(), append_kv() and append_kv_fp4() take
    them; rows from
    cu_seqlens[B] on get position 0 and slot -1.  A sequence whose pages are not there gets none:
    slots -1, its length unchanged, DEV_NO_PAGES (the table keeps whatever it named before, so both
    appends take the slots).  seqused_kv must not be cache_seqlens."""
    i32 = _torch_names()[3]
    if new_lens.dim() != 1:
        raise ValueError(f"new_lens has shape {tuple(new_lens.shape)}, expected [B]")
    B, dev, total = new_lens.shape[0], new_lens.get_device(), int(total)
    _check_all(dev, ("new_lens", new_lens, i32, (B,)), ("cache_seqlens", cache_seqlens, i32, (B,)))
    L = _check_pages(block_table, free_pages, free_count, B, dev)
    if dev_status is not None:
        _check_status(dev_status, dev)
    outs = []
    for name, t, n in (("cu_seqlens", cu_seqlens, B + 1), ("seqused_kv", seqused_kv, B),
                       ("positions", positions, total), ("slot_map", slot_map, total)):
        if t is None:
            t = _empty((n,), i32, new_lens.device, stream)
        elif not (t.dtype is i32 and t.shape == (n,) and t.get_device() == dev
                  and t.is_contiguous()):
            _check(name, t, i32, (n,), dev)
        outs.append(t)
    dims = PagesDims(B, int(page_size), free_pages.shape[0], L, total)
    _call(lib().bsa_assign_pages,
          (ctypes.byref(dims), new_lens.data_ptr(), cache_seqlens.data_ptr(),
           block_table.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(),
           outs[0].data_ptr(), outs[1].data_ptr(), outs[2].data_ptr(), outs[3].data_ptr(),
           _p(dev_status)), dev, stream, "bsa_assign_pages")
    return tuple(outs)


def release_pages(seq_lens, keep_lens, block_table, free_pages, free_count, page_size: int,
                  out=None, dev_status=None, stream=None):
    """Cuts every sequence down to its first keep_lens i32 [B] tokens (0: all of it goes) and puts the
    pages that hold none of them back on the stack, so that a release undoes the assign_pages()
    before it.  Returns the lengths afterwards (`out`, which may be either length itself).  A page must be
    held by one sequence only."""
    i32 = _torch_names()[3]
    if seq_lens.dim() != 1:
        raise ValueError(f"seq_lens has shape {tuple(seq_lens.shape)}, expected [B]")
    B, dev = seq_lens.shape[0], seq_lens.get_device()
    _check_all(dev, ("seq_lens", seq_lens, i32, (B,)), ("keep_lens", keep_lens, i32, (B,)))
    L = _check_pages(block_table, free_pages, free_count, B, dev)
    if dev_status is not None:
        _check_status(dev_status, dev)
    if out is None:
        out = _empty((B,), i32, seq_lens.device, stream)
    else:
        _check("out", out, i32, (B,), dev)
    dims = PagesDims(B, int(page_size), free_pages.shape[0], L, 0)
    _call(lib().bsa_release_pages,
          (ctypes.byref(dims), seq_lens.data_ptr(), keep_lens.data_ptr(), block_table.data_ptr(),
           free_pages.data_ptr(), free_count.data_ptr(), out.data_ptr(), _p(dev_status)), dev,
          stream, "bsa_release_pages")
    return out


def _fp4_kind(given, descale, N2):
    if given is not None:
        return given
    return SCALE_PER_HEAD if descale.numel() == N2 else SCALE_PER_TENSOR


def append_kv_fp4(k_new, v_new, slot_map, k_pages, v_pages, k_scales, v_scales, k_descale, v_descale,
                  dev_status=None, stream=None, k_scale_kind: int | None = None,
                  v_scale_kind: int | None = None, kv_layout: int = KV_HND):
    """Writes bf16 K/V tokens [T_new, N2, 128] (tokens may lie further apart) into the 4-bit cache at
    slot_map i32 [T_new] (page * page_size + slot, as assign_pages() gives it; negative: skipped),
    in place.  Pages uint8 [P, N2, page_size, 64] (KV_HND) or [P, page_size, N2, 64] (KV_NHD) hold
    e2m1 codes, two to a byte; k_scales / v_scales uint8 or float8_e4m3fn [P, N2, page_size, 8] a
    scale for every 16 of them; k_descale / v_descale f32 [1] or [N2], chosen by the caller (the
    largest value expected / 2688 uses the scales' whole range).  value = code * scale * descale."""
    f32, i32 = _torch_names()[2:4]
    T, dev = k_new.shape[0], k_new.get_device()
    k_stride, v_stride = _rows("k_new", k_new, T, dev), _rows("v_new", v_new, T, dev)
    P, N2, ps, half = _pool(k_pages, kv_layout)
    if half != 64 or k_new.shape[1] != N2 or v_new.shape[1] != N2:
        raise ValueError(f"pages of shape {tuple(k_pages.shape)} do not hold rows "
                         f"{tuple(k_new.shape)} and {tuple(v_new.shape)} in 4 bits")
    _check_fp4(k_pages, v_pages, k_scales, v_scales, k_pages.shape, (P, N2, ps, 8), dev)
    k_kind, v_kind = _fp4_kind(k_scale_kind, k_descale, N2), _fp4_kind(v_scale_kind, v_descale, N2)
    _check_all(dev, ("k_descale", k_descale, f32, (N2,) if k_kind == SCALE_PER_HEAD else (1,)),
               ("v_descale", v_descale, f32, (N2,) if v_kind == SCALE_PER_HEAD else (1,)),
               ("slot_map", slot_map, i32, (T,)))
    if dev_status is not None:
        _check_status(dev_status, dev)
    dims = Fp4AppendDims(N2, 128, ps, P, T, k_kind, v_kind, int(kv_layout), k_stride, v_stride)
    _call(lib().bsa_fp4_append_kv,
          (ctypes.byref(dims), k_new.data_ptr(), v_new.data_ptr(), slot_map.data_ptr(),
           k_descale.data_ptr(), v_descale.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
           k_scales.data_ptr(), v_scales.data_ptr(), _p(dev_status)), dev, stream,
          "bsa_fp4_append_kv")
    return k_pages, v_pages, k_scales, v_scales


def gather_kv_fp4(k_pages, v_pages, k_scales, v_scales, k_descale, v_descale, cu_seqlens,
                  block_table, total: int, cache_starts=None, k_out=None, v_out=None,
                  out_dtype=None, dev_status=None, stream=None, k_scale_kind: int | None = None,
                  v_scale_kind: int | None = None, kv_layout: int = KV_HND):
    """gather_kv() from a 4-bit cache (append_kv_fp4() says how it lies)."""
    return _gather(lib().bsa_fp4_gather_kv, "bsa_fp4_gather_kv", True, k_pages, v_pages, k_scales,
                   v_scales, k_descale, v_descale, cu_seqlens, block_table, total, cache_starts,
                   k_out, v_out, out_dtype, dev_status, stream, k_scale_kind, v_scale_kind,
                   kv_layout)


def decode_fp4_workspace_size(dims: DecodeDims) -> int:
    """Bytes of workspace decode_fp4() needs for `dims` on the current device."""
    return int(lib().bsa_fp4_decode_workspace_size(ctypes.byref(dims)))


def decode_fp4(q, k_pages, v_pages, k_scales, v_scales, k_descale, v_descale, seqused_kv, block_table,
               max_kv_len: int, q_descale=None, block_mask=None, sparse_indices=None,
               sparse_seq_len=None, softmax_scale: float | None = None, out=None, lse=None,
               return_lse: bool = True, dev_status=None, workspace=None, stream=None,
               k_scale_kind: int | None = None, v_scale_kind: int | None = None,
               kv_layout: int = KV_HND, cu_seqlens_q=None):
    """decode() over a 4-bit cache (append_kv_fp4() says how it lies): the same queries, packed ones
    too, selection of tiles, outputs and rules; `workspace` has decode_fp4_workspace_size bytes."""
    return _decode("bsa_fp4_decode", decode_fp4_workspace_size, True, cu_seqlens_q, q, k_pages,
                   v_pages, k_scales, v_scales, k_descale, v_descale, seqused_kv, block_table,
                   max_kv_len, q_descale, block_mask, sparse_indices, sparse_seq_len, softmax_scale,
                   out, lse, return_lse, dev_status, workspace, stream, k_scale_kind, v_scale_kind,
                   kv_layout)
