"""What the bindings do around a call (no GPU: the library and the allocator are fakes)."""
import contextlib

import pytest
import torch

import block_sparse_fp8_gb300 as bsa


class _Library:
    """Stands in for the compiled library: every call succeeds, every workspace has 512 bytes."""

    def __getattr__(self, name):
        return lambda *args: 512 if name.endswith("_size") else 0


class _Allocations:
    """Records, for each tensor made, the stream that was current."""

    def __init__(self, monkeypatch):
        self.current, self.seen = None, []
        empty = torch.empty

        @contextlib.contextmanager
        def on(stream):
            before, self.current = self.current, stream
            yield
            self.current = before

        def made(*args, **kw):
            self.seen.append(self.current)
            return empty(*args, **kw)

        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch, "empty", made)
        monkeypatch.setattr(bsa, "lib", lambda: _Library())


class _Stream:
    cuda_stream = 0
    device = torch.device("cuda", 0)


def _calls():
    bf16, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    q8, pages = torch.zeros(4, 8, 128, dtype=u8), torch.zeros(6, 2, 32, 128, dtype=u8)
    kd, vd = torch.zeros(6, 2, 32), torch.zeros(2)
    cu, used, table = (torch.zeros(*s, dtype=i32) for s in ((3,), (2,), (2, 3)))
    dims = bsa.make_dims(q8, pages, table, cu, 4, 90, 1, 2)
    o, l = torch.zeros(3, 4, 128, dtype=bf16), torch.zeros(4, 3)
    host = dict(q=q8, k_pages=pages, v_pages=pages, q_descale=torch.zeros(4, 8), k_descale=kd,
                v_descale=vd, cu_seqlens_q=cu, seqused_kv=used, block_table=table)
    return {
        "prefill": (3, lambda **k: bsa.prefill(q8, pages, pages, torch.zeros(4, 8), kd, vd, cu, used,
                                               table, 4, 90, **k)),
        "prefill_host": (1, lambda **k: bsa.prefill_host(host, host, 4, 90, **k)),
        "compact_tiles": (2, lambda **k: bsa.compact_tiles(cu, used, dims, **k)),
        "quantize_rows": (2, lambda **k: bsa.quantize_rows(o, **k)),
        # refused for their CPU tensors, after the outputs were made
        "decode": (2, lambda **k: bsa.decode(torch.zeros(2, 8, 128, dtype=bf16), pages, pages, kd, vd,
                                             used, table, 90, **k)),
        "gather_kv": (2, lambda **k: bsa.gather_kv(pages, pages, kd, vd, cu, table, 4, **k)),
        "merge_states": (2, lambda **k: bsa.merge_states([o, o], [l, l], **k)),
    }


@pytest.mark.parametrize("name", list(_calls()))
def test_tensors_come_from_the_stream_of_the_call(name, monkeypatch):
    """Whatever a call on a named stream makes for itself is allocated with that stream current."""
    count, call = _calls()[name]
    a = _Allocations(monkeypatch)
    side = _Stream()
    with contextlib.suppress(ValueError):
        call(stream=side)
    assert a.seen == [side] * count


def test_merge_refuses_memory_that_overlaps_in_part():
    """Outputs may be one of the inputs; any other overlap is refused before CUDA is touched."""
    import ctypes
    import os
    import shutil

    from block_sparse_fp8_gb300 import _build

    if _build.needs_build():
        if shutil.which(_build.nvcc()) is None and not os.path.exists(_build.nvcc()):
            pytest.skip("nvcc not available")
        _build.build()
    T, N1 = 4, 8
    O, L = T * N1 * 256, T * N1 * 4                     # bytes of a part's O and LSE
    a, b, la, lb, end = 1 << 20, 2 << 20, 3 << 20, 4 << 20, 5 << 20      # never dereferenced

    def status(out, lse):
        outs, lses = (ctypes.c_void_p * 2)(a, b), (ctypes.c_void_p * 2)(la, lb)
        return bsa.lib().bsa_fp8_merge_states(2, outs, lses, T, N1, out, lse, None)

    for out, lse in ((a + 256, end), (b - 16, end), (b + O - 16, end), (end, la + 4),
                     (end, lb + L - 4), (end, lb - 4), (la, end), (lb - O + 16, end), (end, a),
                     (end, b + O - 4), (end, end), (end, end + O - 4), (a, b), (a + 256, None),
                     (a, la + 4)):
        assert status(out, lse) == 1, (out, lse)
