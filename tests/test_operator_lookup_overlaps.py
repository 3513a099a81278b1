"""Lookups whose outputs lie in the memory of what the call still has to read are refused on the host,
before anything is enqueued (pointers are aligned numbers that nothing reads)."""
import ctypes as C

import pytest

pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from sparse_weight_memory_chunk_b200 import build, fwpkm
    build.build()
    return fwpkm


TABLE, IDX, W, D_OUT, D_TABLE, DW, WORK = (C.c_void_p((i + 2) << 28) for i in range(7))


def test_outputs_in_the_memory_of_inputs_are_refused(lib):
    so, n, R = lib.lib(), 6, 4
    cfg = C.byref(lib.LookupConfig(100, 64, 64, 64, R, lib.F32, lib.I32, 1.0))
    ws = C.c_size_t(0)
    assert so.fwpkm_lookup_backward_workspace_size(cfg, n, C.byref(ws)) == 0
    for out in (TABLE, W):
        assert so.fwpkm_lookup(cfg, TABLE, IDX, W, n, out, None) == lib.ERR_INVALID_ARG

    def back(d_table, dw, w=W):
        return so.fwpkm_lookup_backward(cfg, TABLE, IDX, w, D_OUT, n, d_table, 64, lib.F32, 1, dw, WORK, ws.value, None)

    end = 4 * n * R
    for dw in (W.value, W.value + 4, W.value + end - 4, W.value - 4, W.value - end + 4):
        assert back(D_TABLE, C.c_void_p(dw)) == lib.ERR_INVALID_ARG
    assert back(D_TABLE, D_OUT) == back(D_TABLE, TABLE) == back(None, D_OUT) == back(None, TABLE) == lib.ERR_INVALID_ARG
    assert back(D_OUT, None) == back(D_OUT, DW) == back(W, None) == lib.ERR_INVALID_ARG
