"""Outputs of linear attention that begin where an input or another output does, and scales that
have no finite reciprocal, are refused on the host, before anything is enqueued (pointers are
aligned numbers that nothing reads)."""
import ctypes as C

import pytest

pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from sparse_weight_memory_chunk_b200 import build, fwpkm
    build.build()
    return fwpkm


def test_outputs_in_the_memory_of_inputs_are_refused(lib):
    so = lib.lib()
    cfg = C.byref(lib.LinattnConfig(2, 2, 32, 32, lib.F32, 1.0))
    fake, work = C.c_void_p(1 << 20), C.c_void_p(1 << 30)
    at = [C.byref(lib.Heads((i + 2) << 24, 1 << 16, 1 << 12, 64)) for i in range(8)]
    T, ws = 100, C.c_size_t(0)
    q, k, v, do = at[:4]
    for o in (q, k, v):
        assert so.fwpkm_linear_attention(cfg, q, k, v, T, fake, None, None, o, None, work, 1 << 40, None) == -1
        assert so.fwpkm_linear_attention_step(cfg, q, k, v, 1, fake, None, fake, o, fake, None) == -1
    assert so.fwpkm_linear_attention_workspace_size(cfg, T, 1, C.byref(ws)) == 0
    grads = at[4:7]
    for i in range(3):
        for other in (q, k, v, do, grads[(i + 1) % 3]):
            g = list(grads)
            g[i] = other
            assert so.fwpkm_linear_attention_backward(cfg, q, k, v, T, fake, None, None, do, None, *g, None, work,
                                                      1 << 40, None) == -1


@pytest.mark.parametrize("scale", [0.0, float("inf"), -float("inf"), float("nan"), 1e-39])
def test_scales_without_a_reciprocal_are_refused(lib, scale):
    so = lib.lib()
    cfg = C.byref(lib.LinattnConfig(2, 2, 32, 32, lib.F32, scale))
    fake, work = C.c_void_p(1 << 20), C.c_void_p(1 << 30)
    q, k, v, o = (C.byref(lib.Heads((i + 2) << 24, 1 << 16, 1 << 12, 64)) for i in range(4))
    assert so.fwpkm_linear_attention(cfg, q, k, v, 10, fake, None, None, o, None, work, 1 << 40, None) == -1
    assert so.fwpkm_linear_attention_step(cfg, q, k, v, 1, fake, None, fake, o, fake, None) == -1
