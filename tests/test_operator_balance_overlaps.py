"""The balance loss's gradient in the memory of its logits is refused on the host where the logits are not
contiguous (their rows are then not the gradient's), before anything is enqueued."""
import ctypes as C

import pytest

pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from sparse_weight_memory_chunk_b200 import build, fwpkm
    build.build()
    return fwpkm


X, SLOPE = C.c_void_p(2 << 28), C.c_void_p(3 << 28)


@pytest.mark.parametrize("tokens,ld,stride,groups", [(10, 16, 160, 2), (10, 8, 96, 2), (10, 8, 0, 2), (10, 16, 0, 1)])
def test_a_gradient_in_the_memory_of_strided_logits_is_refused(lib, tokens, ld, stride, groups):
    cfg = C.byref(lib.BalanceConfig(tokens, ld, stride, groups, 8, 0, lib.F32, 1, 1.0))
    assert lib.lib().fwpkm_balance_loss_backward(cfg, X, None, SLOPE, None, X, None) == lib.ERR_INVALID_ARG
