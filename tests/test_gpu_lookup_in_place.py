"""The weights' gradient in the weights' own memory: refused where the table's gradient reads them after
it, and what it should be where nothing does."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_weight_memory_chunk_b200 import fwpkm  # noqa: E402


@pytest.mark.parametrize("n", [300, 30000])  # pairs sorted in one launch, and by passes
def test_dw_in_the_memory_of_w(n):
    g = torch.Generator("cuda").manual_seed(n)
    table, d_out = torch.randn(500, 64, generator=g, device="cuda"), torch.randn(n, 64, generator=g, device="cuda")
    idx = torch.randint(-1, 500, (n, 4), generator=g, device="cuda", dtype=torch.int32)
    both = torch.softmax(torch.randn(n + 1, 4, generator=g, device="cuda"), -1)
    w = both[:n]
    before = both.clone()
    for dw in (w, both[1:]):                   # the same memory, and all but a row of it
        with pytest.raises(fwpkm.FwpkmError) as e:
            fwpkm.lookup_backward(table, idx, d_out, w=w, dw=dw)
        assert e.value.status == fwpkm.ERR_INVALID_ARG
    assert torch.equal(both, before)
    d_table, dw = fwpkm.lookup_backward(table, idx, d_out, w=w)
    own = torch.empty(2 * n, 4, device="cuda")
    own[:n] = w
    d2, dw2 = fwpkm.lookup_backward(table, idx, d_out, w=own[:n], dw=own[n:])  # side by side
    assert torch.equal(d2, d_table) and torch.equal(dw2, dw) and dw2.data_ptr() == own[n:].data_ptr()
