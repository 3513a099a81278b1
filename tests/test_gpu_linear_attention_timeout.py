"""Outputs of a call whose bounded wait ran out are NaN, so that they are not taken for results before
linear_attention_sync reports the wait."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_weight_memory_chunk_b200 import fwpkm  # noqa: E402


@pytest.mark.parametrize("B,H,T,d,dv", [(2, 4, 300, 64, 64), (1, 2, 1100, 128, 72), (80, 1, 128, 64, 128)])
def test_outputs_of_a_wait_that_ran_out_are_nan(B, H, T, d, dv):
    g = torch.Generator("cuda").manual_seed(T)
    q, k = (torch.randn(B, T, H, d, generator=g, device="cuda").bfloat16().transpose(1, 2) for _ in range(2))
    v = torch.randn(B, T, H, dv, generator=g, device="cuda").bfloat16().transpose(1, 2)
    ld = torch.full((H,), -0.1, device="cuda")
    lens = torch.tensor([T if b % 2 == 0 else T - 20 for b in range(B)], dtype=torch.int32, device="cuda")
    out = lambda: torch.full_like(v, 7.0)  # noqa: E731
    want = fwpkm.linear_attention(q, k, v, ld, lens=lens, o=out(), final_state=True)
    fwpkm.linear_attention_sync()
    fwpkm.test_stall_waits(1)
    o, sT = fwpkm.linear_attention(q, k, v, ld, lens=lens, o=out(), final_state=True)
    with pytest.raises(fwpkm.FwpkmError) as e:
        fwpkm.linear_attention_sync()
    assert e.value.status == fwpkm.ERR_TIMEOUT
    for b, n in enumerate(lens.tolist()):
        assert torch.isnan(o[b, :, n - 1].float()).all() and torch.isnan(sT[b]).all()
        assert (o[b, :, n:] == 7.0).all()          # rows behind the end are still the caller's
        if n <= 128:
            assert torch.isnan(o[b, :, :n].float()).all()
    got = fwpkm.linear_attention(q, k, v, ld, lens=lens, o=out(), final_state=True)
    fwpkm.linear_attention_sync()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
