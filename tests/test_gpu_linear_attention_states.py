"""States of linear attention that pass through without a token, beside sequences that keep the GPU
busy: whatever the other heads do, an empty sequence's state leaves as it came, bit for bit."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_weight_memory_chunk_b200 import fwpkm  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,H,T,d,dv", [(16, 16, 1024, 128, 128), (16, 16, 300, 64, 128), (3, 2, 4000, 128, 64)])
def test_states_of_empty_sequences_leave_as_they_came(B, H, T, d, dv, dtype):
    g = torch.Generator("cuda").manual_seed(B + T)
    q, k = (torch.randn(B, T, H, d, generator=g, device="cuda").to(dtype).transpose(1, 2) for _ in range(2))
    v = torch.randn(B, T, H, dv, generator=g, device="cuda").to(dtype).transpose(1, 2)
    s0 = torch.randn(B, H, d, dv, generator=g, device="cuda")
    ld = torch.full((H,), -0.05, device="cuda")
    lens = torch.tensor([T - 7 * b if b % 3 == 0 else 0 for b in range(B)], dtype=torch.int32, device="cuda")
    empty = lens == 0
    first = None
    for _ in range(8):
        o, sT = fwpkm.linear_attention(q, k, v, ld, s0=s0, lens=lens, o=torch.zeros_like(v), final_state=True)
        dq, dk, dv_, ds0 = fwpkm.linear_attention_backward(q, k, v, ld, v, s0=s0, d_sT=s0, lens=lens)
        assert torch.equal(sT[empty], s0[empty])
        assert torch.equal(ds0[empty], s0[empty])
        if first is None:
            first = o, sT, ds0
        assert torch.equal(o, first[0]) and torch.equal(sT, first[1]) and torch.equal(ds0, first[2])
