"""Outputs that a call of linear attention makes itself hold zeros behind a sequence's end, so that what
is formed from whole tensors (a projection's weight gradient) sees nothing there."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_weight_memory_chunk_b200 import fwpkm  # noqa: E402


def poison(*shapes, dtype):
    """Memory of these sizes, full of NaN, goes back to the allocator that new tensors come from."""
    t = [torch.full(s, float("nan"), dtype=dtype, device="cuda") for s in shapes]
    torch.cuda.synchronize()
    del t


@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d,dv", [(3, 16, 16), (200, 64, 32), (400, 72, 100)])
def test_new_outputs_are_zero_behind_the_ends(T, d, dv, dtype, stream):
    B, H = 3, 2
    g = torch.Generator("cuda").manual_seed(T)
    q, k = (torch.randn(B, T, H, d, generator=g, device="cuda").to(dtype).transpose(1, 2) for _ in range(2))
    v = torch.randn(B, T, H, dv, generator=g, device="cuda").to(dtype).transpose(1, 2)
    ld, s0 = torch.full((H,), -0.1, device="cuda"), torch.randn(B, H, d, dv, generator=g, device="cuda")
    lens = torch.tensor([T, T // 2, 0], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    with torch.cuda.stream(side if stream else torch.cuda.current_stream()):
        shapes = [(B, T, H, d)] * 3 + [(B, T, H, dv)] * 3
        poison(*shapes, dtype=dtype)
    o, _ = fwpkm.linear_attention(q, k, v, ld, lens=lens, stream=side)
    dq, dk, dv_, _ = fwpkm.linear_attention_backward(q, k, v, ld, v, lens=lens, stream=side)
    outs = [o, dq, dk, dv_]
    if T <= 16:
        outs.append(fwpkm.linear_attention_step(q, k, v, ld, s0, lens=lens, stream=side)[0])
    torch.cuda.synchronize()
    for x in outs:
        assert torch.isfinite(x.float()).all() and x[0].float().abs().sum() > 0
        for b, n in enumerate(lens.tolist()):
            assert not x[b, :, n:].any()
