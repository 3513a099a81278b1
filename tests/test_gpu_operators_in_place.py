"""Calls of the operators around the memory whose output is an input's own memory, where the header
allows it, and two calls at once on two streams."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_weight_memory_chunk_b200 import fwpkm  # noqa: E402


@pytest.mark.parametrize("n,R", [(300, 4), (30000, 4)])  # pairs sorted in one launch, and by passes
def test_a_step_of_gradient_descent_in_the_table_itself(n, R):
    g = torch.Generator("cuda").manual_seed(n)
    table = torch.randn(500, 64, generator=g, device="cuda")
    idx = torch.randint(-1, 500, (n, R), generator=g, device="cuda", dtype=torch.int32)
    w = torch.softmax(torch.randn(n, R, generator=g, device="cuda"), -1)
    d_out = torch.randn(n, 64, generator=g, device="cuda")
    want = table.clone()
    _, dw = fwpkm.lookup_backward(table, idx, d_out, w=w, scale=-0.5, d_table=want, accumulate=True)
    own = table.clone()
    got, dw2 = fwpkm.lookup_backward(own, idx, d_out, w=w, scale=-0.5, d_table=own, accumulate=True)
    assert got is own and torch.equal(own, want) and torch.equal(dw2, dw) and not torch.equal(own, table)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [5, 8, 64, 256, 1000, 1024, 2048, 3001])
def test_the_gradient_of_logits_in_their_own_memory(E, dtype):
    g = torch.Generator("cuda").manual_seed(E)
    x = torch.randn(3, 1000, E, generator=g, device="cuda").to(dtype)
    mask = torch.rand(3, 1000, generator=g, device="cuda") < 0.8
    r = fwpkm.balance_loss(x, mask=mask, kind="entropy")
    want = fwpkm.balance_loss_backward(x, r, mask=mask)
    got = fwpkm.balance_loss_backward(x, r, mask=mask, dx=x)
    assert got is x and torch.equal(got, want)


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, give what they give alone."""
    g = torch.Generator("cuda").manual_seed(1)
    q, k, v = (torch.randn(2, 3000, 4, 128, generator=g, device="cuda").bfloat16().transpose(1, 2) for _ in range(3))
    ld = torch.full((4,), -0.02, device="cuda")
    table = torch.randn(4000, 128, generator=g, device="cuda")
    idx = torch.randint(4000, (50000,), generator=g, device="cuda")
    d_out = torch.randn(50000, 128, generator=g, device="cuda")
    x = torch.randn(4, 4096, 256, generator=g, device="cuda")

    def calls(stream):
        return (*fwpkm.linear_attention(q, k, v, ld, final_state=True, stream=stream),
                *fwpkm.linear_attention_backward(q, k, v, ld, v, stream=stream),
                fwpkm.lookup_backward(table, idx, d_out, stream=stream)[0],
                fwpkm.balance_loss(x, kind="entropy", stream=stream).slope)

    want = calls(None)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        got = [calls(s) for s in (a, b, a, b)]
        a.synchronize()
        b.synchronize()
        for r in got:
            assert all(torch.equal(y, z) for y, z in zip(r, want))
    fwpkm.linear_attention_sync(stream=a)
