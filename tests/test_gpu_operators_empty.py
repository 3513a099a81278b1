"""Calls of the operators around the memory without anything to work on: no rows, no entries in a bag, no
groups, no sequences, no heads."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_weight_memory_chunk_b200 import fwpkm  # noqa: E402

SIDE = [False, True]


def full(*shape, dtype=torch.float32):
    return torch.full(shape, 7, dtype=dtype, device="cuda")


@pytest.mark.parametrize("side", SIDE)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,n,R", [(0, 5, 2), (9, 5, 0), (0, 5, 0), (0, 0, 2), (9, 0, 2)])
def test_lookups(rows, n, R, dtype, side):
    stream = torch.cuda.Stream() if side else None
    table, idx, w = full(rows, 16, dtype=dtype), torch.zeros(n, R, dtype=torch.int64, device="cuda"), full(n, R)
    d_out, out, d_table = full(n, 16, dtype=dtype), full(n, 16, dtype=dtype), full(rows, 16)
    torch.cuda.synchronize()
    assert fwpkm.lookup_backward_workspace_size(table, idx, w) >= 0
    got = [fwpkm.lookup(table, idx, w=w, stream=stream), fwpkm.lookup(table, idx, w=w, out=out, stream=stream),
           *fwpkm.lookup_backward(table, idx, d_out, w=w, d_table=d_table, stream=stream)]
    torch.cuda.synchronize()
    assert [tuple(t.shape) for t in got] == [(n, 16), (n, 16), (rows, 16), (n, R)]
    assert not any(t.any() for t in got)
    kept = full(rows, 16)
    fwpkm.lookup_backward(table, idx, d_out, w=w, d_table=kept, accumulate=True)
    assert (kept == 7).all()
    if rows == 0:
        one = fwpkm.lookup(table, torch.zeros(n, dtype=torch.int32, device="cuda"))  # no weights
        assert one.shape == (n, 16) and not one.any()


def test_no_groups():
    x, idx = full(0, 6, 8), full(0, 6, 2, dtype=torch.int32)
    r = fwpkm.balance_loss(x, idx)
    assert r.loss.shape == (0,) and r.counts.shape == r.usage.shape == r.slope.shape == (0, 8)
    assert fwpkm.balance_loss_backward(x, r).shape == (0, 6, 8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,H", [(0, 3), (2, 0), (0, 0)])
def test_no_sequences_and_no_heads(B, H, dtype):
    q, v = full(B, H, 40, 16, dtype=dtype), full(B, H, 40, 24, dtype=dtype)
    ld, lens = full(H), torch.zeros(B, dtype=torch.int32, device="cuda")
    assert fwpkm.linear_attention_workspace_size(q, v) == fwpkm.linear_attention_workspace_size(q, v, True) == 0
    o, sT = fwpkm.linear_attention(q, q, v, ld, lens=lens, final_state=True)
    assert o.shape == v.shape and sT.shape == (B, H, 16, 24)
    grads = fwpkm.linear_attention_backward(q, q, v, ld, v, lens=lens)
    assert [g.shape for g in grads] == [q.shape, q.shape, v.shape, sT.shape]
    one = lambda t: t[:, :, :1]  # noqa: E731
    o, s = fwpkm.linear_attention_step(one(q), one(q), one(v), ld, sT)
    assert o.shape == one(v).shape and s is sT
