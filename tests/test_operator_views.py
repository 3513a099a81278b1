"""Tables and logits that are views: rows apart are taken at their stride, rows that share memory are
refused by the binding, on the host, before anything is read."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from sparse_weight_memory_chunk_b200 import build, fwpkm
    build.build()
    return fwpkm


def shared(rows, width):
    """Tables [rows][width] whose rows share memory."""
    yield torch.zeros(width).expand(rows, width)
    yield torch.zeros(1, width).expand(rows, width)
    yield torch.zeros(rows + width).unfold(0, width, 1)[:rows]
    yield torch.zeros(rows * width).as_strided((rows, width), (width - 1, 1))


@pytest.mark.parametrize("i", range(4))
def test_tables_whose_rows_share_memory_are_refused(lib, i):
    table = list(shared(5, 8))[i]
    idx, d_out = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 8)
    for call in (lambda: lib.lookup(table, idx), lambda: lib.lookup_backward(table, idx, d_out),
                 lambda: lib.lookup_backward_workspace_size(table, idx)):
        with pytest.raises(ValueError, match="table: the rows must not share memory"):
            call()
    with pytest.raises(ValueError, match="d_table: the rows must not share memory"):
        lib.lookup_backward(torch.zeros(5, 8), idx, d_out, d_table=table)


@pytest.mark.parametrize("i", range(4))
def test_logits_whose_rows_share_memory_are_refused(lib, i):
    x = list(shared(5, 8))[i].unsqueeze(0).expand(2, 5, 8)
    r = lib.BalanceLoss()
    r.kind, r.coef, r.slope = "load", 1.0, torch.zeros(2, 8)
    for call in (lambda: lib.balance_loss(x, kind="entropy"), lambda: lib.balance_loss_backward(x, r)):
        with pytest.raises(ValueError, match="x: the rows must not share memory"):
            call()


def test_views_with_rows_apart_are_taken_at_their_stride(lib):
    idx = torch.zeros(3, dtype=torch.int32)
    ld = lambda t: lib._lookup_config(t, idx, None, 1.0)[0].table_ld  # noqa: E731
    assert ld(torch.zeros(5, 20)[:, 4:12]) == 20 and ld(torch.zeros(10, 8)[::2]) == 16
    assert ld(torch.zeros(5, 8)) == 8 and ld(torch.zeros(8).expand(1, 8)) == 8 and ld(torch.zeros(5, 9)[:, 3:4]) == 9
    cfg = lambda x: lib._balance_config(x, None, None, "load", 1.0)  # noqa: E731
    c = cfg(torch.zeros(2, 6, 20)[:, ::2, 4:12])
    assert (c.ld, c.group_stride, c.tokens) == (40, 120, 3)
    c = cfg(torch.zeros(6, 8).expand(2, 6, 8))  # groups may share their logits
    assert (c.ld, c.group_stride) == (8, 0)
    assert cfg(torch.zeros(8).expand(4, 1, 8)).ld == 8
