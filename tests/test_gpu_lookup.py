"""Table lookups and their gradients on the GPU against oracle/operators.py (fp64).

Tolerances (u = 2^-24, half a step of fp32; h = 2^-8 half a step of bf16): a result that is a
sum of c products in fp32, in whatever order, is off by at most (c + 2) u times the sum of the
products' sizes (c roundings of running sums or fewer, one of a weight, one of the scale);
the scale itself is given in fp32.  A bf16 result adds half a step of its own size.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_weight_memory_chunk_b200 import fwpkm  # noqa: E402

from oracle import operators as op  # noqa: E402

U, HB = 2.0 ** -24, 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def within(got, ref, size, c, bf16, what):
    """|got - ref| <= (c + 2) u size (+ half a bf16 step of what was rounded)."""
    got = got.double().cpu().numpy()
    tol = (c + 2) * U * size + 1e-40
    if bf16:
        tol = tol + HB * (np.abs(ref) + tol)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst by {np.nanmax(np.abs(got - ref) / tol):.3g} of the bound"


def make(rows, width, n, R, dtype, seed, kind="spread", i64=False, weights=True):
    rng = np.random.default_rng(seed)
    dt = DT[dtype]
    table = torch.from_numpy(rng.normal(size=(rows, width)).astype(np.float32)).to(dt).cuda()
    d_out = torch.from_numpy(rng.normal(size=(n, width)).astype(np.float32)).to(dt).cuda()
    if kind == "one":        # every entry reads one row
        idx = np.full((n, R), rows // 2)
    elif kind == "two":      # two rows, so runs of both lengths
        idx = np.where(rng.random((n, R)) < 0.98, rows - 1, 0)
    else:                    # frequent and rare rows, entries outside the table on both sides
        idx = np.minimum((rows * rng.random((n, R)) ** 3).astype(np.int64), rows - 1)
        idx[rng.random((n, R)) < 0.1] = -1
        idx[rng.random((n, R)) < 0.05] = rows
        if n > 3:
            idx[3] = -5      # a token that reads nothing
    w = rng.normal(size=(n, R)).astype(np.float32) if weights else None
    it = torch.from_numpy(idx.astype(np.int64 if i64 else np.int32)).cuda()
    return table, it, None if w is None else torch.from_numpy(w).cuda(), d_out


def f64(t):
    return None if t is None else t.double().cpu().numpy()


# rows, width, n, R, dtype, int64 indices
SHAPES = [
    (1, 1, 1, 1, "f32", False), (5, 3, 7, 1, "bf16", True), (64, 64, 33, 1, "bf16", True),
    (100, 181, 50, 3, "f32", False), (7, 2048, 40, 1, "bf16", True), (1000, 2056, 21, 2, "bf16", False),
    (300, 1100, 17, 5, "f32", True), (4096, 256, 64, 32, "f32", False), (50, 24, 9, 128, "bf16", False),
    (5000, 40, 3000, 3, "f32", False), (70000, 16, 9000, 1, "bf16", True), (3, 8, 40000, 4, "bf16", False),
]


@pytest.mark.parametrize("rows,width,n,R,dtype,i64", SHAPES)
def test_lookup_and_gradients(rows, width, n, R, dtype, i64):
    table, idx, w, d_out = make(rows, width, n, R, dtype, rows + n, i64=i64)
    scale = 1.75
    bf = dtype == "bf16"
    T, I, W, D = f64(table), idx.cpu().numpy(), f64(w), f64(d_out)
    got = fwpkm.lookup(table, idx, w, scale)
    assert got.dtype == table.dtype and tuple(got.shape) == (n, width)
    within(got, op.lookup(T, I, W, scale), op.lookup(np.abs(T), I, np.abs(W), scale), R, bf, "out")
    ref, rw = op.lookup_backward(T, I, D, W, scale)
    size, sw = op.lookup_backward(np.abs(T), I, np.abs(D), np.abs(W), scale)
    per_row = np.bincount(I[(I >= 0) & (I < rows)].ravel(), minlength=rows)[:, None]
    dt, dw = fwpkm.lookup_backward(table, idx, d_out, w, scale, grad_dtype=torch.float32)
    within(dt, ref, size, per_row, False, "d_table")
    within(dw, rw, sw, width, False, "dw")
    # rows that nothing reads are exactly zero; a bf16 gradient is the fp32 one rounded once
    assert not dt[torch.from_numpy(per_row[:, 0] == 0).cuda()].any()
    db, none = fwpkm.lookup_backward(table, idx, d_out, w, scale, grad_dtype=torch.bfloat16, need_dw=False)
    assert none is None and torch.equal(db, dt.bfloat16())
    # added to what is there: touched rows only, one more rounding
    base = torch.randn(rows, width, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    acc = base.clone()
    back, _ = fwpkm.lookup_backward(table, idx, d_out, w, scale, d_table=acc, accumulate=True)
    assert back is acc
    b64 = f64(base)
    within(acc, b64 + ref, size + np.abs(b64 + ref), per_row + 1, False, "accumulated d_table")
    untouched = torch.from_numpy(per_row[:, 0] == 0).cuda()
    assert torch.equal(acc[untouched], base[untouched])


@pytest.mark.parametrize("kind", ["one", "two"])
@pytest.mark.parametrize("n,R,width", [(31, 1, 64), (33, 1, 72), (4096, 1, 256), (4097, 1, 40), (9000, 3, 64),
                                       (150000, 1, 8)])
def test_gradient_of_crowded_rows(kind, n, R, width):
    # long runs of one row cross tile and range borders: every partial sum has to arrive once
    table, idx, _, d_out = make(9, width, n, R, "f32", 5, kind, weights=False)
    w = torch.ones(n, R, device="cuda")
    dt, _ = fwpkm.lookup_backward(table, idx, d_out, w, 1.0)
    D, I = f64(d_out), idx.cpu().numpy()
    ref, size = np.zeros((9, width)), np.zeros((9, width))
    for r in range(R):
        np.add.at(ref, I[:, r], D)
        np.add.at(size, I[:, r], np.abs(D))
    # runs are summed 32 at a time, then the partial sums: fewer roundings than terms
    c = np.bincount(I.ravel(), minlength=9)[:, None]
    within(dt, ref, size, 34 + c / 32, False, "d_table")


def test_token_shapes_and_strides():
    # [B][T] tokens; a table that is a column slice of a wider one (rows off the 16-byte grid)
    big = torch.randn(50, 103, device="cuda")
    idx = torch.randint(50, (3, 5), device="cuda")
    for table in (big[:, :64], big[:, 1:65], big[:, 3:100]):
        out = fwpkm.lookup(table, idx, scale=2.0)
        assert torch.equal(out, 2.0 * table[idx])
        d = torch.randn_like(out)
        wide = torch.full((50, 128), 7.0, device="cuda")
        for view in (wide[:, :table.shape[1]], wide[:, 5:5 + table.shape[1]]):
            wide.fill_(7.0)
            fwpkm.lookup_backward(table, idx, d, d_table=view)
            ref = op.lookup_backward(f64(table), idx.cpu().numpy().reshape(-1, 1), f64(d).reshape(15, -1))[0]
            size = op.lookup_backward(f64(table), idx.cpu().numpy().reshape(-1, 1), np.abs(f64(d)).reshape(15, -1))[0]
            within(view, ref, size, 15, False, "strided d_table")
            assert int((wide == 7.0).sum()) >= 50 * (128 - table.shape[1])  # nothing outside the view
    assert tuple(fwpkm.lookup(big, torch.zeros((), dtype=torch.int64, device="cuda")).shape) == (103,)


def test_empty_calls():
    table = torch.randn(6, 16, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert tuple(fwpkm.lookup(table, none).shape) == (0, 16)
    d, _ = fwpkm.lookup_backward(table, none, torch.zeros(0, 16, device="cuda"),
                                 d_table=torch.full((6, 16), 3.0, device="cuda"))
    assert not d.any()                                     # a dense gradient of no token is zero
    d, _ = fwpkm.lookup_backward(table, none, torch.zeros(0, 16, device="cuda"),
                                 d_table=torch.full((6, 16), 3.0, device="cuda"), accumulate=True)
    assert bool((d == 3.0).all())
    # only entries outside the table
    idx = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    w = torch.ones(4, 2, device="cuda")
    assert not fwpkm.lookup(table, idx, w).any()
    d, dw = fwpkm.lookup_backward(table, idx, torch.ones(4, 16, device="cuda"), w)
    assert not d.any() and not dw.any()


def test_values_of_rows_that_are_not_read_do_not_matter():
    table = torch.full((8, 32), float("nan"), device="cuda")
    table[2] = 1.0
    idx = torch.tensor([[2, -1], [9, 2]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, float("nan")], [float("inf"), 2.0]], device="cuda")
    out = fwpkm.lookup(table, idx, w)
    assert torch.equal(out, torch.tensor([[0.5], [2.0]], device="cuda").expand(2, 32))
    d, dw = fwpkm.lookup_backward(table, idx, torch.ones(2, 32, device="cuda"), w)
    assert torch.equal(dw, torch.tensor([[32.0, 0.0], [0.0, 32.0]], device="cuda"))
    assert bool((d[2] == 2.5).all()) and not d[:2].any() and not d[3:].any()


def test_offsets_beyond_32_bits():
    rows, width = 2200003, 1024        # 2.25e9 elements
    table = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, rows - 1, rows - 2, 2097152, rows - 1], device="cuda")
    table[at] = torch.randn(5, width, device="cuda").bfloat16()
    out = fwpkm.lookup(table, at)
    assert torch.equal(out, table[at])
    d_out = torch.randn(5, width, device="cuda").bfloat16()
    g, _ = fwpkm.lookup_backward(table, at, d_out)   # dense, bf16: 4.5 GB
    assert torch.equal(g[rows - 2], d_out[2]) and torch.equal(g[2097152], d_out[3]) and torch.equal(g[0], d_out[0])
    assert torch.equal(g[rows - 1], (d_out[1].float() + d_out[4].float()).bfloat16())
    assert int((g != 0).any(1).sum()) == 4


def test_repeated_captured_and_on_another_stream():
    table, idx, w, d_out = make(3000, 128, 700, 8, "f32", 2)
    first = fwpkm.lookup_backward(table, idx, d_out, w)
    again = fwpkm.lookup_backward(table, idx, d_out, w)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])   # deterministic
    out = fwpkm.lookup(table, idx, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2 = fwpkm.lookup(table, idx, w, stream=side)
    side.synchronize()
    assert torch.equal(out, o2)
    # two graphs with one workspace, replayed one after the other on new inputs
    ws = torch.empty(fwpkm.lookup_backward_workspace_size(table, idx, w), dtype=torch.uint8, device="cuda")
    graphs, outs, d2 = [], [], d_out.clone()
    torch.cuda.synchronize()
    for scale in (1.0, -2.0):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fwpkm.lookup_backward(table, idx, d2, w, scale, workspace=ws))
        graphs.append(g)
    d2.copy_(d_out.flip(0))
    for g in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    want = fwpkm.lookup_backward(table, idx, d2, w)
    assert torch.equal(outs[0][0], want[0]) and torch.equal(outs[1][0], -2.0 * want[0])
