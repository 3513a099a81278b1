"""The balance loss, its counts and its gradient on the GPU against oracle/operators.py (fp64).

Tolerances (u = 2^-24): with x - max = y, exp(y) in fp32 is off by (|y| + 2) u of itself (one
rounding of y, at most 2 u of expf), the row's sum by E u, and the division by 2 u, so P is off by dP = (ymax + E + 6) u of
itself.  usage, a sum of up to T terms of one column, by (dP + T u) of itself.  With the
logarithm's own error, loss is off by at most sum_e w_e (that), w_e = |a_e| u_e for the load and
(|log u_e| + 1) u_e for the entropy, and one rounding.  dx = g P (s - c), c = sum s P: off by
g P (2 dP + (E + 8) u)(|s| + sum |s| P) plus what the slope's own error ds moves it,
g P (ds + sum ds P); a bf16 dx by half a step more.  Counts are exact.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_weight_memory_chunk_b200 import fwpkm  # noqa: E402

from oracle import operators as op  # noqa: E402

U, HB = 2.0 ** -24, 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(G, T, E, k, dtype, masked, seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.normal(size=(G, T, E)) + rng.normal(size=(G, 1, E))).astype(np.float32)).to(DT[dtype])
    idx = torch.from_numpy(rng.integers(-1, E + 1, size=(G, T, k)).astype(np.int32))
    mask = None
    if masked:
        mask = torch.from_numpy(rng.random((G, T)) < 0.7)
        x[~mask] = float("nan")
        idx[~mask] = 0
        mask = mask.cuda()
    return x.cuda(), idx.cuda(), mask


def check(x, idx, mask, kind, coef, r, dx, gl):
    G, T, E = x.shape
    X = x.double().cpu().numpy()
    I = None if idx is None else idx.cpu().numpy()
    M = np.ones((G, T), bool) if mask is None else mask.cpu().numpy().astype(bool)
    for g in range(G):
        loss, counts, usage, a, n = op.balance_loss(X[g], None if I is None else I[g], M[g], kind, coef)
        if I is not None:
            assert (r.counts[g].cpu().numpy() == counts).all(), f"group {g}: counts"
        P = np.zeros((T, E))
        P[M[g]] = op.softmax_rows(X[g][M[g]])
        live = P.sum(1) > 0
        span = 0.0
        if live.any():
            fin = np.where(np.isfinite(X[g][live]), X[g][live], np.nan)
            span = float(np.nanmax(np.nanmax(fin, 1) - np.nanmin(fin, 1)))
        dP = (span + E + 6) * U
        du = (dP + (T + 4) * U)
        got_u = r.usage[g].double().cpu().numpy()
        assert (np.abs(got_u - usage) <= du * usage + 1e-40).all(), f"group {g}: usage"
        lw = np.abs(a) * usage if kind == "load" else (np.abs(a - 1.0) + 1.0) * usage
        tol = abs(coef) * (lw.sum() * (du + 4 * U)) + U * abs(loss) + 1e-40
        assert abs(float(r.loss[g]) - loss) <= tol, f"group {g}: loss {float(r.loss[g])} {loss} {tol}"
        if n == 0:
            assert not dx[g].any()
            continue
        ref = op.balance_backward(X[g], None if I is None else I[g], M[g], kind, coef, gl[g])
        # the slope as the header gives it: less the constant of a balanced router
        s = coef / n * np.where(usage > 0, a - (1.0 if kind == "load" else 1.0 - np.log(E)), 0.0)
        ds = 2 * U * np.abs(s) + (0.0 if kind == "load" else abs(coef) / n * (du + 4 * U))
        c = (P * np.abs(s)).sum(1, keepdims=True)
        tol = abs(gl[g]) * P * ((2 * dP + (E + 8) * U) * (np.abs(s)[None] + c) + ds + (P * ds).sum(1, keepdims=True))
        tol = tol + 4 * U * np.abs(ref) + 1e-38
        if x.dtype == torch.bfloat16:
            tol = tol + HB * (np.abs(ref) + tol)
        err = np.abs(dx[g].double().cpu().numpy() - ref)
        assert (err <= tol).all(), f"group {g}: dx off by {np.max(err / tol):.3g} of its bound"


SHAPES = [
    (1, 1, 1, 1, "f32", False), (2, 1, 3, 1, "bf16", False), (1, 17, 8, 2, "bf16", True), (3, 65, 16, 1, "f32", True),
    (1, 500, 64, 8, "bf16", True), (2, 300, 60, 4, "bf16", False), (2, 257, 127, 3, "f32", True),
    (1, 400, 256, 8, "f32", False), (2, 100, 333, 2, "bf16", True), (1, 130, 512, 8, "bf16", False),
    (1, 200, 1000, 32, "f32", True), (2, 129, 1024, 4, "bf16", True), (1, 67, 1028, 5, "f32", False),
    (1, 70, 2049, 3, "f32", True), (1, 40, 4096, 8, "bf16", False), (1, 33, 4096, 2, "f32", True),
    (1, 20000, 5, 1, "f32", True),
]


@pytest.mark.parametrize("kind", ["load", "entropy"])
@pytest.mark.parametrize("G,T,E,k,dtype,masked", SHAPES)
def test_balance_matches_oracle(G, T, E, k, dtype, masked, kind):
    x, idx, mask = make(G, T, E, k, dtype, masked, T + E)
    gl = np.random.default_rng(0).normal(size=G).astype(np.float32)
    r = fwpkm.balance_loss(x, idx, mask, kind, 0.37)
    dx = fwpkm.balance_loss_backward(x, r, mask, torch.from_numpy(gl).cuda())
    assert dx.dtype == x.dtype
    check(x, idx, mask, kind, np.float64(np.float32(0.37)), r, dx, gl.astype(np.float64))


def test_masks_that_leave_nothing_and_infinite_logits():
    x = torch.randn(3, 9, 20, device="cuda")
    idx = torch.randint(20, (3, 9, 2), dtype=torch.int32, device="cuda")
    mask = torch.ones(3, 9, dtype=torch.uint8, device="cuda")
    mask[1] = 0                                 # a group without a token
    x[1] = float("inf")
    x[2, :, 7:] = -float("inf")                 # experts that are switched off
    x[2, 4] = -float("inf")                     # a row of nothing else
    x[0, 3, 5] = torch.finfo(torch.float32).min  # a mask of the type's lowest value
    for kind in ("load", "entropy"):
        r = fwpkm.balance_loss(x, idx, mask, kind)
        dx = fwpkm.balance_loss_backward(x, r, mask)
        assert float(r.loss[1]) == 0.0 and not r.usage[1].any() and not dx[1].any() and not r.counts[1].any()
        assert not dx[2, :, 7:].any() and not dx[2, 4].any() and dx[0, 3, 5] == 0
        assert torch.isfinite(r.loss).all() and torch.isfinite(dx).all() and torch.isfinite(r.slope).all()
        # the oracle takes -inf too; the lowest value makes the span of that row infinite, so
        # it is compared without group 0
        check(x[1:], idx[1:], mask[1:], kind, 1.0, _part(r, 1), dx[1:], np.ones(2))
    # NaN in a row that counts is seen
    x[0, 0, 0] = float("nan")
    r = fwpkm.balance_loss(x, idx, mask)
    assert torch.isnan(r.loss[0]) and torch.isfinite(r.loss[1:]).all()


def _part(r, g):
    class P:
        pass
    p = P()
    p.loss, p.counts, p.usage, p.slope = r.loss[g:], r.counts[g:], r.usage[g:], r.slope[g:]
    return p


def test_strided_logits_entropy_without_selections_and_no_tokens():
    big = torch.randn(4, 50, 70, device="cuda")
    for x in (big[:, :, :64], big[:, :, 1:65], big[::2, ::3, :40], big[1:2, :, :9]):
        r = fwpkm.balance_loss(x, kind="entropy")
        dx = fwpkm.balance_loss_backward(x, r)
        assert r.counts is None
        check(x, None, None, "entropy", 1.0, r, dx, np.ones(x.shape[0]))
    x = torch.zeros(2, 0, 8, device="cuda")
    r = fwpkm.balance_loss(x, torch.zeros(2, 0, 2, dtype=torch.int32, device="cuda"))
    assert not r.loss.any() and not r.counts.any() and not r.usage.any()
    assert tuple(fwpkm.balance_loss_backward(x, r).shape) == (2, 0, 8)


def test_a_balanced_router_has_no_gradient():
    # equal logits and equal counts: loss = coef, gradient exactly 0 (the slope is)
    x = torch.zeros(1, 64, 16, device="cuda")
    idx = (torch.arange(64, device="cuda", dtype=torch.int32) % 16).view(1, 64, 1)
    r = fwpkm.balance_loss(x, idx, coef=0.25)
    assert abs(float(r.loss) - 0.25) <= 0.25 * 80 * U and not r.slope.any()
    assert not fwpkm.balance_loss_backward(x, r).any()


def test_repeated_captured_and_on_another_stream():
    x, idx, mask = make(2, 3000, 96, 4, "bf16", True, 9)
    a, b = fwpkm.balance_loss(x, idx, mask), fwpkm.balance_loss(x, idx, mask)
    assert torch.equal(a.loss, b.loss) and torch.equal(a.slope, b.slope)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = fwpkm.balance_loss(x, idx, mask, stream=side)
    dc = fwpkm.balance_loss_backward(x, c, mask, stream=side)
    side.synchronize()
    assert torch.equal(a.loss, c.loss) and torch.equal(fwpkm.balance_loss_backward(x, a, mask), dc)
    x2 = x.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        r = fwpkm.balance_loss(x2, idx, mask)
        d = fwpkm.balance_loss_backward(x2, r, mask)
    x2.copy_(2 * x)
    g.replay()
    torch.cuda.synchronize()
    want = fwpkm.balance_loss(2 * x, idx, mask)
    assert torch.equal(r.loss, want.loss) and torch.equal(d, fwpkm.balance_loss_backward(2 * x, want, mask))
