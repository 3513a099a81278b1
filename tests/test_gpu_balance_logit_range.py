"""Balance loss of finite logits of any size: rows filled with a mask value, rows whose largest logit
is far from zero.  Only rows of -inf have no softmax.

Tolerances (u = 2^-24): y = x - max is off by u |y| (exact where the logits are equal), y log2 e by
1.3 u of itself (its own rounding and the constant's), 2^x by 4 u: exp(y) by (2.3 |y| + 4) u, the row's sum by as much
and E u, the quotient by 3 u: dP = (4.6 span + E + 11) u of P, span the largest |y| whose exp(y) is
not 0.  usage: dP + (T + 4) u; loss: sum over e of the weights |a_e| u_e ((|log u_e| + 1) u_e for the
entropy) times that; dx = g P (s - c), c = sum s P: g P (2 dP + (E + 8) u)(|s| + sum |s| P) and what
the slope's own error moves it; a bf16 dx half a step, 2^-8, more.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_weight_memory_chunk_b200 import fwpkm  # noqa: E402

from oracle import operators as op  # noqa: E402

U, HB = 2.0 ** -24, 2.0 ** -8


def logits(T, E, dtype, seed):
    """Ordinary rows, and rows of every size of logits that the type holds."""
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32)).to(dtype)
    lowest = torch.finfo(dtype).min
    levels = [lowest, -lowest, -1e30, 1e30, -1e10, 1e10, 3e9, -6e9, 1e4, -3e38]
    for i, level in enumerate(levels):
        x[3 * i] = level                                    # a row of one value
        x[3 * i + 1] = level                                # its maximum on some experts only
        x[3 * i + 1, rng.random(E) < 0.5] = lowest
    x[3 * len(levels)] = lowest
    x[3 * len(levels), E // 2] = 0.5
    return x


@pytest.mark.parametrize("kind", ["load", "entropy"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [3, 8, 60, 64, 333, 1024, 1028, 2049, 4096])
def test_rows_of_finite_logits_count(E, dtype, kind):
    T, coef = 80, 0.5
    x = logits(T, E, dtype, E)
    idx = torch.randint(E, (T, 2), generator=torch.Generator().manual_seed(E), dtype=torch.int32)
    r = fwpkm.balance_loss(x[None].cuda(), idx[None].cuda(), kind=kind, coef=coef)
    dx = fwpkm.balance_loss_backward(x[None].cuda(), r)[0].double().cpu().numpy()
    X = x.double().numpy()
    loss, counts, usage, a, n = op.balance_loss(X, idx.numpy(), None, kind, coef)
    assert n == T and (r.counts[0].cpu().numpy() == counts).all()
    P = op.softmax_rows(X)
    y = X - X.max(1, keepdims=True)
    dP = (4.6 * np.abs(y[y > -104.0]).max() + E + 11) * U
    du = dP + (T + 4) * U
    assert (np.abs(r.usage[0].double().cpu().numpy() - usage) <= du * usage + 1e-40).all()
    w = np.abs(a) * usage if kind == "load" else (np.abs(a - 1.0) + 1.0) * usage
    assert abs(float(r.loss[0]) - loss) <= coef * w.sum() * (du + 4 * U) + U * abs(loss) + 1e-40
    ref = op.balance_backward(X, idx.numpy(), None, kind, coef)
    s = coef / n * (a - (1.0 if kind == "load" else 1.0 - np.log(E)))
    ds = 2 * U * np.abs(s) + (0.0 if kind == "load" else coef / n * (du + 4 * U))
    c = (P * np.abs(s)).sum(1, keepdims=True)
    tol = P * ((2 * dP + (E + 8) * U) * (np.abs(s)[None] + c) + ds + (P * ds).sum(1, keepdims=True))
    tol = tol + 4 * U * np.abs(ref) + 1e-38
    if dtype == torch.bfloat16:
        tol = tol + HB * (np.abs(ref) + tol)
    off = np.abs(dx - ref)
    assert (off <= tol).all(), f"rows {np.nonzero((off > tol).any(1))[0]}, worst {np.max(off / tol):.3g} of the bound"
