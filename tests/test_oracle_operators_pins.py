"""Pins of oracle/operators.py: hand-worked cases and central differences of the forward
functions.  A central difference with step h of a function with third derivative M has error
<= M h^2 / 6 + eps |f| / h; at h = 1e-5 and values and derivatives of order 1 to 10 that is
under 1e-8, so 1e-6 absolute is loose by two orders of magnitude."""
import numpy as np
import pytest

from oracle import operators as op

H = 1e-5
TOL = 1e-6


def diff(f, x):
    """Central differences of the scalar f() with respect to the array x (changed in place)."""
    g = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + H
        hi = f()
        x[i] = old - H
        lo = f()
        x[i] = old
        g[i] = (hi - lo) / (2 * H)
    return g


def test_lookup_by_hand():
    table = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    out = op.lookup(table, [[0, 2], [1, -1], [3, 3]], [[0.5, 2.0], [1.0, 9.0], [1.0, 1.0]], 10.0)
    assert np.array_equal(out, [[105.0, 130.0], [30.0, 40.0], [0.0, 0.0]])


def test_lookup_gradient_by_differences():
    rng = np.random.default_rng(0)
    table, w, c = rng.normal(size=(6, 3)), rng.normal(size=(5, 4)), rng.normal(size=(5, 3))
    idx = rng.integers(-1, 7, size=(5, 4))
    idx[0] = 2  # the same row in every place of a bag
    f = lambda: float((c * op.lookup(table, idx, w, 1.7)).sum())  # noqa: E731
    dt, dw = op.lookup_backward(table, idx, c, w, 1.7)
    assert np.abs(dt - diff(f, table)).max() < TOL
    assert np.abs(dw - diff(f, w)).max() < TOL


def test_balance_by_hand():
    # two experts, P = (3/4, 1/4) for both tokens, both select expert 0
    x = np.log([[3.0, 1.0], [3.0, 1.0]])
    loss, counts, usage, a, n = op.balance_loss(x, [[0], [0]], None, "load", 2.0)
    assert (counts == [2, 0]).all() and n == 2
    assert np.allclose(usage, [0.75, 0.25], atol=1e-15) and abs(loss - 2.0 * 2 * 0.75) < 1e-14
    # uniform logits: entropy log E, loss -log E, gradient 0
    loss, _, _, _, _ = op.balance_loss(np.zeros((3, 8)), None, None, "entropy")
    assert abs(loss + np.log(8)) < 1e-14
    assert np.abs(op.balance_backward(np.zeros((3, 8)), None, None, "entropy")).max() < 1e-15


def test_balance_masks_and_empty_rows():
    x = np.array([[1.0, -np.inf], [-np.inf, -np.inf], [np.nan, np.nan], [0.0, 0.0]])
    mask = [1, 1, 0, 1]
    loss, counts, usage, _, n = op.balance_loss(x, [[0], [1], [1], [7]], mask, "load")
    assert n == 2 and (counts == [1, 1]).all() and np.allclose(usage, [0.75, 0.25])
    dx = op.balance_backward(x, [[0], [1], [1], [7]], mask, "load")
    assert np.isfinite(dx).all() and (dx[1:3] == 0).all()
    loss, counts, usage, _, n = op.balance_loss(x, [[0], [1], [1], [0]], [0, 0, 0, 0], "entropy")
    assert n == 0 and loss == 0.0 and not usage.any() and not counts.any()


@pytest.mark.parametrize("kind", ["load", "entropy"])
def test_balance_gradient_by_differences(kind):
    rng = np.random.default_rng(1)
    x, idx, mask = rng.normal(size=(7, 5)), rng.integers(0, 5, size=(7, 2)), np.array([1, 1, 0, 1, 1, 0, 1])
    f = lambda: 0.7 * op.balance_loss(x, idx, mask, kind, 1.3)[0]  # noqa: E731
    dx = op.balance_backward(x, idx, mask, kind, 1.3, 0.7)
    assert np.abs(dx - diff(f, x)).max() < TOL


def test_linear_attention_by_hand():
    # one head, d = d_v = 1: S_t = S_{t-1}/2 + k v
    q, k, v = (np.array(x, float).reshape(1, 1, 3, 1) for x in ([1, 1, 2], [1, 2, 3], [4, 1, 1]))
    o, sT = op.linear_attention(q, k, v, [np.log(0.5)], 10.0, np.full((1, 1, 1, 1), 2.0))
    # S: 1 + 4 = 5; 2.5 + 2 = 4.5; 2.25 + 3 = 5.25
    assert np.allclose(o.ravel(), [50.0, 45.0, 105.0], atol=1e-12) and abs(sT.item() - 5.25) < 1e-13
    # no decay at all is the sum; -inf keeps the last token only
    o, _ = op.linear_attention(q, k, v, [0.0])
    assert np.allclose(o.ravel(), [4.0, 6.0, 18.0])
    o, _ = op.linear_attention(q, k, v, [-np.inf])
    assert np.allclose(o.ravel(), [4.0, 2.0, 6.0])


def test_linear_attention_gradient_by_differences():
    rng = np.random.default_rng(2)
    B, Hn, T, d, dv = 2, 2, 4, 3, 2
    q, k, v = rng.normal(size=(B, Hn, T, d)), rng.normal(size=(B, Hn, T, d)), rng.normal(size=(B, Hn, T, dv))
    s0, ld, lens = rng.normal(size=(B, Hn, d, dv)), np.array([-0.3, -1.2]), [3, 0]
    co, cs = rng.normal(size=(B, Hn, T, dv)), rng.normal(size=(B, Hn, d, dv))

    def f():
        o, sT = op.linear_attention(q, k, v, ld, 0.8, s0, lens)
        return float((co * o).sum() + (cs * sT).sum())

    grads = op.linear_attention_backward(q, k, v, ld, co, 0.8, s0, cs, lens)
    for g, x in zip(grads, (q, k, v, s0)):
        assert np.abs(g - diff(f, x)).max() < TOL
