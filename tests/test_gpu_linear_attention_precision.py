"""Linear attention of bf16 prompts is off by its outputs' own rounding and fp32 arithmetic, no more.

Tolerances (u = 2^-24, h = 2^-8, A the same sums over absolute values).  fp32 arithmetic is off by
c u A, c = T + d + d_v + 32 (the roundings that a term passes through).  On the tensor cores a
weighted score, or the state before a chunk, enters o as two bf16 pieces: the high one leaves less
than 2^-7 of it, the low one is off by half a step of that, 2^-16; the keys in that state likewise.
2^-16 A + 2^-16 A is 2^9 u A.  The bf16 result adds h of itself.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_weight_memory_chunk_b200 import fwpkm  # noqa: E402

from oracle import operators as op  # noqa: E402

U, HB = 2.0 ** -24, 2.0 ** -8


def f64(t):
    return t.double().cpu().numpy()


def rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def close(got, ref, size, c, what):
    tol = c * U * size + 1e-40
    tol = tol + HB * (np.abs(ref) + tol)
    off = np.abs(f64(got) - ref)
    assert (off <= tol).all(), f"{what}: {int((off > tol).sum())} off, worst {np.max(off / tol):.3g} of the bound"


def check(B, H, T, d, dv, ld, s_qk=1.0, s_do=1.0):
    g = torch.Generator("cuda").manual_seed(B * H + T)
    q, k = ((s_qk * rand(g, B, T, H, d)).bfloat16().transpose(1, 2) for _ in range(2))
    v = rand(g, B, T, H, dv).bfloat16().transpose(1, 2)
    do = (s_do * rand(g, B, T, H, dv)).bfloat16().transpose(1, 2)
    s0, dsT = s_qk * rand(g, B, H, d, dv), s_qk * s_do * rand(g, B, H, d, dv)
    decay = torch.tensor([ld[h % len(ld)] for h in range(H)], device="cuda")
    c = T + d + dv + 32 + 2.0 ** 9
    o, _ = fwpkm.linear_attention(q, k, v, decay, 0.5, s0=s0)
    grads = fwpkm.linear_attention_backward(q, k, v, decay, do, 0.5, s0=s0, d_sT=dsT)
    fwpkm.linear_attention_sync()
    x = [f64(t) for t in (q, k, v)]
    a = [np.abs(t) for t in x]
    dn, S, dS, D = f64(decay), f64(s0), f64(dsT), f64(do)
    close(o, op.linear_attention(*x, dn, 0.5, S)[0], op.linear_attention(*a, dn, 0.5, np.abs(S))[0], c, "o")
    ref = op.linear_attention_backward(*x, dn, D, 0.5, S, dS)
    size = op.linear_attention_backward(*a, dn, np.abs(D), 0.5, np.abs(S), np.abs(dS))
    for got, r, s, n in zip(grads[:3], ref, size, ("dq", "dk", "dv")):
        close(got, r, s, c, n)


@pytest.mark.parametrize("ld", [[-0.002, -0.1, -0.4, -3.0], [0.0, -0.01]])
@pytest.mark.parametrize("B,H,T,d,dv", [(1, 4, 300, 128, 128), (1, 2, 1000, 128, 64), (20, 4, 150, 64, 128),
                                        (2, 3, 257, 72, 104), (1, 1, 40, 64, 64)])
def test_scores_and_states_keep_more_than_one_bf16_rounding(B, H, T, d, dv, ld):
    check(B, H, T, d, dv, ld)


@pytest.mark.parametrize("s_qk,s_do", [(1e-8, 1.0), (1e-5, 1e-10), (1e6, 1e8)])
@pytest.mark.parametrize("B,H,T,d,dv", [(1, 2, 300, 128, 128), (20, 4, 150, 64, 64), (1, 1, 600, 64, 128)])
def test_inputs_of_any_size_on_heads_that_decay_quickly(B, H, T, d, dv, s_qk, s_do):
    """Weights of up to |log a| 127 on one side of a chunk must not take small scores out of range."""
    check(B, H, T, d, dv, [-0.46, -0.3], s_qk, s_do)


@pytest.mark.parametrize("B,H,T", [(25, 3, 16384), (1, 8, 16384)])
def test_a_state_decays_over_many_chunks(B, H, T):
    """Keys in the first chunk only, so that the state after T tokens is a^(T - 128) times that after
    128.  Each chunk rounds every element once, by at most u of it and in either direction: over the
    4096 elements of a head the mean of T / 128 roundings has a standard deviation of at most
    u / sqrt(3) sqrt(T / 128 / 4096) = 0.1 u; the bound is 2 u.  (a^128 as one fp32 number is off by
    its rounding and expf's in the same direction every time: up to 124 u here.)"""
    g = torch.Generator("cuda").manual_seed(T)
    k = torch.zeros(B, T, H, 64, device="cuda", dtype=torch.bfloat16)
    k[:, :128] = rand(g, B, 128, H, 64).bfloat16()
    k, v = k.transpose(1, 2), rand(g, B, T, H, 64).bfloat16().transpose(1, 2)
    ld = -torch.exp(torch.linspace(-11.0, -7.0, H, device="cuda"))
    first = fwpkm.linear_attention(*(x[:, :, :128] for x in (k, k, v)), ld, final_state=True)[1]
    got = f64(fwpkm.linear_attention(k, k, v, ld, final_state=True)[1])
    fwpkm.linear_attention_sync()
    want = f64(first) * np.exp(f64(ld) * (T - 128))[None, :, None, None]
    bias = ((got - want) * want).sum((2, 3)) / (want * want).sum((2, 3))
    assert (np.abs(bias) <= 2 * U).all(), f"worst {np.abs(bias).max() / U:.3g} u"
