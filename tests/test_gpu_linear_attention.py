"""Linear attention with a decay per head on the GPU against oracle/operators.py (fp64): prompts,
their gradients, and token by token.

Tolerances (u = 2^-24, h = 2^-8).  Every result is a sum of products a^e x y z over the tokens.
With A the same sum over absolute values (the oracle on |q|, |k|, |v|, |s0|), fp32 arithmetic is
off by at most c u A, c the roundings a term passes through: one per token of running sums and
decays, d or d_v of the product with the state and a few of the weights, c = T + d + d_v + 32.
On the tensor cores every term of o passes through one more rounding to bf16 (the weighted score
q_t k_s inside a chunk of 128 tokens, the state before it): half a step, h A; the keys in the
state enter as two bf16 pieces, which leave out at most 2^-17 of a key.  2^-8 A + 2^-16 A is
(2^16 + 2^8) u A.  States that leave in fp32 take three pieces, exact to 2^-25.  The decay
itself is exp of an fp32 number taken to the e-th power: e |log a| u of a weight a^e, which is
below u / e_(natural) <= u.  A bf16 result adds h of itself.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_weight_memory_chunk_b200 import fwpkm  # noqa: E402

from oracle import operators as op  # noqa: E402

U, HB = 2.0 ** -24, 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def tensors(B, H, T, d, dv, dtype, seed, order="bthd"):
    """q, k, v, d_o seen as [B][H][T][.], s0 and d_sT."""
    g = torch.Generator("cuda").manual_seed(seed)
    out = []
    for w in (d, d, dv, dv):
        if order == "bthd":
            x = torch.randn(B, T, H, w, generator=g, device="cuda").to(DT[dtype]).transpose(1, 2)
        elif order == "bhtd":
            x = torch.randn(B, H, T, w, generator=g, device="cuda").to(DT[dtype])
        else:  # rows off the 16-byte grid
            x = torch.randn(B, T, H, w + 3, generator=g, device="cuda").to(DT[dtype])[..., 1:w + 1].transpose(1, 2)
        out.append(x)
    s0, dsT = (torch.randn(B, H, d, dv, generator=g, device="cuda") for _ in range(2))
    return (*out, s0, dsT)


def close(got, ref, size, c, bf16, what):
    got = f64(got)
    tol = c * U * size + 1e-40
    if bf16:
        tol = tol + HB * (np.abs(ref) + tol)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {np.nanmax(np.abs(got - ref) / tol):.3g} of the bound"


def check_forward(q, k, v, ld, scale, s0, lens, o, sT, what, before=None):
    T, d, dv, bf = q.shape[2], q.shape[3], v.shape[3], q.dtype == torch.bfloat16
    ln = None if lens is None else lens.tolist()
    c = T + d + dv + 32 + (2.0 ** 16 + 2.0 ** 8 if bf else 0.0)
    ro, rs = op.linear_attention(f64(q), f64(k), f64(v), f64(ld), scale, f64(s0), ln)
    ao, as_ = op.linear_attention(*(np.abs(f64(x)) for x in (q, k, v)), f64(ld), abs(scale),
                                  None if s0 is None else np.abs(f64(s0)), ln)
    if lens is not None:  # rows behind the end keep what was there
        for b, n in enumerate(ln):
            n = min(max(n, 0), T)
            assert torch.equal(o[b, :, n:], before[b, :, n:]), f"{what}: rows behind the end were written"
            ro[b, :, n:], ao[b, :, n:] = f64(o[b, :, n:]), 0.0
    close(o, ro, ao, c, bf, f"{what}: o")
    if sT is not None:
        # the state's keys enter as three pieces, so fp32's bound holds
        close(sT, rs, as_, T + d + dv + 32, False, f"{what}: sT")


def check_backward(q, k, v, ld, do, scale, s0, dsT, lens, grads, ds0, what):
    T, d, dv, bf = q.shape[2], q.shape[3], v.shape[3], q.dtype == torch.bfloat16
    ln = None if lens is None else lens.tolist()
    c = T + d + dv + 32 + (2.0 ** 16 + 2.0 ** 8 if bf else 0.0)
    a = lambda x: None if x is None else np.abs(f64(x))  # noqa: E731
    ref = op.linear_attention_backward(f64(q), f64(k), f64(v), f64(ld), f64(do), scale, f64(s0), f64(dsT), ln)
    size = op.linear_attention_backward(a(q), a(k), a(v), f64(ld), a(do), abs(scale), a(s0), a(dsT), ln)
    for g, r, s, n in zip(grads, ref, size, ("dq", "dk", "dv")):
        close(g, r, s, c, bf, f"{what}: {n}")
    if ds0 is not None:
        close(ds0, ref[3], size[3], T + d + dv + 32, False, f"{what}: ds0")


def decays(H, kind="mixed"):
    x = {"mixed": [-0.002, -0.1, -0.5, -3.0], "none": [0.0], "off": [-INF], "strong": [-30.0, -2.49, -2.51],
         "slow": [-0.0005]}[kind]
    return torch.tensor([x[h % len(x)] for h in range(H)], device="cuda")


# B, H, T, d, dv, dtype, memory order, decays
CASES = [
    (1, 1, 1, 1, 1, "f32", "bthd", "mixed"), (2, 3, 2, 5, 7, "bf16", "off", "mixed"),
    (1, 2, 15, 16, 16, "f32", "bhtd", "strong"), (2, 2, 16, 64, 64, "bf16", "bthd", "mixed"),
    (1, 4, 17, 72, 100, "f32", "bthd", "mixed"), (3, 1, 33, 40, 36, "bf16", "bthd", "off"),
    (1, 4, 127, 128, 128, "bf16", "bthd", "mixed"), (2, 4, 128, 128, 128, "bf16", "bhtd", "mixed"),
    (1, 4, 129, 128, 64, "bf16", "bthd", "strong"), (1, 2, 255, 64, 128, "bf16", "bthd", "none"),
    (2, 4, 300, 64, 64, "bf16", "bthd", "mixed"), (1, 3, 385, 24, 120, "bf16", "bthd", "mixed"),
    (1, 2, 257, 256, 256, "f32", "bthd", "mixed"), (1, 2, 300, 200, 130, "bf16", "off", "mixed"),
    (1, 2, 1000, 128, 128, "bf16", "bthd", "mixed"), (1, 1, 1100, 64, 32, "f32", "bhtd", "slow"),
    (1, 1, 1300, 16, 8, "bf16", "bthd", "slow"), (40, 4, 200, 32, 32, "bf16", "bthd", "off"),
    (1, 3, 700, 96, 80, "bf16", "off", "mixed"), (1, 4, 513, 8, 128, "bf16", "bthd", "strong"),
]


@pytest.mark.parametrize("B,H,T,d,dv,dtype,order,dec", CASES)
def test_prompt_and_gradients(B, H, T, d, dv, dtype, order, dec):
    q, k, v, do, s0, dsT = tensors(B, H, T, d, dv, dtype, T + d, order)
    ld, scale = decays(H, dec), 0.25
    o, sT = fwpkm.linear_attention(q, k, v, ld, scale, s0=s0, final_state=True)
    check_forward(q, k, v, ld, scale, s0, None, o, sT, "forward")
    o2, none = fwpkm.linear_attention(q, k, v, ld, scale)          # no states
    assert none is None
    check_forward(q, k, v, ld, scale, None, None, o2, None, "no states")
    dq, dk, dv_, ds0 = fwpkm.linear_attention_backward(q, k, v, ld, do, scale, s0=s0, d_sT=dsT)
    check_backward(q, k, v, ld, do, scale, s0, dsT, None, (dq, dk, dv_), ds0, "backward")
    dq, dk, dv_, none = fwpkm.linear_attention_backward(q, k, v, ld, do, scale, state_grad=False)
    assert none is None
    check_backward(q, k, v, ld, do, scale, None, None, None, (dq, dk, dv_), None, "backward, no states")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,lens", [(1, [1, 0]), (130, [130, 0, 1, 128, 129, 64, 999, -3]), (700, [700, 257, 256, 0]),
                                    (600, [0])])
def test_sequences_of_different_lengths(T, lens, dtype):
    B, H, d, dv = len(lens), 2, 64, 48
    q, k, v, do, s0, dsT = tensors(B, H, T, d, dv, dtype, T)
    for b, n in enumerate(lens):
        n = min(max(n, 0), T)
        for x in (q, k, v, do):
            x[b, :, n:] = float("nan")       # what lies behind the end is nobody's business
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ld = decays(H)
    mark = lambda w: torch.full((B, T, H, w), 5.0, dtype=DT[dtype], device="cuda").transpose(1, 2)  # noqa: E731
    o = mark(dv)
    _, sT = fwpkm.linear_attention(q, k, v, ld, 0.5, s0=s0, lens=ln, o=o, final_state=True)
    zq, zk, zv, zdo = q.clone(), k.clone(), v.clone(), do.clone()
    for b, n in enumerate(lens):
        for x in (zq, zk, zv, zdo):
            x[b, :, min(max(n, 0), T):] = 0
    check_forward(zq, zk, zv, ld, 0.5, s0, ln, o, sT, "ragged", before=mark(dv))
    grads = (mark(d), mark(d), mark(dv))
    *_, ds0 = fwpkm.linear_attention_backward(q, k, v, ld, do, 0.5, s0=s0, d_sT=dsT, lens=ln, grads=grads)
    for g in grads:
        for b, n in enumerate(lens):
            n = min(max(n, 0), T)
            assert bool((g[b, :, n:] == 5.0).all()), "gradient rows behind the end were written"
            g[b, :, n:] = 0
    check_backward(zq, zk, zv, ld, zdo, 0.5, s0, dsT, ln, grads, ds0, "ragged backward")
    if 0 in lens:
        b = lens.index(0)
        assert torch.equal(sT[b], s0[b]) and torch.equal(ds0[b], dsT[b])


@pytest.mark.parametrize("B,H,d,dv,dtype,n", [(1, 8, 64, 64, "bf16", 1), (3, 2, 128, 128, "f32", 1), (2, 1, 256, 256, "bf16", 2),
                                              (1, 2, 5, 3, "f32", 4), (70, 4, 72, 100, "bf16", 1), (2, 3, 130, 17, "f32", 16),
                                              (1, 1, 16, 200, "bf16", 5), (200, 2, 64, 64, "f32", 3)])
def test_tokens_against_oracle_in_place_and_not(B, H, d, dv, dtype, n):
    q, k, v, _, s0, _ = tensors(B, H, n, d, dv, dtype, d + dv, "off" if d == 5 else "bthd")
    ld = decays(H, "strong" if B == 3 else "mixed")
    o, s1 = fwpkm.linear_attention_step(q, k, v, ld, s0, 0.5, in_place=False)
    check_forward(q, k, v, ld, 0.5, s0, None, o, s1, "tokens")
    live, keep = s0.clone(), s0.clone()
    o2, same = fwpkm.linear_attention_step(q, k, v, ld, live, 0.5)
    assert same is live and torch.equal(live, s1) and torch.equal(o2, o) and torch.equal(s0, keep)
    # a sequence without a token keeps its state, bit for bit, and its rows
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    lens[0] = 0
    o3 = torch.full_like(o, 3.0)
    _, s3 = fwpkm.linear_attention_step(q, k, v, ld, s0, 0.5, lens=lens, o=o3, in_place=False)
    assert torch.equal(s3[0], s0[0]) and torch.equal(s3[1:], s1[1:])
    assert bool((o3[0] == 3.0).all()) and torch.equal(o3[1:], o[1:])


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64), ("bf16", 40)])
def test_prompt_in_parts_then_token_by_token(dtype, d):
    # a prompt, a second prompt from its state, then single tokens: one sequence
    B, H, T, dv, ld = 2, 2, 420, 64, decays(2)
    q, k, v, _, s0, _ = tensors(B, H, T, d, dv, dtype, 7)
    o = torch.empty(B, H, T, dv, dtype=DT[dtype], device="cuda")
    st = s0.clone()
    for a, b in ((0, 200), (200, 413)):
        fwpkm.linear_attention(q[:, :, a:b], k[:, :, a:b], v[:, :, a:b], ld, 0.5, s0=st, o=o[:, :, a:b], sT=st)
    for t in range(413, T):
        fwpkm.linear_attention_step(q[:, :, t:t + 1], k[:, :, t:t + 1], v[:, :, t:t + 1], ld, st, 0.5, o=o[:, :, t:t + 1])
    check_forward(q, k, v, ld, 0.5, s0, None, o, st, "in parts")


def test_broadcast_inputs_and_gradient_by_differences():
    # keys and values shared by the heads (stride 0); their gradient is the sum over the heads
    B, H, T, d, dv = 1, 3, 70, 16, 16
    q, k, v, do, s0, _ = tensors(B, H, T, d, dv, "f32", 3, "bhtd")
    k, v, ld = k[:, :1].expand(B, H, T, d), v[:, :1].expand(B, H, T, dv), decays(H)
    o, _ = fwpkm.linear_attention(q, k, v, ld, 1.0, s0=s0)
    check_forward(q, k, v, ld, 1.0, s0, None, o, None, "shared heads")
    dq, dk, dv_, _ = fwpkm.linear_attention_backward(q, k, v, ld, do, 1.0, s0=s0)
    check_backward(q, k, v, ld, do, 1.0, s0, None, None, (dq, dk, dv_), None, "shared heads")
    # central differences of the kernel's own loss in fp64 (o is linear in k): the difference of
    # the oracle's loss at k + e and k - e, divided by 2 e, is the gradient itself
    e = np.random.default_rng(0).normal(size=(T, d))
    K = f64(k)
    loss = lambda s: float((f64(do) * op.linear_attention(f64(q), K + s * e, f64(v), f64(ld), 1.0, f64(s0))[0]).sum())  # noqa: E731
    want = (loss(1.0) - loss(-1.0)) / 2
    got = float((f64(dk).sum(1)[0] * e).sum())
    size = float((np.abs(f64(dk)).sum(1)[0] * np.abs(e)).sum())
    assert abs(got - want) <= 1e-4 * size


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_prompt_and_masked_values(dtype):
    B, H, d, dv = 2, 2, 64, 64
    q, k, v, do, s0, dsT = tensors(B, H, 0, d, dv, dtype, 1, "bhtd")
    ld = decays(H)
    o, sT = fwpkm.linear_attention(q, k, v, ld, s0=s0, final_state=True)
    assert tuple(o.shape) == (B, H, 0, dv) and torch.equal(sT, s0)
    _, sT = fwpkm.linear_attention(q, k, v, ld, final_state=True)
    assert not sT.any()
    *_, ds0 = fwpkm.linear_attention_backward(q, k, v, ld, do, 0.5, d_sT=dsT)
    assert torch.equal(ds0, dsT)
    # infinities travel with their token: earlier rows stay finite
    q, k, v, _, _, _ = tensors(1, 1, 300, d, dv, dtype, 1, "bhtd")
    v[0, 0, 200, 3] = INF
    o, _ = fwpkm.linear_attention(q, k, v, ld[:1])
    assert torch.isfinite(o[0, 0, :128]).all() and not torch.isfinite(o[0, 0, 200:, 3]).any()
    assert torch.isfinite(o[0, 0, :, 4:]).all()


def test_offsets_beyond_32_bits():
    # two sequences 2.3e9 elements apart
    B, H, T, d = 2, 2, 140, 64
    flat = torch.zeros(2300000000 + 3 * 2 * 140 * 64, dtype=torch.bfloat16, device="cuda")
    view = lambda i: torch.as_strided(flat, (B, H, T, d), (2300000000, T * d, d, 1), i * H * T * d)  # noqa: E731
    src = tensors(B, H, T, d, d, "bf16", 4, "bhtd")
    far = [view(i) for i in range(3)]
    for x, y in zip(far, src[:3]):
        x.copy_(y)
    ld = decays(H)
    o, sT = fwpkm.linear_attention(*far, ld, s0=src[4], final_state=True)
    want, wT = fwpkm.linear_attention(*src[:3], ld, s0=src[4], final_state=True)
    assert torch.equal(o, want) and torch.equal(sT, wT)
    o, sT = fwpkm.linear_attention_step(*far, ld, src[4], in_place=False)
    want, wT = fwpkm.linear_attention_step(*src[:3], ld, src[4], in_place=False)
    assert torch.equal(o, want) and torch.equal(sT, wT)


@pytest.mark.parametrize("dtype,d,T", [("bf16", 128, 900), ("f32", 64, 600)])
def test_repeated_captured_and_on_another_stream(dtype, d, T):
    B, H, dv, ld = 1, 2, 64, decays(2)
    q, k, v, do, s0, dsT = tensors(B, H, T, d, dv, dtype, 11)
    first = fwpkm.linear_attention(q, k, v, ld, s0=s0, final_state=True)
    again = fwpkm.linear_attention(q, k, v, ld, s0=s0, final_state=True)
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = fwpkm.linear_attention(q, k, v, ld, s0=s0, final_state=True)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, other))
    # two graphs that share a workspace, replayed in turn on changed inputs
    ws = torch.empty(max(1, fwpkm.linear_attention_workspace_size(q, v), fwpkm.linear_attention_workspace_size(q, v, True)),
                     dtype=torch.uint8, device="cuda")
    q2 = q.clone()
    torch.cuda.synchronize()
    gf, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gf):
        f = fwpkm.linear_attention(q2, k, v, ld, s0=s0, final_state=True, workspace=ws)
    with torch.cuda.graph(gb):
        g = fwpkm.linear_attention_backward(q2, k, v, ld, do, s0=s0, d_sT=dsT, workspace=ws)
    q2.mul_(-2)
    for x in (gf, gb, gf, gb):
        x.replay()
    torch.cuda.synchronize()
    want = fwpkm.linear_attention(q2, k, v, ld, s0=s0, final_state=True)
    assert all(torch.equal(x, y) for x, y in zip(f, want))
    want = fwpkm.linear_attention_backward(q2, k, v, ld, do, s0=s0, d_sT=dsT)
    assert all(torch.equal(x, y) for x, y in zip(g, want))
    # ds0 in d_sT's own memory
    own = dsT.clone()
    got = fwpkm.linear_attention_backward(q2, k, v, ld, do, s0=s0, d_sT=own, ds0=own)
    assert got[3] is own and all(torch.equal(x, y) for x, y in zip(got, want))
