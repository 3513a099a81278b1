"""The operators around the memory as a program uses them together.

Training: tokens are looked up in an embedding, their rows hold q, k and v of linear attention,
whose output is a router's logits; the selected slots of a second table are read with weights,
and the balance loss keeps the router's use of them even.  The gradients run back through all
four into both tables.  Serving: a prompt, then token by token, through the same calls.

Tolerances (u = 2^-24): each operator alone is off by what its own tests allow, fp32 sums of
absolute values A times c u.  In the chain
  * o is off by eo = c u A_o, c = T + d + d_v + 32;
  * with m = max eo a probability is off by a relative 2 m (e^(2 max) over its sum) and 8 u of
    its own arithmetic (exponential, sum of E terms as a tree, quotient), so the gradient
    g P (a - sum a P) is off by e = g (2 m + (E + 16) u) P (|a - sum a P| + 2 sum |a| P);
  * linear attention's gradients are linear in d_o: off by its backward of e over absolute
    values, and c u times its backward of |d_o|; with q, k, v exact;
  * the embedding's gradient adds its tokens' errors, and (tokens + 2) u of their sum.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_weight_memory_chunk_b200 import fwpkm  # noqa: E402

from oracle import operators as op  # noqa: E402

U = 2.0 ** -24
B, T, H, D, K, WORDS = 2, 150, 2, 16, 4, 40
E = H * D              # slots of the router


def f64(t):
    return t.double().cpu().numpy()


def program(seed, dtype):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    tok = torch.randint(WORDS, (B, T), generator=g, device="cuda", dtype=torch.int32)
    tok[:, -3:] = -1                                       # padding
    return dict(emb=r(WORDS, 3 * E).to(dtype), slots=r(E, 24).to(dtype), tok=tok, ld=torch.tensor([-0.05, -1.0], device="cuda"),
                mask=(tok >= 0).contiguous(), dy=r(B, T, 24).to(dtype), w=torch.softmax(r(B, T, K), -1), scale=0.25)


def heads(x):
    """q, k, v [B][H][T][D] of rows [B][T][3 H D]."""
    return [x.view(B, T, 3, H, D)[:, :, i].transpose(1, 2) for i in range(3)]


def train_step(p):
    x = fwpkm.lookup(p["emb"], p["tok"])
    q, k, v = heads(x)
    o, _ = fwpkm.linear_attention(q, k, v, p["ld"], scale=p["scale"])
    logits = o.transpose(1, 2).reshape(B, T, E)
    idx = logits.float().topk(K, -1).indices.to(torch.int32)
    loss = fwpkm.balance_loss(logits, idx, mask=p["mask"])
    y = fwpkm.lookup(p["slots"], idx, w=p["w"])
    d_slots, dw = fwpkm.lookup_backward(p["slots"], idx, p["dy"], w=p["w"], grad_dtype=torch.float32)
    d_logits = fwpkm.balance_loss_backward(logits, loss, mask=p["mask"])
    d_o = d_logits.view(B, T, H, D).transpose(1, 2)
    dx = torch.empty_like(x)
    fwpkm.linear_attention_backward(q, k, v, p["ld"], d_o, scale=p["scale"], grads=heads(dx), state_grad=False)
    d_emb = torch.zeros(WORDS, 3 * E, device="cuda")
    fwpkm.lookup_backward(p["emb"], p["tok"], dx, d_table=d_emb, accumulate=True)
    return dict(o=o, logits=logits, idx=idx, loss=loss.loss, counts=loss.counts, y=y, d_slots=d_slots, dw=dw,
                d_logits=d_logits, d_emb=d_emb)


def near(got, ref, tol, what):
    off = np.abs(f64(got) - ref)
    assert (off <= tol).all(), f"{what}: worst {np.max(off / np.maximum(tol, 1e-300)):.3g} of the bound"


def test_a_training_step_against_the_oracle():
    p = program(5, torch.float32)
    r = train_step(p)
    emb, tok, idx, ld = f64(p["emb"]), p["tok"].cpu().numpy(), r["idx"].cpu().numpy(), f64(p["ld"])
    x = op.lookup(emb, tok.reshape(-1, 1)).reshape(B, T, 3, H, D)
    q, k, v = (x[:, :, i].transpose(0, 2, 1, 3) for i in range(3))
    c = T + 2 * D + 32
    o, _ = op.linear_attention(q, k, v, ld, p["scale"])
    eo = c * U * op.linear_attention(np.abs(q), np.abs(k), np.abs(v), ld, p["scale"])[0]
    near(r["o"], o, eo, "o")
    logits, m = o.transpose(0, 2, 1, 3).reshape(B, T, E), 2 * eo.max()
    d_logits, e_logits = np.zeros((B, T, E)), np.zeros((B, T, E))
    for b in range(B):
        on = tok[b] >= 0
        loss, counts, _, a, n = op.balance_loss(logits[b], idx[b], on)
        assert np.array_equal(r["counts"][b].cpu().numpy(), counts)
        P = op.softmax_rows(logits[b])
        g = 1.0 / n
        c_ = (P * a).sum(1, keepdims=True)
        d_logits[b] = op.balance_backward(logits[b], idx[b], on)
        e_logits[b] = g * (m + (E + 16) * U) * P * (np.abs(a - c_) + 2 * (P * np.abs(a)).sum(1, keepdims=True))
        e_logits[b][~on] = 0.0
        # the loss: E sum f u, its u off by the probabilities' relative error (fp64 sums)
        near(r["loss"][b], loss, (m + (E + n + 16) * U) * loss, "loss")
    near(r["d_logits"], d_logits, e_logits, "d_logits")
    as_heads = lambda z: z.reshape(B, T, H, D).transpose(0, 2, 1, 3)  # noqa: E731
    ab = [np.abs(z) for z in (q, k, v)]
    ref = op.linear_attention_backward(q, k, v, ld, as_heads(d_logits), p["scale"])
    e1 = op.linear_attention_backward(*ab, ld, as_heads(e_logits), p["scale"])
    e2 = op.linear_attention_backward(*ab, ld, np.abs(as_heads(d_logits)), p["scale"])
    rows = lambda z: np.stack([y.transpose(0, 2, 1, 3) for y in z[:3]], 2).reshape(B * T, 3 * E)  # noqa: E731
    dx, ex = rows(ref), rows(e1) + c * U * rows(e2)
    d_emb, _ = op.lookup_backward(emb, tok.reshape(-1, 1), dx)
    tol, _ = op.lookup_backward(emb, tok.reshape(-1, 1), ex + (B * T + 2) * U * np.abs(dx))
    near(r["d_emb"], d_emb, tol, "d_emb")
    # the bag of slots
    flat, wf, dy = idx.reshape(-1, K), f64(p["w"]).reshape(-1, K), f64(p["dy"]).reshape(B * T, -1)
    slots = f64(p["slots"])
    near(r["y"].reshape(B * T, -1), op.lookup(slots, flat, wf), (K + 2) * U * op.lookup(np.abs(slots), flat, wf), "y")
    ds, dw = op.lookup_backward(slots, flat, dy, wf)
    es, ew = op.lookup_backward(np.abs(slots), flat, np.abs(dy), wf)
    near(r["d_slots"], ds, (B * T * K + 2) * U * es, "d_slots")
    near(r["dw"].reshape(-1, K), dw, (24 + 2) * U * ew, "dw")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_training_step_captured_and_replayed(dtype):
    """The whole step in one graph, replayed on other inputs, gives what eager calls give."""
    p = program(6, dtype)
    train_step(p)                                          # (first calls load the kernels)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = train_step(p)
    other = program(7, dtype)
    for name in ("emb", "slots", "tok", "mask", "dy", "w"):
        p[name].copy_(other[name])
    graph.replay()
    graph.replay()
    want = train_step(other)
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(r[name], want[name]), name
        assert torch.isfinite(want[name].float()).all(), name


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_prompt_then_token_by_token(dtype):
    """Serving: each new token's row is looked up and its heads step from the prompt's state; the
    router reads single tokens.  Against the oracle over the whole sequence."""
    p, n0 = program(8, dtype), 130
    q, k, v = heads(fwpkm.lookup(p["emb"], p["tok"]))
    part = lambda t: t[:, :, :n0]  # noqa: E731
    o, state = fwpkm.linear_attention(part(q), part(k), part(v), p["ld"], scale=p["scale"], final_state=True)
    outs = [o]
    for t in range(n0, T):
        row = fwpkm.lookup(p["emb"], p["tok"][:, t:t + 1].contiguous())
        q1, k1, v1 = [row.view(B, 1, 3, H, D)[:, :, i].transpose(1, 2) for i in range(3)]
        o1, same = fwpkm.linear_attention_step(q1, k1, v1, p["ld"], state, scale=p["scale"])
        assert same is state
        outs.append(o1)
    fwpkm.linear_attention_sync()
    qkv = [f64(z) for z in (q, k, v)]
    ro, rs = op.linear_attention(*qkv, f64(p["ld"]), p["scale"])
    ao, as_ = op.linear_attention(*(np.abs(z) for z in qkv), f64(p["ld"]), p["scale"])
    bf = dtype == torch.bfloat16
    c = T + 2 * D + 32 + (2.0 ** 16 + 2.0 ** 8 if bf else 0.0)
    tol = c * U * ao
    near(torch.cat(outs, 2), ro, tol + (2.0 ** -8 * (np.abs(ro) + tol) if bf else 0.0), "o")
    near(state, rs, (T + 2 * D + 32) * U * as_, "state")


def test_on_a_stream_of_its_own():
    """A call on another stream takes its workspace and outputs from that stream's memory: what the
    current stream allocates and writes meanwhile is other memory."""
    side = torch.cuda.Stream()
    g = torch.Generator("cuda").manual_seed(3)
    table = torch.randn(3000, 64, generator=g, device="cuda")
    idx = torch.randint(3000, (20000,), generator=g, device="cuda")
    d_out = torch.randn(20000, 64, generator=g, device="cuda")
    q, k, v = (torch.randn(1, 2, 3000, 64, generator=g, device="cuda") for _ in range(3))
    ld = torch.tensor([-0.01, -0.1], device="cuda")
    x = torch.randn(2, 5000, 128, generator=g, device="cuda")
    want = (fwpkm.lookup_backward(table, idx, d_out)[0], *fwpkm.linear_attention(q, k, v, ld, final_state=True),
            fwpkm.balance_loss(x, kind="entropy").slope)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(3):
        got = (fwpkm.lookup_backward(table, idx, d_out, stream=side)[0],
               *fwpkm.linear_attention(q, k, v, ld, final_state=True, stream=side),
               fwpkm.balance_loss(x, kind="entropy", stream=side).slope)
        # what a freed workspace of the current stream's memory would be handed out for
        junk = [torch.full((1 << s,), float("nan"), device="cuda") for s in range(8, 24)]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk


def test_a_wait_that_runs_out_is_reported():
    """The bounded wait of the tensor-core pass is made to run out: linear_attention_sync raises, and
    the next call runs clean (tensor memory was freed)."""
    g = torch.Generator("cuda").manual_seed(4)
    q, k, v = (torch.randn(2, 4, 300, 64, generator=g, device="cuda").bfloat16() for _ in range(3))
    ld = torch.full((4,), -0.1, device="cuda")
    want = fwpkm.linear_attention(q, k, v, ld, final_state=True)
    fwpkm.linear_attention_sync()
    fwpkm.test_stall_waits(1)
    fwpkm.linear_attention(q, k, v, ld, final_state=True)
    with pytest.raises(fwpkm.FwpkmError) as e:
        fwpkm.linear_attention_sync()
    assert e.value.status == fwpkm.ERR_TIMEOUT
    fwpkm.linear_attention_sync()  # cleared
    got = fwpkm.linear_attention(q, k, v, ld, final_state=True)
    fwpkm.linear_attention_sync()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
