"""The operators around the memory: table lookups, the balance loss and linear attention.

Three families, each in a plain form (elementary torch operations in 32 bits, rounded once)
and, where ``own`` is true, through this package's public entry points:

  lookup       out_t = scale * sum_r w[t,r] table[idx[t,r]] (one row per token without w), and its
               gradients: d_table by sorted indices (dense, or added to the touched rows), dw.
  balance      usage and load of experts (sub-keys, slots): the loss, the counts and the
               gradient with respect to the logits.
  attention    linear attention with a decay per head, S_t = a S_{t-1} + k_t v_t^T,
               o_t = scale q_t S_t: a prompt in chunks, its backward, and token by token.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of a small batch: the token embedding of 16 sequences
        {"name": "lookup_decode", "op": "lookup", "rows": 32768, "width": 1024, "n": 16, "R": 1, "dtype": "bf16"},
        # the token embedding of a training batch (8 x 4096 tokens, d_model = 2048)
        {"name": "lookup_train", "op": "lookup", "rows": 131072, "width": 2048, "n": 32768, "R": 1, "dtype": "bf16"},
        # its gradient: dense fp32 rows, half the batch, a tail of padding (index -1)
        {"name": "lookup_train_grad", "op": "lookup_grad", "rows": 131072, "width": 2048, "n": 16384, "R": 1,
         "dtype": "bf16", "add": False},
        # a product-key value table of 2^20 slots trained as slow weights: 32 weighted rows per
        # token, the gradient added to the touched rows, and the weights' gradient
        {"name": "lookup_slots_grad", "op": "lookup_grad", "rows": 1048576, "width": 256, "n": 2048, "R": 32,
         "dtype": "f32", "add": True},
        # a router of 64 experts over a micro-batch with padding: loss, counts and gradient
        {"name": "balance_router", "op": "balance", "G": 1, "T": 4096, "E": 64, "k": 8, "dtype": "bf16",
         "kind": "load", "masked": True},
        # sub-key usage of 8 memories (two halves each, n = 1024) over a sequence of 4096 tokens
        {"name": "balance_subkeys", "op": "balance", "G": 16, "T": 4096, "E": 1024, "k": 32, "dtype": "f32",
         "kind": "entropy", "masked": False},
        # a long prompt of one sequence: few heads, so the work has to be split along the tokens
        {"name": "attention_prompt_long", "op": "attention", "B": 1, "H": 16, "T": 16384, "d": 128, "dv": 128,
         "dtype": "bf16", "ragged": False},
        # a batch of prompts of different lengths, one of them empty
        {"name": "attention_prompt_batch", "op": "attention", "B": 16, "H": 16, "T": 4096, "d": 128, "dv": 128,
         "dtype": "bf16", "ragged": True},
        # fp32 heads of odd sizes at an odd length
        {"name": "attention_prompt_f32", "op": "attention", "B": 2, "H": 5, "T": 1003, "d": 72, "dv": 100,
         "dtype": "f32", "ragged": True},
        # the backward pass of a training batch
        {"name": "attention_grad", "op": "attention_grad", "B": 8, "H": 16, "T": 4096, "d": 128, "dv": 128,
         "dtype": "bf16", "ragged": False},
        # one token of one sequence: latency
        {"name": "attention_token", "op": "attention_token", "B": 1, "H": 8, "T": 1, "d": 64, "dv": 64,
         "dtype": "bf16", "ragged": False},
        # one token of a serving batch: every head's state read and written once
        {"name": "attention_token_batch", "op": "attention_token", "B": 128, "H": 16, "T": 1, "d": 128, "dv": 128,
         "dtype": "bf16", "ragged": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "lookup_grad", "balance", "attention", "attention", "attention_grad",
                     "attention_token"])
    dtype = rng.choice(["bf16", "f32"])
    if op in ("lookup", "lookup_grad"):
        R = rng.choice([1, 1, 1, 8, 32, _log(rng, 2, 128)])
        width = rng.choice([64, 128, 256, 512, 1024, 2048, _log(rng, 17, 2048)])
        rows = _log(rng, 64, min(1 << 20, (1 << 28) // width))
        n = _log(rng, 1, max(1, min(32768, (1 << 26) // (width * R))))
        c = {"op": op, "rows": rows, "width": width, "n": n, "R": R, "dtype": dtype}
        if op == "lookup_grad":
            c["add"] = rng.random() < 0.5
        return c
    if op == "balance":
        E = rng.choice([8, 16, 64, 128, 256, 512, 1024, _log(rng, 3, 4096)])
        G = rng.choice([1, 2, 8, 16])
        T = _log(rng, 1, max(1, min(65536, (1 << 26) // (G * E))))
        return {"op": op, "G": G, "T": T, "E": E, "k": min(E, rng.choice([1, 2, 4, 8, 32])), "dtype": dtype,
                "kind": rng.choice(["load", "entropy"]), "masked": rng.random() < 0.5}
    d = rng.choice([64, 128, 128, 8 * rng.randint(2, 16), rng.randint(16, 256)])
    dv = rng.choice([d, d, 64, 128, 8 * rng.randint(2, 16)])
    c = {"op": op, "B": _log(rng, 1, 16), "H": rng.choice([1, 4, 8, 16, rng.randint(2, 24)]), "T": 1, "d": d, "dv": dv,
         "dtype": dtype, "ragged": rng.random() < 0.5}
    if op == "attention_token":
        c["B"] = _log(rng, 1, max(1, (1 << 25) // (c["H"] * d * dv)))
        c["T"] = rng.choice([1, 1, 1, 2, rng.randint(2, 16)])
    else:
        # fp32 heads and heads wider than 128 take shorter prompts, so that no draw outweighs the listed cases
        most = (1 << 18) // (c["B"] * c["H"])
        if dtype == "f32" or d > 128:
            most = (1 << 16) // (c["B"] * c["H"])
        c["T"] = _log(rng, 1, max(2, min(16384, most)))
    return c


# ----------------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _lens(case):
    """Lengths of the batch's sequences: full, then shorter in even steps, the last one of several empty."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return None
    if B == 1:
        return [T - T // 8]
    return [T - (T * b) // (B - 1) if b < B - 1 else 0 for b in range(B)]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    dt = DT[case["dtype"]]
    if case["op"] in ("lookup", "lookup_grad"):
        rows, width, n, R = case["rows"], case["width"], case["n"], case["R"]
        s["table"] = torch.empty(rows, width, dtype=dt, device="cuda")
        for r0 in range(0, rows, 65536):
            part = s["table"][r0:r0 + 65536]
            part.copy_(0.02 * _randn(g, *part.shape))
        s["scale"] = math.sqrt(width)
        if R == 1:
            # token frequencies fall off about as 1 / rank; the ranks are spread over the table, and
            # the last thirty-second of the tokens is padding
            u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
            rank = torch.exp(u * math.log(rows + 1.0)).long().clamp(1, rows) - 1
            step = 2654435761 % rows
            while math.gcd(step, rows) != 1:
                step += 1
            s["idx"] = (rank * step) % rows
            s["idx"][n - n // 32:] = -1
            s["w"] = None
        else:
            # slots of a product-key selection: distinct enough to be uniform, softmax weights
            s["idx"] = torch.randint(rows, (n, R), generator=g, device="cuda", dtype=torch.int32)
            s["w"] = torch.softmax(_randn(g, n, R), -1)
            s["scale"] = 1.0
        if case["op"] == "lookup_grad":
            s["d_out"] = _randn(g, n, width).to(dt)
            s["d_table"] = _randn(g, rows, width) if case["add"] else None
    elif case["op"] == "balance":
        G, T, E, k = case["G"], case["T"], case["E"], case["k"]
        # skewed experts: a bias per expert on top of the tokens' own logits
        s["x"] = (_randn(g, G, T, E) + 0.5 * _randn(g, G, 1, E)).to(dt)
        s["idx"] = s["x"].float().topk(k, -1).indices.to(torch.int32)
        s["mask"] = None
        if case["masked"]:
            s["mask"] = torch.rand(G, T, generator=g, device="cuda") < 0.9
            s["mask"][:, T - T // 8:] = False
            s["mask"][:, :1] = True
            s["x"][~s["mask"]] = float("nan")  # what a padded row holds is nobody's business
        s["d_loss"] = 0.5 + torch.rand(G, generator=g, device="cuda")
    else:
        B, H, T, d, dv = (case[x] for x in ("B", "H", "T", "d", "dv"))
        # [B][T][H][.] as a projection writes it, seen as [B][H][T][.]; unit-norm keys
        s["q"] = _randn(g, B, T, H, d).to(dt).transpose(1, 2)
        s["k"] = (_randn(g, B, T, H, d) / math.sqrt(d)).to(dt).transpose(1, 2)
        s["v"] = _randn(g, B, T, H, dv).to(dt).transpose(1, 2)
        # decays from 1 - 2^-3 to 1 - 2^-9 over the heads
        h = torch.arange(H, device="cuda", dtype=torch.float64)
        s["log_decay"] = torch.log1p(-torch.exp2(-3.0 - 6.0 * h / max(1, H - 1))).float()
        s["scale"] = 1.0 / math.sqrt(d)
        s["s0"] = _randn(g, B, H, d, dv)
        ln = _lens(case)
        s["lens"] = None if ln is None else torch.tensor(ln, dtype=torch.int32, device="cuda")
        # outputs: rows behind a sequence's end are left as they were
        s["o"] = torch.zeros(B, T, H, dv, dtype=dt, device="cuda").transpose(1, 2)
        if case["op"] == "attention_grad":
            s["d_o"] = _randn(g, B, T, H, dv).to(dt).transpose(1, 2)
            s["d_sT"] = _randn(g, B, H, d, dv)
            s["grads"] = tuple(torch.zeros(B, T, H, w, dtype=dt, device="cuda").transpose(1, 2) for w in (d, d, dv))
    return s


# ----------------------------------------------------------------------------- the plain forms

def _lookup_plain(s):
    idx, dt = s["idx"].long(), s["table"].dtype
    ok = (idx >= 0) & (idx < s["rows"])
    rows = s["table"][torch.where(ok, idx, 0)].float()
    if s["w"] is None:
        return (torch.where(ok[:, None], rows, 0.0) * s["scale"]).to(dt)
    return ((torch.where(ok, s["w"], 0.0)[..., None] * rows).sum(1) * s["scale"]).to(dt)


def _lookup_grad_plain(s):
    idx, n, width = s["idx"].long(), s["n"], s["width"]
    ok = (idx >= 0) & (idx < s["rows"])
    at = torch.where(ok, idx, 0)
    d_out = s["d_out"].float() * s["scale"]
    d_table = s["d_table"] if s["add"] else torch.zeros(s["rows"], width, device=d_out.device)
    if s["w"] is None:
        d_table.index_add_(0, at, torch.where(ok[:, None], d_out, 0.0))
        return {"d_table": d_table}
    part = torch.where(ok, s["w"], 0.0)[..., None] * d_out[:, None, :]
    d_table.index_add_(0, at.reshape(-1), part.reshape(-1, width))
    dw = torch.where(ok, (s["table"][at].float() * d_out[:, None, :]).sum(-1), 0.0)
    return {"d_table": d_table, "dw": dw}


def _balance_plain(s):
    x, G, T, E = s["x"].float(), s["G"], s["T"], s["E"]
    on = torch.ones(G, T, dtype=torch.bool, device=x.device) if s["mask"] is None else s["mask"]
    x = torch.where(on[..., None], x, 0.0)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    P = torch.where(on[..., None], e / e.sum(-1, keepdim=True), 0.0)
    n = on.sum(-1, keepdim=True).float()
    usage = P.sum(1) / n
    counts = torch.zeros(G, E, dtype=torch.int32, device=x.device)
    counts.scatter_add_(1, s["idx"].long().reshape(G, -1), on[..., None].expand(s["idx"].shape).reshape(G, -1).int())
    if s["kind"] == "load":
        f = counts / counts.sum(-1, keepdim=True).float()
        loss = E * (f * usage).sum(-1)
        slope = E * f - 1.0  # less a constant, which the softmax's gradient does not see
    else:
        loss = torch.where(usage > 0, usage * torch.log(usage), 0.0).sum(-1)
        slope = torch.log(usage * E)
    c = (P * slope[:, None, :]).sum(-1, keepdim=True)
    dx = (s["d_loss"] / n[:, 0])[:, None, None] * P * (slope[:, None, :] - c)
    return {"loss": loss, "counts": counts, "usage": usage, "dx": dx.to(s["x"].dtype)}


def _powers(log_decay, e):
    """decay^e for every head, 0 where e < 0: [H] + e's shape, angles in 64 bits."""
    ld = log_decay.double().view(-1, *([1] * e.dim()))
    return torch.where(e >= 0, torch.exp(ld * e.clamp(min=0).double()), 0.0).float()


def _scan(q, k, v, log_decay, reverse=False, C=128):
    """sum over s <= t (s >= t if reverse) of decay^|t-s| (q_t . k_s) v_s, all chunks at once."""
    B, H, T, d = q.shape
    dv = v.shape[-1]
    if reverse:
        q, k, v = q.flip(2), k.flip(2), v.flip(2)
    n = -(-T // C)
    pad = n * C - T
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)).view(B, H, n, C, -1) for x in (q, k, v))
    i = torch.arange(C, device=q.device)
    P = (q @ k.transpose(-1, -2)) * _powers(log_decay, i[:, None] - i[None, :])[:, None]
    o = P @ v
    if n > 1:
        kw = k * _powers(log_decay, C - 1 - i)[:, None, :, None]
        part = kw.transpose(-1, -2) @ v                                    # every chunk's own state
        c = torch.arange(n, device=q.device)
        carry = _powers(log_decay, C * (c[:, None] - 1 - c[None, :]))       # chunk c' into chunk c's start
        start = (carry @ part.view(B, H, n, d * dv)).view(B, H, n, d, dv)
        o = o + (q * _powers(log_decay, i + 1)[:, None, :, None]) @ start
    o = o.view(B, H, n * C, dv)[:, :, :T]
    return o.flip(2) if reverse else o


def _live(s, x):
    """x in 32 bits with zeros behind every sequence's end."""
    x = x.float()
    if s["lens"] is None:
        return x
    t = torch.arange(s["T"], device=x.device)
    return torch.where((t < s["lens"][:, None])[:, None, :, None], x, 0.0)


def _ends(s):
    """[B] lengths."""
    if s["lens"] is None:
        return torch.full((s["B"],), s["T"], device=s["q"].device)
    return s["lens"].long()


def _attention_plain(s):
    q, k, v = (_live(s, s[x]) for x in "qkv")
    ld, ln, t = s["log_decay"], _ends(s), torch.arange(s["T"], device=q.device)
    o = _scan(q, k, v, ld) + (q * _powers(ld, t + 1)[..., None]) @ s["s0"]
    w = _powers(ld, ln[:, None] - 1 - t).transpose(0, 1)                     # [B][H][T]
    sT = (k * w[..., None]).transpose(-1, -2) @ v + _powers(ld, ln).transpose(0, 1)[..., None, None] * s["s0"]
    return {"o": (o * s["scale"]).to(s["q"].dtype), "sT": sT}


def _attention_grad_plain(s):
    q, k, v, do = (_live(s, s[x]) for x in ("q", "k", "v", "d_o"))
    ld, ln, t, dt = s["log_decay"], _ends(s), torch.arange(s["T"], device=q.device), s["q"].dtype
    do = do * s["scale"]
    first = _powers(ld, t + 1)[..., None]                                   # [H][T][1]
    last = _powers(ld, ln[:, None] - 1 - t).transpose(0, 1)[..., None]       # [B][H][T][1]
    dq = _scan(do, v, k, ld) + (do * first) @ s["s0"].transpose(-1, -2)
    dk = _scan(v, do, q, ld, True) + (v * last) @ s["d_sT"].transpose(-1, -2)
    dv = _scan(k, q, do, ld, True) + (k * last) @ s["d_sT"]
    ds0 = (q * first).transpose(-1, -2) @ do + _powers(ld, ln).transpose(0, 1)[..., None, None] * s["d_sT"]
    return {"dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt), "ds0": ds0}


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "lookup":
        return _lookup_plain(s)
    if op == "lookup_grad":
        return _lookup_grad_plain(s)
    if op == "balance":
        return _balance_plain(s)
    if op == "attention_grad":
        return _attention_grad_plain(s)
    return _attention_plain(s)  # a prompt, or a few tokens: the same formula


def _run_own(s):
    from sparse_weight_memory_chunk_b200 import fwpkm
    op = s["op"]
    if op == "lookup":
        return fwpkm.lookup(s["table"], s["idx"], w=s["w"], scale=s["scale"])
    if op == "lookup_grad":
        d_table, dw = fwpkm.lookup_backward(s["table"], s["idx"], s["d_out"], w=s["w"], scale=s["scale"],
                                            d_table=s["d_table"], accumulate=s["add"], grad_dtype=torch.float32)
        return {"d_table": d_table} if dw is None else {"d_table": d_table, "dw": dw}
    if op == "balance":
        r = fwpkm.balance_loss(s["x"], idx=s["idx"], mask=s["mask"], kind=s["kind"])
        dx = fwpkm.balance_loss_backward(s["x"], r, mask=s["mask"], d_loss=s["d_loss"])
        return {"loss": r.loss, "counts": r.counts, "usage": r.usage, "dx": dx}
    if op == "attention":
        o, sT = fwpkm.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], s0=s["s0"],
                                       lens=s["lens"], o=s["o"], final_state=True)
        return {"o": o, "sT": sT}
    if op == "attention_token":
        o, sT = fwpkm.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["s0"], scale=s["scale"],
                                            lens=s["lens"], o=s["o"], in_place=False)
        return {"o": o, "sT": sT}
    dq, dk, dv, ds0 = fwpkm.linear_attention_backward(s["q"], s["k"], s["v"], s["log_decay"], s["d_o"],
                                                      scale=s["scale"], s0=s["s0"], d_sT=s["d_sT"], lens=s["lens"],
                                                      grads=s["grads"])
    return {"dq": dq, "dk": dk, "dv": dv, "ds0": ds0}


# ----------------------------------------------------------------------------- floors

def _distinct(rows, draws):
    """Expected distinct rows of uniform draws."""
    return rows * -math.expm1(draws * math.log1p(-1.0 / rows)) if rows > 1 else 1.0


def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("lookup", "lookup_grad"):
        rows, width, n, R = case["rows"], case["width"], case["n"], case["R"]
        live = n - n // 32 if R == 1 else n
        # log-uniform ranks: rank r is drawn with chance about 1 / (r ln rows)
        if R == 1:
            r = np.arange(1, rows + 1)
            p = np.log1p(1.0 / r) / math.log(rows + 1.0)
            used = float(-np.expm1(live * np.log1p(-np.minimum(p, 1 - 1e-12))).sum())
        else:
            used = _distinct(rows, live * R)
        index = n * R * (8 if R == 1 else 4 + 4)
        if op == "lookup":
            return {"bytes": index + used * width * b + n * width * b, "flops": 2.0 * n * R * width}
        grad = 2 * 4 * used * width if case["add"] else 4 * rows * width
        dw = used * width * b + 4 * n * R if R > 1 else 0
        return {"bytes": index + n * width * b + grad + dw, "flops": (2.0 if R == 1 else 4.0) * n * R * width}
    if op == "balance":
        G, T, E, k = case["G"], case["T"], case["E"], case["k"]
        return {"bytes": 2 * G * T * E * b + G * T * (4 * k + (1 if case["masked"] else 0)) + G * E * 8,
                "flops": 8.0 * G * T * E}
    B, H, T, d, dv = (case[x] for x in ("B", "H", "T", "d", "dv"))
    ln = _lens(case)
    rows = H * (B * T if ln is None else sum(ln))
    state = 4 * B * H * d * dv
    if op == "attention_grad":
        # q, k, v, d_o in and dq, dk, dv out; s0 and d_sT in, ds0 out; six products with a state-sized matrix
        return {"bytes": rows * b * (2 * d + 2 * dv + 2 * d + dv) + 3 * state, "flops": 10.0 * rows * d * dv}
    return {"bytes": rows * b * (2 * d + 2 * dv) + 2 * state, "flops": 4.0 * rows * d * dv}


# ----------------------------------------------------------------------------- 64 bits

def _exact_attention(s, grad):
    """Token after token, as the recurrence is written."""
    q, k, v, s0 = (s[x].double() for x in ("q", "k", "v", "s0"))
    B, H, T = q.shape[:3]
    a = torch.exp(s["log_decay"].double()).view(1, H, 1, 1)
    ln = [T] * B if s["lens"] is None else s["lens"].tolist()
    live = torch.tensor([[t < n for n in ln] for t in range(T)], device=q.device).view(T, B, 1, 1, 1)
    col = lambda x, t: x[:, :, t, :, None]  # noqa: E731
    S, o = s0.clone(), torch.zeros(B, H, T, v.shape[-1], dtype=torch.float64, device=q.device)
    if not grad:
        for t in range(T):
            on = live[t]
            S = torch.where(on, a * S + col(k, t) * col(v, t).transpose(-1, -2), S)
            o[:, :, t] = torch.where(on, (col(q, t) * S).sum(-2, keepdim=True), 0.0)[:, :, 0] * s["scale"]
        return {"o": o, "sT": S}
    do = s["d_o"].double()
    dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device=q.device) for x in (q, k, v))
    for t in range(T):
        on = live[t]
        S = torch.where(on, a * S + col(k, t) * col(v, t).transpose(-1, -2), S)
        dq[:, :, t] = torch.where(on, S @ col(do, t), 0.0)[..., 0] * s["scale"]
    D = s["d_sT"].double()
    for t in reversed(range(T)):
        on = live[t]
        D = torch.where(on, D + s["scale"] * (col(q, t) * col(do, t).transpose(-1, -2)), D)
        dk[:, :, t] = torch.where(on, D @ col(v, t), 0.0)[..., 0]
        dv[:, :, t] = torch.where(on, D.transpose(-1, -2) @ col(k, t), 0.0)[..., 0]
        D = torch.where(on, a * D, D)
    return {"dq": dq, "dk": dk, "dv": dv, "ds0": D}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("attention", "attention_token"):
        return _exact_attention(s, False)
    if op == "attention_grad":
        return _exact_attention(s, True)
    if op == "balance":
        G, T, E = case["G"], case["T"], case["E"]
        loss, counts, usages, dxs = [], [], [], []
        for g in range(G):
            on = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"][g]
            x = s["x"][g][on].double()
            logP = x - torch.logsumexp(x, -1, keepdim=True)
            n = x.shape[0]
            u = logP.exp().mean(0)
            c = torch.bincount(s["idx"][g][on].long().reshape(-1), minlength=E)
            if case["kind"] == "load":
                slope = E * c.double() / c.sum()
                loss.append((slope * u).sum())
            else:
                slope = torch.log(u) + 1.0
                loss.append((u * torch.log(u)).sum())
            P = logP.exp() / n
            dx = torch.zeros(T, E, dtype=torch.float64, device="cuda")
            slope = slope - slope.mean()
            dx[on] = s["d_loss"][g].double() * P * (slope - n * (P * slope).sum(-1, keepdim=True))
            counts.append(c.int())
            usages.append(u)
            dxs.append(dx)
        return {"loss": torch.stack(loss), "counts": torch.stack(counts), "usage": torch.stack(usages),
                "dx": torch.stack(dxs)}
    idx = s["idx"].long().view(case["n"], case["R"])
    ok = (idx >= 0) & (idx < case["rows"])
    w = (torch.ones_like(idx, dtype=torch.float64) if s["w"] is None else s["w"].double()) * ok * s["scale"]
    at = idx.clamp(0, case["rows"] - 1)
    if op == "lookup":
        out = torch.zeros(case["n"], case["width"], dtype=torch.float64, device="cuda")
        for r in range(case["R"]):
            out += w[:, r, None] * s["table"][at[:, r]].double()
        return out
    d_out = s["d_out"].double()
    d_table = (s["d_table"].double() if case["add"]
               else torch.zeros(case["rows"], case["width"], dtype=torch.float64, device="cuda"))
    dw = torch.zeros(case["n"], case["R"], dtype=torch.float64, device="cuda")
    for r in range(case["R"]):
        d_table.index_add_(0, at[:, r], w[:, r, None] * d_out)
        dw[:, r] = ok[:, r] * s["scale"] * (d_out * s["table"][at[:, r]].double()).sum(-1)
    return {"d_table": d_table} if s["w"] is None else {"d_table": d_table, "dw": dw}
