"""CPU oracle of the operators around the memory: table lookups, the balance loss and linear
attention, each with its gradients.

TEST INFRASTRUCTURE ONLY (see oracle/backward.py).  Plain fp64 numpy from the definitions
that include/fwpkm.h states; the gradients are the formulas', pinned by central differences
of the forward functions in tests/test_oracle_operators_pins.py.
"""
from __future__ import annotations

import numpy as np


def lookup(table, idx, w=None, scale=1.0):
    """table [rows][width]; idx [n][R]; w [n][R] or None (ones) -> out [n][width]."""
    table, idx = np.asarray(table, np.float64), np.asarray(idx)
    ok = (idx >= 0) & (idx < table.shape[0])
    f = (np.ones(idx.shape) if w is None else np.asarray(w, np.float64)) * scale
    out = np.zeros((idx.shape[0], table.shape[1]))
    for t, r in zip(*np.nonzero(ok)):
        out[t] += f[t, r] * table[idx[t, r]]
    return out


def lookup_backward(table, idx, d_out, w=None, scale=1.0):
    """-> (d_table [rows][width], dw [n][R])."""
    table, idx, d_out = np.asarray(table, np.float64), np.asarray(idx), np.asarray(d_out, np.float64)
    ok = (idx >= 0) & (idx < table.shape[0])
    f = (np.ones(idx.shape) if w is None else np.asarray(w, np.float64)) * scale
    d_table, dw = np.zeros(table.shape), np.zeros(idx.shape)
    for t, r in zip(*np.nonzero(ok)):
        d_table[idx[t, r]] += f[t, r] * d_out[t]
        dw[t, r] = scale * np.dot(d_out[t], table[idx[t, r]])
    return d_table, dw


def softmax_rows(x):
    """Softmax of each row; zeros for a row without a logit above -inf."""
    x = np.asarray(x, np.float64)
    m = x.max(axis=-1, keepdims=True) if x.shape[-1] else x
    dead = m == -np.inf
    e = np.exp(x - np.where(dead, 0.0, m))
    e = np.where(dead, 0.0, e)
    s = e.sum(axis=-1, keepdims=True)
    return e / np.where(s == 0.0, 1.0, s)


def balance_loss(x, idx=None, mask=None, kind="load", coef=1.0):
    """One group: x [T][E], idx [T][k], mask [T] -> (loss, counts [E], usage [E], a [E], T used)."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    on = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    P = np.zeros((T, E))
    P[on] = softmax_rows(x[on])
    live = on & (P.sum(axis=1) > 0)
    n = int(live.sum())
    usage = P[live].sum(axis=0) / max(n, 1)
    counts = np.zeros(E, np.int64)
    if idx is not None:
        for t in np.nonzero(on)[0]:
            for e in np.asarray(idx)[t]:
                if 0 <= e < E:
                    counts[e] += 1
    if kind == "load":
        f = counts / max(int(counts.sum()), 1)
        return coef * E * float(f @ usage), counts, usage, E * f, n
    with np.errstate(divide="ignore"):
        lg = np.where(usage > 0, np.log(np.where(usage > 0, usage, 1.0)), 0.0)
    return coef * float(usage @ lg), counts, usage, np.where(usage > 0, lg + 1.0, 0.0), n


def balance_backward(x, idx=None, mask=None, kind="load", coef=1.0, d_loss=1.0):
    """-> dx [T][E]."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    on = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    _, _, _, a, n = balance_loss(x, idx, mask, kind, coef)
    P = np.zeros((T, E))
    P[on] = softmax_rows(x[on])
    if n == 0:
        return np.zeros((T, E))
    return d_loss * coef / n * P * (a[None, :] - (P @ a)[:, None])


def decay_of(log_decay):
    return np.exp(np.asarray(log_decay, np.float64))


def linear_attention(q, k, v, log_decay, scale=1.0, s0=None, lens=None):
    """q, k [B][H][T][d], v [B][H][T][d_v] -> (o, sT); rows of o behind a sequence's end are 0."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, H, T, d = q.shape
    dv = v.shape[3]
    a = decay_of(log_decay)
    o = np.zeros((B, H, T, dv))
    sT = np.zeros((B, H, d, dv)) if s0 is None else np.array(s0, np.float64)
    for b in range(B):
        n = T if lens is None else int(np.clip(lens[b], 0, T))
        S = sT[b]
        for t in range(n):
            S = a[:, None, None] * S + k[b, :, t, :, None] * v[b, :, t, None, :]
            o[b, :, t] = scale * np.einsum("hd,hde->he", q[b, :, t], S)
        sT[b] = S
    return o, sT


def linear_attention_backward(q, k, v, log_decay, d_o, scale=1.0, s0=None, d_sT=None, lens=None):
    """-> (dq, dk, dv, ds0); rows behind a sequence's end are 0."""
    q, k, v, d_o = (np.asarray(x, np.float64) for x in (q, k, v, d_o))
    B, H, T, d = q.shape
    dvw = v.shape[3]
    a = decay_of(log_decay)[:, None, None]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    ds0 = np.zeros((B, H, d, dvw)) if d_sT is None else np.array(d_sT, np.float64)
    for b in range(B):
        n = T if lens is None else int(np.clip(lens[b], 0, T))
        S = np.zeros((H, d, dvw)) if s0 is None else np.asarray(s0, np.float64)[b]
        for t in range(n):
            S = a * S + k[b, :, t, :, None] * v[b, :, t, None, :]
            dq[b, :, t] = scale * np.einsum("hde,he->hd", S, d_o[b, :, t])
        D = ds0[b]
        for t in range(n - 1, -1, -1):
            D = D + scale * q[b, :, t, :, None] * d_o[b, :, t, None, :]
            dk[b, :, t] = np.einsum("hde,he->hd", D, v[b, :, t])
            dv[b, :, t] = np.einsum("hde,hd->he", D, k[b, :, t])
            D = a * D
        ds0[b] = D
    return dq, dk, dv, ds0
