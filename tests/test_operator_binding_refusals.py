"""What the binding of the operators around the memory refuses, each call by the message of its own check:
without that check the call would end elsewhere (here, where there are CPU tensors, with the refusal
of those, which the last test shows every sound call to reach)."""
import re

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from sparse_weight_memory_chunk_b200 import build, fwpkm
    build.build()
    return fwpkm


F32, BF16, I32, I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64


def z(*s, dt=F32):
    return torch.zeros(*s, dtype=dt)


IDX, TABLE, D_OUT, BAG, W = z(3, dt=I32), z(4, 8), z(3, 8), z(3, 2, dt=I32), z(3, 2)

LOOKUP = [
    (dict(idx=z(3)), "idx must be int32 or int64"),
    (dict(idx=z(6, dt=I32)[::2]), "idx must be contiguous"),
    (dict(table=z(4)), "table must be [rows][width]"),
    (dict(table=z(8, 4).t()), "table must be [rows][width], its rows contiguous"),
    (dict(table=z(4, 8, dt=torch.float16)), "table must be float32 or bfloat16"),
    (dict(idx=BAG, w=z(2, 3)), "w must be a contiguous torch.float32 tensor of shape (3, 2)"),
    (dict(idx=BAG, w=z(3, 2, dt=BF16)), "w must be a contiguous torch.float32"),
    (dict(idx=z(1, dt=I32)[0], w=z(1)[0]), "with w the last axis of idx is the bag"),
    (dict(out=z(3, 7)), "out must be a contiguous torch.float32 tensor of shape (3, 8)"),
    (dict(out=z(3, 8, dt=BF16)), "out must be a contiguous torch.float32"),
    (dict(out=z(3, 16)[:, :8]), "out must be a contiguous"),
]


def refused(call, message):
    with pytest.raises(ValueError, match=re.escape(message)):
        call()


@pytest.mark.parametrize("i", range(len(LOOKUP)))
def test_lookup(lib, i):
    over, message = LOOKUP[i]
    kw = dict(table=TABLE, idx=IDX)
    kw.update(over)
    refused(lambda: lib.lookup(**kw), message)


BACKWARD = [
    (dict(idx=z(3)), "idx must be int32 or int64"),
    (dict(table=z(4, 8, dt=torch.float16)), "table must be float32 or bfloat16"),
    (dict(d_out=z(2, 8)), "d_out must be a contiguous"),
    (dict(d_out=z(3, 8, dt=BF16)), "d_out must be a contiguous"),
    (dict(d_out=None), "d_out is needed"),
    (dict(accumulate=True), "accumulate needs the d_table"),
    (dict(d_table=z(5, 8)), "d_table must have the table's shape"),
    (dict(d_table=z(8, 4).t()), "d_table must have the table's shape and device, its rows contiguous"),
    (dict(d_table=z(1, 8).expand(4, 8)), "d_table: the rows must not share memory"),
    (dict(d_table=z(4, 8, dt=BF16), grad_dtype=F32), "d_table is not of grad_dtype"),
    (dict(d_table=z(4, 8, dt=torch.float16)), "d_table must be float32 or bfloat16"),
    (dict(dw=z(3)), "dw needs w and need_dw"),
    (dict(idx=BAG, w=W, dw=z(3, 2), need_dw=False), "dw needs w and need_dw"),
    (dict(idx=BAG, w=W, dw=z(3, 3)), "dw must be a contiguous torch.float32 tensor of shape (3, 2)"),
    (dict(workspace=z(4096)[::2]), "lookup_backward: the workspace must be contiguous"),
]


@pytest.mark.parametrize("i", range(len(BACKWARD)))
def test_lookup_backward(lib, i):
    over, message = BACKWARD[i]
    kw = dict(table=TABLE, idx=IDX, d_out=D_OUT)
    kw.update(over)
    refused(lambda: lib.lookup_backward(**kw), message)


X, SEL = z(1, 4, 8), z(1, 4, 2, dt=I32)
BALANCE = [
    (dict(x=z(4, 8)), "x must be [groups][tokens][experts]"),
    (dict(x=z(1, 8, 4).transpose(1, 2)), "x must be [groups][tokens][experts], its rows contiguous"),
    (dict(x=z(1, 4, 8, dt=torch.float16)), "x must be float32 or bfloat16"),
    (dict(idx=z(4, 2, dt=I32)), "idx must be [groups][tokens][k]"),
    (dict(idx=z(1, 4, 2)), "idx must be a contiguous torch.int32"),
    (dict(idx=z(1, 4, 2, dt=I64)), "idx must be a contiguous torch.int32"),
    (dict(idx=z(1, 3, 2, dt=I32)), "idx must be a contiguous torch.int32 tensor of shape (1, 4, 2)"),
    (dict(mask=z(1, 4)), "mask must be bool or uint8"),
    (dict(mask=z(1, 5, dt=torch.bool)), "mask must be a contiguous torch.bool tensor of shape (1, 4)"),
    (dict(kind="even"), "kind must be one of"),
    (dict(workspace=z(1 << 16)[::2]), "balance_loss: the workspace must be contiguous"),
]


@pytest.mark.parametrize("i", range(len(BALANCE)))
def test_balance_loss(lib, i):
    over, message = BALANCE[i]
    kw = dict(x=X, idx=SEL)
    kw.update(over)
    refused(lambda: lib.balance_loss(**kw), message)


def result(lib, slope):
    r = lib.BalanceLoss()
    r.kind, r.coef, r.slope = "load", 1.0, slope
    return r


@pytest.mark.parametrize("slope,over,message", [
    (z(1, 7), {}, "result.slope must be a contiguous"), (z(1, 8), dict(mask=z(1, 4)), "mask must be bool or uint8"),
    (z(1, 8), dict(d_loss=z(2)), "d_loss must be a contiguous"), (z(1, 8), dict(dx=z(1, 4, 9)), "dx must be a contiguous"),
    (z(1, 8), dict(dx=z(1, 4, 8, dt=BF16)), "dx must be a contiguous")])
def test_balance_loss_backward(lib, slope, over, message):
    refused(lambda: lib.balance_loss_backward(X, result(lib, slope), **over), message)


QK, V, LD, S = z(2, 3, 5, 8), z(2, 3, 5, 16), z(3), z(2, 3, 8, 16)
SHARED = [
    (dict(q=z(2, 3, 8)), "q, k, v must be [B][H][T][width]"),
    (dict(k=z(2, 3, 5, 9)), "k must be a torch.float32 tensor of shape (2, 3, 5, 8)"),
    (dict(v=z(2, 3, 4, 16)), "v must be a torch.float32 tensor of shape (2, 3, 5, 16)"),
    (dict(v=z(2, 3, 5, 16, dt=BF16)), "v must be a torch.float32 tensor"),
    (dict(q=z(2, 3, 8, 5).transpose(2, 3)), "q: the rows must be contiguous"),
    (dict(v=z(2, 3, 16, 5).transpose(2, 3)), "v: the rows must be contiguous"),
    (dict(log_decay=None), "log_decay is needed"),
    (dict(log_decay=z(2)), "log_decay must be a contiguous torch.float32 tensor of shape (3,)"),
    (dict(log_decay=z(3, dt=BF16)), "log_decay must be a contiguous torch.float32"),
    (dict(lens=z(1, dt=I32)), "lens must be a contiguous torch.int32 tensor of shape (2,)"),
    (dict(lens=z(2, dt=I64)), "lens must be a contiguous torch.int32"),
]
FORWARD = SHARED + [
    (dict(s0=z(2, 3, 8, 15)), "s0 must be a contiguous torch.float32 tensor of shape (2, 3, 8, 16)"),
    (dict(sT=z(2, 3, 8, 16, dt=BF16)), "sT must be a contiguous torch.float32"),
    (dict(o=z(2, 3, 5, 8)), "o must be a torch.float32 tensor of shape (2, 3, 5, 16)"),
    (dict(o=z(2, 3, 16, 5).transpose(2, 3)), "o: the rows must be contiguous"),
    (dict(workspace=z(64)[::2]), "linear_attention: the workspace must be contiguous"),
]
GRADIENTS = SHARED + [
    (dict(s0=z(2, 3, 16, 8)), "s0 must be a contiguous"), (dict(d_sT=z(2, 3, 8, 15)), "d_sT must be a contiguous"),
    (dict(ds0=z(2, 3, 8, 15)), "ds0 must be a contiguous"), (dict(d_o=z(2, 3, 5, 8)), "d_o must be a torch.float32"),
    (dict(grads=(V, QK, V)), "dq must be a torch.float32"), (dict(grads=(QK, V, V)), "dk must be a torch.float32"),
    (dict(grads=(QK, QK, QK)), "dv must be a torch.float32"),
    (dict(workspace=z(64)[::2]), "linear_attention_backward: the workspace must be contiguous"),
]
STEP = SHARED + [
    (dict(state=None), "state is needed"), (dict(state=z(2, 3, 8, 9)), "state must be a contiguous"),
    (dict(state_out=z(2, 3, 8, 9)), "state_out must be a contiguous"), (dict(o=QK), "o must be a torch.float32"),
]


@pytest.mark.parametrize("name,more", [("linear_attention", {}), ("linear_attention_backward", dict(d_o=V)),
                                       ("linear_attention_step", dict(state=S))])
def test_linear_attention(lib, name, more):
    cases = {"linear_attention": FORWARD, "linear_attention_backward": GRADIENTS, "linear_attention_step": STEP}[name]
    for over, message in cases:
        kw = dict(q=QK, k=QK, v=V, log_decay=LD, **more)
        kw.update(over)
        refused(lambda: getattr(lib, name)(**kw), message)


def test_sound_calls_reach_the_check_of_the_device(lib):
    for call in [
        lambda: lib.lookup(TABLE, IDX), lambda: lib.lookup(TABLE, BAG, w=W, out=D_OUT), lambda: lib.lookup(z(0, 8), IDX),
        lambda: lib.lookup_backward(TABLE, IDX, D_OUT, grad_dtype=BF16),
        lambda: lib.lookup_backward(TABLE, BAG, D_OUT, w=W, dw=z(3, 2), d_table=z(4, 16)[:, 8:], accumulate=True),
        lambda: lib.balance_loss(X, SEL, mask=z(1, 4, dt=torch.bool)), lambda: lib.balance_loss(X, kind="entropy"),
        lambda: lib.balance_loss_backward(X, result(lib, z(1, 8)), d_loss=z(1), dx=z(1, 4, 8)),
        lambda: lib.linear_attention(QK, QK, V, LD, s0=S, lens=z(2, dt=I32), final_state=True),
        lambda: lib.linear_attention_backward(QK, QK, V, LD, V, s0=S, d_sT=S, grads=(z(2, 3, 5, 8), z(2, 3, 5, 8), z(2, 3, 5, 16))),
        lambda: lib.linear_attention_step(QK, QK, V, LD, S, in_place=False),
    ]:
        refused(call, "the tensors must be on a CUDA device")
