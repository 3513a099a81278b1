"""What the operators around the memory refuse, on the host: every call below returns before
anything is enqueued (pointers are aligned numbers that nothing reads)."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from sparse_weight_memory_chunk_b200 import build, fwpkm
    build.build()
    return fwpkm


FAKE = C.c_void_p(1 << 20)
ODD = C.c_void_p((1 << 20) + 1)


def lookup_cfg(lib, **over):
    c = dict(rows=100, table_ld=64, out_ld=64, width=64, R=2, dtype=0, idx_dtype=0, scale=1.0)
    c.update(over)
    return C.byref(lib.LookupConfig(**c))


@pytest.mark.parametrize("over,n,want", [
    (dict(rows=0), 4, -1), (dict(width=0), 4, -1), (dict(R=0), 4, -1), (dict(table_ld=63), 4, -1),
    (dict(out_ld=63), 4, -1), (dict(dtype=2), 4, -1), (dict(idx_dtype=2), 4, -1), ({}, -1, -1),
    (dict(rows=1 << 31), 4, -2), (dict(width=(1 << 20) + 1, table_ld=1 << 21, out_ld=1 << 21), 4, -2),
    (dict(R=1025), 4, -2), ({}, 1 << 31, -2)])
def test_lookup_config_is_checked(lib, over, n, want):
    so = lib.lib()
    out = C.c_size_t(0)
    cfg = lookup_cfg(lib, **over)
    assert so.fwpkm_lookup(cfg, FAKE, FAKE, None, n, FAKE, None) == want
    assert so.fwpkm_lookup_backward_workspace_size(cfg, n, C.byref(out)) == want
    assert so.fwpkm_lookup_backward(cfg, FAKE, FAKE, None, FAKE, n, FAKE, 1 << 21, 0, 0, None, FAKE, 1 << 40,
                                    None) == want


def test_lookup_arguments_are_checked(lib):
    so = lib.lib()
    cfg = lookup_cfg(lib)
    ws = C.c_size_t(0)
    assert so.fwpkm_lookup_backward_workspace_size(cfg, 4, None) == -1
    assert so.fwpkm_lookup_backward_workspace_size(cfg, 4, C.byref(ws)) == 0 and ws.value > 0
    assert so.fwpkm_lookup(cfg, FAKE, FAKE, None, 0, FAKE, None) == 0  # no tokens
    for bad in [(None, FAKE, None, FAKE), (FAKE, None, None, FAKE), (FAKE, FAKE, None, None),
                (ODD, FAKE, None, FAKE), (FAKE, ODD, None, FAKE), (FAKE, FAKE, ODD, FAKE), (FAKE, FAKE, None, ODD)]:
        assert so.fwpkm_lookup(cfg, bad[0], bad[1], bad[2], 4, bad[3], None) == -1

    def back(table=FAKE, idx=FAKE, w=None, d_out=FAKE, n=4, d_table=FAKE, ld=64, gdt=0, acc=0, dw=None, work=FAKE,
             nb=ws.value):
        return so.fwpkm_lookup_backward(cfg, table, idx, w, d_out, n, d_table, ld, gdt, acc, dw, work, nb, None)

    assert back(idx=None) == -1 and back(d_out=None) == -1 and back(d_out=ODD) == -1
    assert back(ld=63) == -1 and back(gdt=2) == -1 and back(d_table=ODD) == -1
    assert back(work=None) == -1 and back(work=C.c_void_p((1 << 20) + 128)) == -1
    assert back(nb=ws.value - 1) == lib.ERR_WORKSPACE
    assert back(table=None, dw=FAKE) == -1 and back(dw=ODD) == -1 and back(w=ODD) == -1
    assert back(n=0, d_table=None, work=None, nb=0) == 0  # nothing to do


def balance_cfg(lib, **over):
    c = dict(tokens=16, ld=8, group_stride=128, groups=2, experts=8, k=2, dtype=0, kind=0, coef=1.0)
    c.update(over)
    return C.byref(lib.BalanceConfig(**c))


@pytest.mark.parametrize("over,want", [
    (dict(groups=0), -1), (dict(tokens=-1), -1), (dict(experts=0), -1), (dict(k=-1), -1), (dict(ld=7), -1),
    (dict(group_stride=-1), -1), (dict(dtype=5), -1), (dict(kind=2), -1), (dict(experts=4097, ld=5000), -2),
    (dict(groups=65536), -2), (dict(k=4097), -2), (dict(tokens=1 << 31, k=4), -2)])
def test_balance_config_is_checked(lib, over, want):
    so = lib.lib()
    out = C.c_size_t(0)
    cfg = balance_cfg(lib, **over)
    assert so.fwpkm_balance_workspace_size(cfg, C.byref(out)) == want
    assert so.fwpkm_balance_loss(cfg, FAKE, FAKE, None, FAKE, 1 << 40, FAKE, FAKE, FAKE, FAKE, None) == want
    assert so.fwpkm_balance_loss_backward(cfg, FAKE, None, FAKE, None, FAKE, None) == want


def test_balance_arguments_are_checked(lib):
    so = lib.lib()
    cfg = balance_cfg(lib)
    ws = C.c_size_t(0)
    assert so.fwpkm_balance_workspace_size(cfg, None) == -1
    assert so.fwpkm_balance_workspace_size(cfg, C.byref(ws)) == 0

    def fwd(cfg=cfg, x=FAKE, idx=FAKE, mask=None, work=FAKE, nb=ws.value, loss=FAKE, counts=FAKE, usage=FAKE,
            slope=FAKE):
        return so.fwpkm_balance_loss(cfg, x, idx, mask, work, nb, loss, counts, usage, slope, None)

    assert fwd(x=None) == -1 and fwd(x=ODD) == -1 and fwd(loss=None) == -1 and fwd(usage=None) == -1
    assert fwd(slope=None) == -1 and fwd(counts=ODD) == -1 and fwd(idx=ODD) == -1
    assert fwd(idx=None) == -1                                     # the load needs selections
    assert fwd(cfg=balance_cfg(lib, k=0)) == -1                    # idx without k
    assert fwd(work=None) == -1 and fwd(work=C.c_void_p((1 << 20) + 64)) == -1
    assert fwd(nb=ws.value - 1) == lib.ERR_WORKSPACE
    bwd = lambda x=FAKE, s=FAKE, g=None, dx=FAKE: so.fwpkm_balance_loss_backward(cfg, x, None, s, g, dx, None)  # noqa: E731
    assert bwd(x=None) == -1 and bwd(s=None) == -1 and bwd(dx=None) == -1 and bwd(dx=ODD) == -1 and bwd(g=ODD) == -1
    assert so.fwpkm_balance_loss_backward(balance_cfg(lib, tokens=0), None, None, None, None, None, None) == 0


def la_cfg(lib, **over):
    c = dict(B=2, H=3, d=64, d_v=32, dtype=0, scale=0.5)
    c.update(over)
    return C.byref(lib.LinattnConfig(**c))


@pytest.mark.parametrize("over,T,want", [
    (dict(B=0), 8, -1), (dict(H=0), 8, -1), (dict(d=0), 8, -1), (dict(d_v=0), 8, -1), (dict(dtype=7), 8, -1),
    (dict(scale=0.0), 8, -1), (dict(scale=float("nan")), 8, -1), ({}, -1, -1), (dict(d=257), 8, -2),
    (dict(d_v=257), 8, -2), (dict(B=1 << 20, H=32), 8, -2), ({}, (1 << 28) + 1, -2)])
def test_linear_attention_config_is_checked(lib, over, T, want):
    so = lib.lib()
    out = C.c_size_t(0)
    cfg = la_cfg(lib, **over)
    x = C.byref(lib.Heads(1 << 20, 1 << 16, 1 << 12, 64))
    for back in (0, 1):
        assert so.fwpkm_linear_attention_workspace_size(cfg, T, back, C.byref(out)) == want
    assert so.fwpkm_linear_attention(cfg, x, x, x, T, FAKE, None, None, x, None, FAKE, 1 << 40, None) == want
    assert so.fwpkm_linear_attention_step(cfg, x, x, x, T, FAKE, None, FAKE, x, FAKE, None) == want
    assert so.fwpkm_linear_attention_backward(cfg, x, x, x, T, FAKE, None, None, x, None, x, x, x, None, FAKE, 1 << 40,
                                              None) == want


def test_linear_attention_arguments_are_checked(lib):
    so = lib.lib()
    cfg = la_cfg(lib)
    hd = lambda p=1 << 20, sb=1 << 16, sh=1 << 12, st=64: C.byref(lib.Heads(p, sb, sh, st))  # noqa: E731
    ok = hd()
    T = 4096  # few heads and a long prompt: the tokens are split, so a workspace is needed
    ws = C.c_size_t(0)
    assert so.fwpkm_linear_attention_workspace_size(cfg, T, 0, None) == -1
    assert so.fwpkm_linear_attention_workspace_size(cfg, T, 0, C.byref(ws)) == 0 and ws.value > 0

    def fwd(q=ok, k=ok, v=ok, T=T, ld=FAKE, lens=None, s0=None, o=ok, sT=None, work=FAKE, nb=ws.value):
        return so.fwpkm_linear_attention(cfg, q, k, v, T, ld, lens, s0, o, sT, work, nb, None)

    for bad in (None, hd(p=None), hd(p=(1 << 20) + 2), hd(sb=-1), hd(sh=-1), hd(st=-1)):
        assert fwd(q=bad) == -1 and fwd(k=bad) == -1 and fwd(v=bad) == -1 and fwd(o=bad) == -1
    # output rows that share memory
    assert fwd(o=hd(st=31)) == -1 and fwd(o=hd(sh=0)) == -1 and fwd(o=hd(sb=0)) == -1
    assert fwd(ld=None) == -1 and fwd(ld=ODD) == -1 and fwd(lens=ODD) == -1 and fwd(s0=ODD) == -1 and fwd(sT=ODD) == -1
    assert fwd(work=None) == -1 and fwd(work=C.c_void_p((1 << 20) + 8)) == -1
    assert fwd(nb=ws.value - 1) == lib.ERR_WORKSPACE
    assert so.fwpkm_linear_attention(cfg, None, None, None, 0, FAKE, None, None, None, None, None, 0, None) == 0

    step = lambda s=FAKE, so_=FAKE, o=ok: so.fwpkm_linear_attention_step(  # noqa: E731
        cfg, ok, ok, ok, 1, FAKE, None, s, o, so_, None)
    assert step(s=None) == -1 and step(so_=None) == -1 and step(s=ODD) == -1 and step(so_=ODD) == -1
    assert step(o=None) == -1 and step(o=hd(st=31)) == -1

    assert so.fwpkm_linear_attention_workspace_size(cfg, T, 1, C.byref(ws)) == 0
    bwd = lambda dq=ok, dk=ok, dv=ok, do=ok, ds0=None, nb=ws.value: so.fwpkm_linear_attention_backward(  # noqa: E731
        cfg, ok, ok, ok, T, FAKE, None, None, do, None, dq, dk, dv, ds0, FAKE, nb, None)
    for bad in (None, hd(st=31), hd(sh=0)):
        assert bwd(dq=bad) == -1 and bwd(dk=bad) == -1 and bwd(dv=bad) == -1
    assert bwd(do=None) == -1 and bwd(ds0=ODD) == -1 and bwd(nb=ws.value - 1) == lib.ERR_WORKSPACE


def test_binding_checks(lib):
    f32, i32 = torch.float32, torch.int32
    z = lambda *s, dt=f32: torch.zeros(*s, dtype=dt)  # noqa: E731
    for call in [
        lambda: lib.lookup(z(4, 8), z(3)),                                            # float indices
        lambda: lib.lookup(z(4), z(3, dt=i32)),                                       # not a table
        lambda: lib.lookup(z(8, 4).t(), z(3, dt=i32)),                                # rows not contiguous
        lambda: lib.lookup(z(4, 8, dt=torch.float16), z(3, dt=i32)),
        lambda: lib.lookup(z(4, 8), z(3, 2, dt=i32), w=z(2, 3)),
        lambda: lib.lookup(z(4, 8), z(3, dt=i32), out=z(3, 7)),
        lambda: lib.lookup(z(4, 8), z(3, dt=i32)),                                    # no GPU tensors
        lambda: lib.lookup_backward(z(4, 8), z(3, dt=i32), z(2, 8)),
        lambda: lib.lookup_backward(z(4, 8), z(3, dt=i32), z(3, 8), accumulate=True),
        lambda: lib.lookup_backward(z(4, 8), z(3, dt=i32), z(3, 8), d_table=z(5, 8)),
        lambda: lib.lookup_backward(z(4, 8), z(3, dt=i32), z(3, 8), d_table=z(1, 8).expand(4, 8)),
        lambda: lib.lookup_backward(z(4, 8), z(3, dt=i32), z(3, 8), dw=z(3)),
        lambda: lib.balance_loss(z(4, 8)),
        lambda: lib.balance_loss(z(1, 4, 8), z(1, 4, 2)),
        lambda: lib.balance_loss(z(1, 4, 8), z(1, 3, 2, dt=i32)),
        lambda: lib.balance_loss(z(1, 4, 8), z(1, 4, 2, dt=i32), mask=z(1, 4)),
        lambda: lib.balance_loss(z(1, 4, 8), z(1, 4, 2, dt=i32), kind="even"),
        lambda: lib.linear_attention(z(1, 2, 3, 8), z(1, 2, 3, 9), z(1, 2, 3, 8), z(2)),
        lambda: lib.linear_attention(z(1, 2, 3, 8), z(1, 2, 3, 8), z(1, 2, 3, 8, dt=torch.bfloat16), z(2)),
        lambda: lib.linear_attention(z(1, 2, 3, 8), z(1, 2, 3, 8), z(1, 2, 3, 8), z(3)),
        lambda: lib.linear_attention(z(1, 2, 3, 8), z(1, 2, 3, 8), z(1, 2, 3, 8), None),
        lambda: lib.linear_attention(z(1, 2, 8, 3).transpose(2, 3), z(1, 2, 3, 8), z(1, 2, 3, 8), z(2)),
        lambda: lib.linear_attention(z(1, 2, 3, 8), z(1, 2, 3, 8), z(1, 2, 3, 8), z(2), s0=z(1, 2, 8, 7)),
        lambda: lib.linear_attention(z(1, 2, 3, 8), z(1, 2, 3, 8), z(1, 2, 3, 8), z(2), lens=z(1)),
        lambda: lib.linear_attention_step(z(1, 2, 1, 8), z(1, 2, 1, 8), z(1, 2, 1, 8), z(2), z(1, 2, 8, 9)),
    ]:
        with pytest.raises(ValueError):
            call()
