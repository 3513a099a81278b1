"""Thin ctypes binding of ``libfwpkm.so`` (declared in ``include/fwpkm.h``).

Argument marshalling only: every step of the FwPKM hot path runs in the library's
CUDA kernels.  Functions keep the C names without the ``fwpkm_`` prefix; device
buffers are passed as torch tensors (their ``data_ptr``) and streams as
``torch.cuda.Stream`` (default: the current stream).  A non-OK status raises
``FwpkmError``.  If the library is missing, loading raises instead of falling back
to anything else.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfwpkm.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_STATE, ERR_BAD_SLOT = \
    0, -1, -2, -3, -4, -5, -6, -7
F32, BF16 = 0, 1
I32, I64 = 0, 1
BALANCE_KIND = {"load": 0, "entropy": 1}
KEY_UPDATE, TARGET_NORM, LOOKAHEAD, GATE_WEIGHT = 1, 2, 4, 8
DEFAULT_FLAGS = TARGET_NORM | LOOKAHEAD | GATE_WEIGHT
KIND = {"gather": 1, "write": 2, "score": 3, "cartesian": 4, "sort": 5, "address": 6, "other": 7, "topk": 8,
        "prep": 9, "pbar": 10, "wbuild": 11, "fused": 12, "value_loop": 13, "all": 100}
KIND_NAME = {v: k for k, v in KIND.items()}


class FwpkmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class Config(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("d", ctypes.c_int), ("d_v", ctypes.c_int), ("k", ctypes.c_int),
                ("chunk", ctypes.c_int), ("num_mem", ctypes.c_int), ("qv_dtype", ctypes.c_int),
                ("eps_idw", ctypes.c_float), ("eps_norm", ctypes.c_float), ("lr_key", ctypes.c_float),
                ("flags", ctypes.c_uint), ("v_heads", ctypes.c_int)]


def make_config(n, d, d_v, k, chunk, num_mem, bf16, eps_idw=1e-3, eps_norm=1e-5, lr_key=1.0,
                key_update=False, target_norm=True, lookahead=True, gate_weight=True, v_heads=1) -> Config:
    flags = ((KEY_UPDATE if key_update else 0) | (TARGET_NORM if target_norm else 0)
             | (LOOKAHEAD if lookahead else 0) | (GATE_WEIGHT if gate_weight else 0))
    return Config(n, d, d_v, k, chunk, num_mem, BF16 if bf16 else F32, eps_idw, eps_norm, lr_key, flags, v_heads)


_lib = None
_P = ctypes.c_void_p


class LayerConfig(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int), ("d", ctypes.c_int), ("d_v", ctypes.c_int), ("max_rows", ctypes.c_int),
                ("eps_rms", ctypes.c_float), ("qv_dtype", ctypes.c_int)]


class LayerParams(ctypes.Structure):
    _fields_ = [("W_q", _P), ("gamma_q", _P), ("b_q", _P),
                ("W_v", _P), ("gamma_v", _P), ("b_v", _P),
                ("w_g", _P), ("gamma_g", _P), ("b_g", ctypes.c_float),
                ("W_o", _P), ("gamma_o", _P), ("b_o", _P)]


class LookupConfig(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("table_ld", ctypes.c_longlong), ("out_ld", ctypes.c_longlong),
                ("width", ctypes.c_int), ("R", ctypes.c_int), ("dtype", ctypes.c_int), ("idx_dtype", ctypes.c_int),
                ("scale", ctypes.c_float)]


class BalanceConfig(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_longlong), ("ld", ctypes.c_longlong), ("group_stride", ctypes.c_longlong),
                ("groups", ctypes.c_int), ("experts", ctypes.c_int), ("k", ctypes.c_int), ("dtype", ctypes.c_int),
                ("kind", ctypes.c_int), ("coef", ctypes.c_float)]


class Heads(ctypes.Structure):
    _fields_ = [("p", _P), ("sb", ctypes.c_longlong), ("sh", ctypes.c_longlong), ("st", ctypes.c_longlong)]


class LinattnConfig(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("d", ctypes.c_int), ("d_v", ctypes.c_int),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float)]


def lib():
    """Load libfwpkm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python sparse_weight_memory_chunk_b200/build.py`")
        L = ctypes.CDLL(LIB_PATH)
        C = ctypes.POINTER(Config)
        sig = {
            "fwpkm_workspace_size": ([C, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
            "fwpkm_init_state": ([C, _P, _P, _P, ctypes.c_int, _P, ctypes.c_size_t, ctypes.POINTER(_P)],
                                 ctypes.c_int),
            "fwpkm_forward_chunk": ([_P, _P, _P, _P, ctypes.c_int, ctypes.c_int, _P, _P, _P, _P], ctypes.c_int),
            "fwpkm_write_chunk": ([_P, _P, _P], ctypes.c_int),
            "fwpkm_run_sequence": ([_P, _P, _P, _P, ctypes.c_int, ctypes.c_int, _P, _P], ctypes.c_int),
            "fwpkm_read_backward": ([C, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int, _P, _P, _P, _P],
                                    ctypes.c_int),
            "fwpkm_run_sequence_host_scratch_size": ([C, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
                                                     ctypes.c_int),
            "fwpkm_run_sequence_host": ([_P, _P, _P, _P, ctypes.c_int, ctypes.c_int, _P, _P, ctypes.c_size_t, _P],
                                        ctypes.c_int),
            "fwpkm_last_addressing": ([_P, ctypes.c_int, _P, _P, _P], ctypes.c_int),
            "fwpkm_chunk_step_noalloc": ([C, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int, ctypes.c_int, _P, _P],
                                         ctypes.c_int),
            "fwpkm_stream_tokens": ([_P, _P, _P, _P, ctypes.c_int, ctypes.c_int, _P, _P], ctypes.c_int),
            "fwpkm_stream_flush": ([_P, _P], ctypes.c_int),
            "fwpkm_stream_pending": ([_P, ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
            "fwpkm_sync": ([_P, _P], ctypes.c_int),
            "fwpkm_destroy_state": ([_P], None),
            "fwpkm_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "fwpkm_launch_count": ([], ctypes.c_uint64),
            "fwpkm_profile_kernel": ([_P, ctypes.c_int], ctypes.c_int),
            "fwpkm_kernel_time": ([_P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int)],
                                  ctypes.c_int),
            "fwpkm_kernel_timeline": ([_P, ctypes.c_int, _P, _P, _P, ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
            "fwpkm_layer_workspace_size": ([ctypes.POINTER(LayerConfig), ctypes.POINTER(ctypes.c_size_t)],
                                           ctypes.c_int),
            "fwpkm_layer_init": ([ctypes.POINTER(LayerConfig), _P, ctypes.c_size_t, ctypes.POINTER(_P)],
                                 ctypes.c_int),
            "fwpkm_layer_set_params": ([_P, ctypes.POINTER(LayerParams), _P], ctypes.c_int),
            "fwpkm_layer_in": ([_P, _P, ctypes.c_int, _P, _P, _P, _P], ctypes.c_int),
            "fwpkm_layer_out": ([_P, _P, ctypes.c_int, _P, _P], ctypes.c_int),
            "fwpkm_layer_sync": ([_P, _P], ctypes.c_int),
            "fwpkm_layer_destroy": ([_P], None),
            "fwpkm_run_layer_scratch_size": ([C, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
            "fwpkm_run_layer": ([_P, _P, _P, ctypes.c_int, ctypes.c_int, _P, ctypes.c_size_t, _P, _P], ctypes.c_int),
            "fwpkm_test_stall_waits": ([ctypes.c_int], None),
            "fwpkm_metrics_workspace_size": ([ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                              ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
            "fwpkm_addressing_metrics": ([_P, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                          _P, ctypes.c_size_t, _P, _P, _P], ctypes.c_int),
        }
        LC, BC, AC, HP = (ctypes.POINTER(t) for t in (LookupConfig, BalanceConfig, LinattnConfig, Heads))
        ll, sz, i32 = ctypes.c_longlong, ctypes.c_size_t, ctypes.c_int
        sig.update({
            "fwpkm_lookup": ([LC, _P, _P, _P, ll, _P, _P], i32),
            "fwpkm_lookup_backward_workspace_size": ([LC, ll, ctypes.POINTER(sz)], i32),
            "fwpkm_lookup_backward": ([LC, _P, _P, _P, _P, ll, _P, ll, i32, i32, _P, _P, sz, _P], i32),
            "fwpkm_balance_workspace_size": ([BC, ctypes.POINTER(sz)], i32),
            "fwpkm_balance_loss": ([BC, _P, _P, _P, _P, sz, _P, _P, _P, _P, _P], i32),
            "fwpkm_balance_loss_backward": ([BC, _P, _P, _P, _P, _P, _P], i32),
            "fwpkm_linear_attention_workspace_size": ([AC, i32, i32, ctypes.POINTER(sz)], i32),
            "fwpkm_linear_attention": ([AC, HP, HP, HP, i32, _P, _P, _P, HP, _P, _P, sz, _P], i32),
            "fwpkm_linear_attention_backward": ([AC, HP, HP, HP, i32, _P, _P, _P, HP, _P, HP, HP, HP, _P, _P, sz, _P],
                                                i32),
            "fwpkm_linear_attention_sync": ([_P], i32),
            "fwpkm_linear_attention_step": ([AC, HP, HP, HP, i32, _P, _P, _P, HP, _P, _P], i32),
        })
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != OK:
        raise FwpkmError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def status_string(status: int) -> str:
    return lib().fwpkm_status_string(status).decode()


def launch_count() -> int:
    return int(lib().fwpkm_launch_count())


def test_stall_waits(n_launches: int):
    """Test hook: the next n tensor-core launches wait once on a barrier that nothing
    completes, so their bounded wait runs out (no fault; see include/fwpkm.h)."""
    lib().fwpkm_test_stall_waits(int(n_launches))


def run_layer_scratch_size(cfg: Config, T: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().fwpkm_run_layer_scratch_size(ctypes.byref(cfg), T, ctypes.byref(out)), "run_layer_scratch_size")
    return out.value


def read_backward(cfg: Config, K1, K2, V, q, v, g, idx, d_o, dq, dv, dg, len_=None, seq_stride=None, stream=None):
    """fwpkm_read_backward: dq, dv, dg (fp32, the q, v, g layouts) from d_o for the tokens
    whose slots `idx` ([M][len][k]) the forward read with the state K1, K2, V."""
    len_ = idx.shape[1] if len_ is None else len_
    seq_stride = q.shape[1] if seq_stride is None else seq_stride
    _check(lib().fwpkm_read_backward(ctypes.byref(cfg), _ptr(K1), _ptr(K2), _ptr(V), _ptr(q), _ptr(v), _ptr(g),
                                     _ptr(idx), _ptr(d_o), len_, seq_stride, _ptr(dq), _ptr(dv), _ptr(dg),
                                     _stream(stream)), "read_backward")


def run_sequence_host_scratch_size(cfg: Config, T: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().fwpkm_run_sequence_host_scratch_size(ctypes.byref(cfg), T, ctypes.byref(out)),
           "run_sequence_host_scratch_size")
    return out.value


def run_layer_parts(cfg: Config, T: int, scratch):
    """Views of the q, v, g, o that fwpkm_run_layer leaves in `scratch` (a uint8 tensor)."""
    import torch
    M, d, dv = cfg.num_mem, cfg.d, cfg.d_v
    es = 2 if cfg.qv_dtype == BF16 else 4
    qdt = torch.bfloat16 if cfg.qv_dtype == BF16 else torch.float32
    al = lambda x: (x + 255) // 256 * 256  # noqa: E731
    sizes = [es * M * T * d, es * M * T * dv, 4 * M * T, 4 * M * T * dv]
    offs, o = [], 0
    for b in sizes:
        offs.append(o)
        o = al(o + b)
    q = scratch[offs[0]:offs[0] + sizes[0]].view(qdt).view(M, T, d)
    v = scratch[offs[1]:offs[1] + sizes[1]].view(qdt).view(M, T, dv)
    g = scratch[offs[2]:offs[2] + sizes[2]].view(torch.float32).view(M, T)
    ob = scratch[offs[3]:offs[3] + sizes[3]].view(torch.float32).view(M, T, dv)
    return q, v, g, ob


def workspace_size(cfg: Config, max_T: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().fwpkm_workspace_size(ctypes.byref(cfg), max_T, ctypes.byref(out)), "workspace_size")
    return out.value


def chunk_step_noalloc(cfg: Config, K1, K2, V, q, v, g, o, c_len, seq_stride=None, v_next=None,
                       stream=None):
    """One chunk step (read + write + key step) with no workspace and no allocation."""
    seq_stride = c_len if seq_stride is None else seq_stride
    _check(lib().fwpkm_chunk_step_noalloc(ctypes.byref(cfg), _ptr(K1), _ptr(K2), _ptr(V), _ptr(q), _ptr(v),
                                          _ptr(g), _ptr(v_next), c_len, seq_stride, _ptr(o), _stream(stream)),
           "chunk_step_noalloc")


def metrics_workspace_size(num_mem: int, T: int, N: int, window: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().fwpkm_metrics_workspace_size(num_mem, T, N, window, ctypes.byref(out)), "metrics_workspace_size")
    return out.value


def addressing_metrics(idx, N: int, window: int = 32768, workspace=None, stream=None, out=None):
    """Addressing metrics of selections idx (int32 CUDA tensor [M][T][k]) per window of tokens.

    Returns (metrics fp64 [M][W][3]: coverage, collision rate, KLD; counts int64 [M][W][4]:
    rows accessed, accesses, competitive accesses, invalid entries), W = ceil(T / window);
    `out` = (metrics, counts) tensors of those shapes to fill instead of new ones.
    """
    import torch
    M, T, k = idx.shape
    W = (T + window - 1) // window
    if out is None:
        met = torch.zeros(M, W, 3, dtype=torch.float64, device=idx.device)
        cnt = torch.zeros(M, W, 4, dtype=torch.int64, device=idx.device)
    else:
        met, cnt = out
        if tuple(met.shape) != (M, W, 3) or tuple(cnt.shape) != (M, W, 4) or met.dtype != torch.float64 \
                or cnt.dtype != torch.int64 or not (met.is_contiguous() and cnt.is_contiguous()):
            raise ValueError("out must be contiguous fp64 [M][W][3] and int64 [M][W][4] tensors")
    if workspace is None:
        workspace = torch.empty(metrics_workspace_size(M, T, N, window), dtype=torch.uint8, device=idx.device)
    _check(lib().fwpkm_addressing_metrics(_ptr(idx), M, T, k, N, window, _ptr(workspace), workspace.numel(),
                                          _ptr(met), _ptr(cnt), _stream(stream)), "addressing_metrics")
    return met, cnt


# ---- operators around the memory -------------------------------------------------------
# Torch tensors in, torch tensors out; every call only enqueues on `stream` (default: the
# current stream of the tensors' device; for another one the caller keeps the inputs alive and
# waits, as for any kernel there).  Single tokens and small batches take about as long
# on the host as on the GPU, so the checks below stay with what costs little.

def _need(ok, what):
    if not ok:
        raise ValueError(what)


_DTYPES = None


def _dtype(t, what):
    global _DTYPES
    if _DTYPES is None:
        import torch
        _DTYPES = {torch.float32: F32, torch.bfloat16: BF16}
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be float32 or bfloat16, not {t.dtype}")
    return code


def _call(t, stream, where, fn, *args):
    """fn(*args, stream) with the device of `t` current; a non-OK status raises."""
    import torch
    _need(t.is_cuda, "the tensors must be on a CUDA device")
    dev = t.get_device()
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev)
    else:
        _need(stream.device_index == dev, "the stream is another device's than the tensors")
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status != OK:
        raise FwpkmError(status, where)


def _side(t, like, dtype, shape, what):
    """The pointer of a contiguous tensor of this type, shape and `like`'s device (None passes)."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {like.device}")
    return t.data_ptr()


def _empty(stream, shape, dtype, like, zero=False):
    """A new tensor on `like`'s device.  With a stream given it comes from that stream's memory:
    the current one's may still be in use, or be handed out again, while the call runs there."""
    import torch
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=like.device)


def _zero(stream, *tensors):
    """The outputs of sums without a term (a table without rows, a bag without entries)."""
    import torch
    for t in tensors:
        _need(t.is_cuda, "the tensors must be on a CUDA device")
        with torch.cuda.stream(stream):
            t.zero_()


def _scratch(workspace, nbytes, like, stream, what):
    """(tensor, pointer, bytes) of a workspace: the caller's, or a new one of nbytes."""
    if workspace is None:
        if not nbytes:
            return None, None, 0
        import torch
        workspace = _empty(stream, nbytes, torch.uint8, like)
        return workspace, workspace.data_ptr(), nbytes
    if workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError(f"{what}: the workspace must be contiguous, on {like.device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _bytes(fn, where, *args):
    out = ctypes.c_size_t(0)
    status = fn(*args, ctypes.byref(out))
    if status != OK:
        raise FwpkmError(status, where)
    return out.value


def _row_stride(t, axis, what):
    """Elements between the rows of t along `axis`, rows being its last axis."""
    width, ld = t.shape[-1], t.stride(axis)
    if ld >= width:
        return ld
    if t.shape[axis] > 1:
        raise ValueError(f"{what}: the rows must not share memory (expand, unfold)")
    return width  # (of a single row any stride will do)


def _lookup_config(table, idx, w, scale):
    import torch
    _need(table.dim() == 2 and (table.stride(1) == 1 or table.shape[1] <= 1),
          "table must be [rows][width], its rows contiguous")
    i64 = idx.dtype == torch.int64
    _need(i64 or idx.dtype == torch.int32, "idx must be int32 or int64")
    _need(idx.device == table.device and idx.is_contiguous(), "idx must be contiguous, on the table's device")
    rows, width = table.shape
    R, lead = 1, idx.shape
    if w is not None:
        _need(idx.dim() >= 1, "with w the last axis of idx is the bag")
        R, lead = idx.shape[-1], idx.shape[:-1]
        _side(w, table, torch.float32, idx.shape, "w")
    n = idx.numel() // R if R and rows else None  # (None: no sum has a term)
    return LookupConfig(rows, _row_stride(table, 0, "table"), width, width, R, _dtype(table, "table"),
                        I64 if i64 else I32, scale), lead + (width,), n


def lookup(table, idx, w=None, scale=1.0, out=None, stream=None):
    """fwpkm_lookup: scale * table[idx], shape idx.shape + [width]; with weights w (fp32, the
    shape of idx) the last axis of idx is summed: scale * sum_r w[.., r] table[idx[.., r]].
    Indices outside the table read zeros, and so do all in a table without rows and bags without
    entries."""
    cfg, shape, n = _lookup_config(table, idx, w, scale)
    if out is None:
        out = _empty(stream, shape, table.dtype, table)
    else:
        _side(out, table, table.dtype, shape, "out")
    if n is None:
        _zero(stream, out)
        return out
    _call(table, stream, "lookup", lib().fwpkm_lookup, ctypes.byref(cfg), table.data_ptr(), idx.data_ptr(),
          None if w is None else w.data_ptr(), n, out.data_ptr())
    return out


def lookup_backward_workspace_size(table, idx, w=None) -> int:
    cfg, _, n = _lookup_config(table, idx, w, 1.0)
    if n is None:
        return 0
    return _bytes(lib().fwpkm_lookup_backward_workspace_size, "lookup_backward_workspace_size", ctypes.byref(cfg), n)


def lookup_backward(table, idx, d_out, w=None, scale=1.0, d_table=None, accumulate=False, grad_dtype=None, dw=None,
                    need_dw=True, workspace=None, stream=None):
    """fwpkm_lookup_backward: (d_table, dw) of lookup(table, idx, w, scale) from d_out.
    d_table [rows][width] (grad_dtype, default the table's type) is written whole, or with
    accumulate added to the rows that were read (then it must be given); dw (fp32, the shape
    of idx) is None without w or with need_dw=False."""
    import torch
    cfg, shape, n = _lookup_config(table, idx, w, scale)
    p_out = _side(d_out, table, table.dtype, shape, "d_out")
    _need(d_out is not None, "d_out is needed")
    _need(not accumulate or d_table is not None, "accumulate needs the d_table to add to")
    if d_table is None:
        d_table = _empty(stream, table.shape, grad_dtype or table.dtype, table)
    _need(d_table.shape == table.shape and d_table.device == table.device
          and (d_table.stride(1) == 1 or table.shape[1] <= 1),
          "d_table must have the table's shape and device, its rows contiguous")
    grad_ld = _row_stride(d_table, 0, "d_table")
    _need(grad_dtype is None or d_table.dtype == grad_dtype, "d_table is not of grad_dtype")
    if w is None or not need_dw:
        _need(dw is None, "dw needs w and need_dw")
    elif dw is None:
        dw = _empty(stream, idx.shape, torch.float32, table)
    else:
        _side(dw, table, torch.float32, idx.shape, "dw")
    if n is None:
        _zero(stream, *(t for t in (None if accumulate else d_table, dw) if t is not None))
        return d_table, dw
    L, c = lib(), ctypes.byref(cfg)
    keep, pw, nw = _scratch(workspace, 0 if workspace is not None else
                            _bytes(L.fwpkm_lookup_backward_workspace_size, "lookup_backward", c, n), table,
                            stream, "lookup_backward")
    _call(table, stream, "lookup_backward", L.fwpkm_lookup_backward, c, table.data_ptr(), idx.data_ptr(),
          None if w is None else w.data_ptr(), p_out, n, d_table.data_ptr(), grad_ld,
          _dtype(d_table, "d_table"), int(accumulate), None if dw is None else dw.data_ptr(), pw, nw)
    return d_table, dw


class BalanceLoss:
    """What balance_loss returns: loss [G], counts [G][E] (None without idx), usage [G][E], and
    the slope [G][E] that balance_loss_backward needs."""
    __slots__ = ("loss", "counts", "usage", "slope", "kind", "coef")


def _balance_config(x, idx, mask, kind, coef):
    import torch
    _need(x.dim() == 3 and (x.stride(2) == 1 or x.shape[2] <= 1),
          "x must be [groups][tokens][experts], its rows contiguous")
    if kind not in BALANCE_KIND:
        raise ValueError(f"kind must be one of {sorted(BALANCE_KIND)}")
    G, T, E = x.shape
    k = 0
    if idx is not None:
        _need(idx.dim() == 3, "idx must be [groups][tokens][k]")
        k = idx.shape[2]
        _side(idx, x, torch.int32, (G, T, k), "idx")
    if mask is not None:
        _need(mask.dtype in (torch.bool, torch.uint8), "mask must be bool or uint8")
        _side(mask, x, mask.dtype, (G, T), "mask")
    return BalanceConfig(T, _row_stride(x, 1, "x"), x.stride(0) if G > 1 else 0, G, E, k, _dtype(x, "x"),
                         BALANCE_KIND[kind], coef)


def balance_loss(x, idx=None, mask=None, kind="load", coef=1.0, workspace=None, stream=None) -> BalanceLoss:
    """fwpkm_balance_loss of router logits x [groups][tokens][experts] with the selections idx
    [groups][tokens][k] int32 (kind "load"; optional for "entropy") and a mask
    [groups][tokens] of the tokens that count."""
    import torch
    cfg = _balance_config(x, idx, mask, kind, coef)
    G, E = cfg.groups, cfg.experts
    r = BalanceLoss()
    r.kind, r.coef = kind, coef
    r.loss = _empty(stream, G, torch.float32, x)
    r.usage, r.slope = _empty(stream, (G, E), torch.float32, x), _empty(stream, (G, E), torch.float32, x)
    r.counts = None if idx is None else _empty(stream, (G, E), torch.int32, x)
    if not G:
        return r
    L, c = lib(), ctypes.byref(cfg)
    keep, pw, nw = _scratch(workspace, 0 if workspace is not None else
                            _bytes(L.fwpkm_balance_workspace_size, "balance_loss", c), x, stream, "balance_loss")
    _call(x, stream, "balance_loss", L.fwpkm_balance_loss, c, x.data_ptr(), None if idx is None else idx.data_ptr(),
          None if mask is None else mask.data_ptr(), pw, nw, r.loss.data_ptr(),
          None if idx is None else r.counts.data_ptr(), r.usage.data_ptr(), r.slope.data_ptr())
    return r


def balance_loss_backward(x, result: BalanceLoss, mask=None, d_loss=None, dx=None, stream=None):
    """fwpkm_balance_loss_backward: dx [groups][tokens][experts] of balance_loss's result for
    the same x and mask, from d_loss [groups] (None: ones)."""
    import torch
    cfg = _balance_config(x, None, mask, result.kind, result.coef)
    G, T, E = x.shape
    ps = _side(result.slope, x, torch.float32, (G, E), "result.slope")
    pl = _side(d_loss, x, torch.float32, (G,), "d_loss")
    if dx is None:
        dx = _empty(stream, (G, T, E), x.dtype, x)
    else:
        _side(dx, x, x.dtype, (G, T, E), "dx")
    if not G:
        return dx
    _call(x, stream, "balance_loss_backward", lib().fwpkm_balance_loss_backward, ctypes.byref(cfg), x.data_ptr(),
          None if mask is None else mask.data_ptr(), ps, pl, dx.data_ptr())
    return dx


def _heads(t, dtype, device, shape, what):
    """A [B][H][T][w] tensor of any strides with contiguous rows."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{what} must be a {dtype} tensor of shape {tuple(shape)} on {device}")
    sb, sh, st, se = t.stride()
    if se != 1 and shape[3] > 1:
        raise ValueError(f"{what}: the rows must be contiguous")
    return ctypes.byref(Heads(t.data_ptr(), sb, sh, st))


def _linattn_args(q, k, v, log_decay, scale, lens):
    import torch
    _need(q.dim() == 4 and v.dim() == 4, "q, k, v must be [B][H][T][width]")
    _need(log_decay is not None, "log_decay is needed")
    qs, dt, dev = q.shape, q.dtype, q.device
    B, H, T, d = qs
    dv = v.shape[3]
    like = dt, dev
    hq, hk, hv = _heads(q, dt, dev, qs, "q"), _heads(k, dt, dev, qs, "k"), _heads(v, dt, dev, (B, H, T, dv), "v")
    ld = _side(log_decay, q, torch.float32, (H,), "log_decay")
    ln = None if lens is None else _side(lens, q, torch.int32, (B,), "lens")
    return ctypes.byref(LinattnConfig(B, H, d, dv, _dtype(q, "q"), scale)), hq, hk, hv, ld, ln, B, H, T, d, dv, like


def _rows_like(t, B, H, T, w, stream, lens):
    """A new [B][H][T][w] tensor in the memory order [B][T][H][w] of a projection's output; with
    lengths it holds zeros, which stay behind a sequence's end."""
    return _empty(stream, (B, T, H, w), t.dtype, t, lens is not None).transpose(1, 2)


def linear_attention_workspace_size(q, v, backward=False) -> int:
    cfg = LinattnConfig(q.shape[0], q.shape[1], q.shape[3], v.shape[3], _dtype(q, "q"), 1.0)
    if not cfg.B * cfg.H:
        return 0
    return _bytes(lib().fwpkm_linear_attention_workspace_size, "linear_attention_workspace_size", ctypes.byref(cfg),
                  q.shape[2], int(backward))


def linear_attention(q, k, v, log_decay, scale=1.0, s0=None, lens=None, o=None, sT=None, final_state=False,
                     workspace=None, stream=None):
    """fwpkm_linear_attention: (o, sT) of q, k [B][H][T][d], v [B][H][T][d_v] (any strides with
    contiguous rows), log_decay [H] fp32, start states s0 [B][H][d][d_v] fp32 and lengths lens
    [B] int32.  sT is None unless given or asked for with final_state.  Rows of o behind a
    sequence's end are left as they were (zeros in a new o)."""
    import torch
    c, hq, hk, hv, ld, ln, B, H, T, d, dv, like = _linattn_args(q, k, v, log_decay, scale, lens)
    if o is None:
        o = _rows_like(v, B, H, T, dv, stream, lens)
    ho = _heads(o, *like, (B, H, T, dv), "o")
    if sT is None and final_state:
        sT = _empty(stream, (B, H, d, dv), torch.float32, q)
    p0 = _side(s0, q, torch.float32, (B, H, d, dv), "s0")
    pT = _side(sT, q, torch.float32, (B, H, d, dv), "sT")
    if not B * H:
        return o, sT
    L = lib()
    keep, pw, nw = _scratch(workspace, 0 if workspace is not None else
                            _bytes(L.fwpkm_linear_attention_workspace_size, "linear_attention", c, T, 0), q, stream,
                            "linear_attention")
    _call(q, stream, "linear_attention", L.fwpkm_linear_attention, c, hq, hk, hv, T, ld, ln, p0, ho, pT, pw, nw)
    return o, sT


def linear_attention_backward(q, k, v, log_decay, d_o, scale=1.0, s0=None, d_sT=None, lens=None, grads=None, ds0=None,
                              state_grad=True, workspace=None, stream=None):
    """fwpkm_linear_attention_backward: (dq, dk, dv, ds0) of linear_attention from d_o and the
    final state's gradient d_sT (None: zero).  `grads`: (dq, dk, dv) to fill; ds0 is None with
    state_grad=False.  Rows behind a sequence's end are left as they were (zeros in new gradients)."""
    import torch
    c, hq, hk, hv, ld, ln, B, H, T, d, dv, like = _linattn_args(q, k, v, log_decay, scale, lens)
    ho = _heads(d_o, *like, (B, H, T, dv), "d_o")
    if grads is None:
        grads = tuple(_rows_like(q, B, H, T, w, stream, lens) for w in (d, d, dv))
    hg = [_heads(t, *like, (B, H, T, w), n) for t, w, n in zip(grads, (d, d, dv), ("dq", "dk", "dv"))]
    if ds0 is None and state_grad:
        ds0 = _empty(stream, (B, H, d, dv), torch.float32, q)
    p0 = _side(s0, q, torch.float32, (B, H, d, dv), "s0")
    pT = _side(d_sT, q, torch.float32, (B, H, d, dv), "d_sT")
    pd = _side(ds0, q, torch.float32, (B, H, d, dv), "ds0")
    if not B * H:
        return (*grads, ds0)
    L = lib()
    keep, pw, nw = _scratch(workspace, 0 if workspace is not None else
                            _bytes(L.fwpkm_linear_attention_workspace_size, "linear_attention_backward", c, T, 1), q, stream,
                            "linear_attention_backward")
    _call(q, stream, "linear_attention_backward", L.fwpkm_linear_attention_backward, c, hq, hk, hv, T, ld, ln, p0, ho,
          pT, *hg, pd, pw, nw)
    return (*grads, ds0)


def linear_attention_step(q, k, v, log_decay, state, scale=1.0, lens=None, o=None, state_out=None, in_place=True,
                          stream=None):
    """fwpkm_linear_attention_step: (o, new state) of a few new tokens [B][H][n][..] from the
    states [B][H][d][d_v], which are updated in place unless state_out is given or
    in_place=False (then a new tensor is).  Rows of o behind a sequence's end are left as they
    were (zeros in a new o)."""
    import torch
    c, hq, hk, hv, ld, ln, B, H, T, d, dv, like = _linattn_args(q, k, v, log_decay, scale, lens)
    if o is None:
        o = _rows_like(v, B, H, T, dv, stream, lens)
    ho = _heads(o, *like, (B, H, T, dv), "o")
    _need(state is not None, "state is needed")
    ps = _side(state, q, torch.float32, (B, H, d, dv), "state")
    if state_out is None:
        state_out = state if in_place else _empty(stream, state.shape, torch.float32, q)
    po = _side(state_out, q, torch.float32, (B, H, d, dv), "state_out")
    if not B * H:
        return o, state_out
    _call(q, stream, "linear_attention_step", lib().fwpkm_linear_attention_step, c, hq, hk, hv, T, ld, ln, ps, ho, po)
    return o, state_out


def linear_attention_sync(device=None, stream=None):
    """fwpkm_linear_attention_sync: wait for the stream and raise what linear-attention kernels
    on the device have latched (a wait that timed out: what its heads should have given is NaN)."""
    import torch
    with torch.cuda.device(device if stream is None else stream.device):
        handle = (torch.cuda.current_stream() if stream is None else stream).cuda_stream
        _check(lib().fwpkm_linear_attention_sync(handle), "linear_attention_sync")


class State:
    """A handle from ``fwpkm_init_state``; keeps the caller's tensors alive."""

    def __init__(self, cfg: Config, K1, K2, V, max_T: int, workspace=None):
        import torch
        self.cfg = cfg
        self.max_T = max_T
        nbytes = workspace_size(cfg, max_T)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=V.device)
        for t in (K1, K2, V):
            assert t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()
        self.K1, self.K2, self.V, self.workspace = K1, K2, V, workspace
        h = _P()
        _check(lib().fwpkm_init_state(ctypes.byref(cfg), _ptr(K1), _ptr(K2), _ptr(V), max_T,
                                      _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      ctypes.byref(h)), "init_state")
        self.handle = h
        self._pending = None

    def forward_chunk(self, q, v, g, o, c_len, seq_stride=None, idx_out=None, w_out=None, stream=None):
        seq_stride = c_len if seq_stride is None else seq_stride
        self._pending = (q, v, g)
        _check(lib().fwpkm_forward_chunk(self.handle, _ptr(q), _ptr(v), _ptr(g), c_len, seq_stride, _ptr(o),
                                         _ptr(idx_out), _ptr(w_out), _stream(stream)), "forward_chunk")

    def write_chunk(self, v_next=None, stream=None):
        _check(lib().fwpkm_write_chunk(self.handle, _ptr(v_next), _stream(stream)), "write_chunk")
        self._pending = None

    def run_sequence(self, q, v, g, o, T=None, n_iter=1, stream=None):
        T = q.shape[1] if T is None else T
        _check(lib().fwpkm_run_sequence(self.handle, _ptr(q), _ptr(v), _ptr(g), T, n_iter, _ptr(o),
                                        _stream(stream)), "run_sequence")

    def run_sequence_host(self, q, v, g, o, T=None, n_iter=1, scratch=None, stream=None):
        """run_sequence on page-locked HOST tensors q, v, g, o (copies overlap the compute);
        `scratch`: a device uint8 tensor of run_sequence_host_scratch_size bytes (made here if
        None).  Returns the scratch so that repeated calls can reuse it."""
        import torch
        T = q.shape[1] if T is None else T
        if scratch is None:
            scratch = torch.empty(run_sequence_host_scratch_size(self.cfg, T), dtype=torch.uint8, device="cuda")
        _check(lib().fwpkm_run_sequence_host(self.handle, _ptr(q), _ptr(v), _ptr(g), T, n_iter, _ptr(o),
                                             _ptr(scratch), scratch.numel(), _stream(stream)), "run_sequence_host")
        return scratch

    def stream_tokens(self, q, v, g, o, n_tok=None, seq_stride=None, stream=None):
        """Read n_tok new tokens of every memory ([M][seq_stride][..] rows); writes o for them."""
        n_tok = q.shape[1] if n_tok is None else n_tok
        seq_stride = q.shape[1] if seq_stride is None else seq_stride
        _check(lib().fwpkm_stream_tokens(self.handle, _ptr(q), _ptr(v), _ptr(g), n_tok, seq_stride, _ptr(o),
                                         _stream(stream)), "stream_tokens")

    def stream_flush(self, stream=None):
        """Write the pending tokens of a token-at-a-time sequence (no lookahead for the last)."""
        _check(lib().fwpkm_stream_flush(self.handle, _stream(stream)), "stream_flush")

    def stream_pending(self) -> int:
        """Tokens read by stream_tokens and not yet written (host-side count)."""
        n = ctypes.c_int(0)
        _check(lib().fwpkm_stream_pending(self.handle, ctypes.byref(n)), "stream_pending")
        return n.value

    def last_addressing(self, T, idx_out=None, w_out=None, stream=None):
        _check(lib().fwpkm_last_addressing(self.handle, T, _ptr(idx_out), _ptr(w_out), _stream(stream)),
               "last_addressing")

    def sync(self, stream=None):
        _check(lib().fwpkm_sync(self.handle, _stream(stream)), "sync")

    def profile_kernel(self, kind):
        kind = KIND.get(kind, kind) if isinstance(kind, str) else kind
        _check(lib().fwpkm_profile_kernel(self.handle, int(kind)), "profile_kernel")

    def kernel_timeline(self, max_launches=4096):
        """[(kind name, start ms, end ms)] of the launches timed in the last call."""
        import numpy as np
        kinds = np.zeros(max_launches, dtype=np.int32)
        t0 = np.zeros(max_launches, dtype=np.float32)
        t1 = np.zeros(max_launches, dtype=np.float32)
        n = ctypes.c_int(0)
        _check(lib().fwpkm_kernel_timeline(self.handle, max_launches, kinds.ctypes.data_as(_P), t0.ctypes.data_as(_P),
                                           t1.ctypes.data_as(_P), ctypes.byref(n)), "kernel_timeline")
        m = min(n.value, max_launches)
        return [(KIND_NAME.get(int(kinds[i]), str(int(kinds[i]))), float(t0[i]), float(t1[i])) for i in range(m)]

    def kernel_time(self):
        ms = ctypes.c_double(0.0)
        n = ctypes.c_int(0)
        _check(lib().fwpkm_kernel_time(self.handle, ctypes.byref(ms), ctypes.byref(n)), "kernel_time")
        return ms.value, n.value

    def destroy(self):
        if getattr(self, "handle", None):
            lib().fwpkm_destroy_state(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


class Layer:
    """A handle from ``fwpkm_layer_init``: the slow-weight projections (method steps 1
    and 3).  Weights are bf16 tensors [out][in]; norm weights and biases fp32 (None:
    ones / zeros)."""

    def __init__(self, d_model, d, d_v, max_rows, eps_rms=1e-6, qv_bf16=False, device="cuda"):
        import torch
        self.cfg = LayerConfig(d_model, d, d_v, max_rows, eps_rms, BF16 if qv_bf16 else F32)
        out = ctypes.c_size_t(0)
        _check(lib().fwpkm_layer_workspace_size(ctypes.byref(self.cfg), ctypes.byref(out)), "layer_workspace_size")
        self.workspace = torch.empty(out.value, dtype=torch.uint8, device=device)
        h = _P()
        _check(lib().fwpkm_layer_init(ctypes.byref(self.cfg), _ptr(self.workspace), out.value, ctypes.byref(h)),
               "layer_init")
        self.handle = h

    def set_params(self, W_q, W_v, w_g, W_o, gamma_q=None, gamma_v=None, gamma_g=None, gamma_o=None,
                   b_q=None, b_v=None, b_g=0.0, b_o=None, stream=None):
        p = LayerParams(_ptr(W_q), _ptr(gamma_q), _ptr(b_q), _ptr(W_v), _ptr(gamma_v), _ptr(b_v),
                        _ptr(w_g), _ptr(gamma_g), float(b_g), _ptr(W_o), _ptr(gamma_o), _ptr(b_o))
        _check(lib().fwpkm_layer_set_params(self.handle, ctypes.byref(p), _stream(stream)), "layer_set_params")

    def project_in(self, h, q, v, g, rows=None, stream=None):
        rows = h.shape[0] if rows is None else rows
        _check(lib().fwpkm_layer_in(self.handle, _ptr(h), rows, _ptr(q), _ptr(v), _ptr(g), _stream(stream)),
               "layer_in")

    def project_out(self, o, o_out, rows=None, stream=None):
        rows = o.shape[0] if rows is None else rows
        _check(lib().fwpkm_layer_out(self.handle, _ptr(o), rows, _ptr(o_out), _stream(stream)), "layer_out")

    def sync(self, stream=None):
        _check(lib().fwpkm_layer_sync(self.handle, _stream(stream)), "layer_sync")

    def run_layer(self, state, h, o_out, T=None, n_iter=1, scratch=None, stream=None):
        """fwpkm_run_layer: h [M][T][d_model] bf16 -> o_out [M][T][d_model] bf16 through the
        projections and the memory `state`.  Returns the scratch tensor (see run_layer_parts)."""
        import torch
        T = h.shape[1] if T is None else T
        if scratch is None:
            scratch = torch.empty(run_layer_scratch_size(state.cfg, T), dtype=torch.uint8, device=h.device)
        _check(lib().fwpkm_run_layer(self.handle, state.handle, _ptr(h), T, n_iter, _ptr(scratch), scratch.numel(),
                                     _ptr(o_out), _stream(stream)), "run_layer")
        return scratch

    def destroy(self):
        if getattr(self, "handle", None):
            lib().fwpkm_layer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass
