"""Python binding of the library's dense side (include/emb_dense.h): attention over event sequences
with a sliding window and sinks, the gated residual norms around a block, and AdamW.  Argument
marshalling only; the work runs in the library's HIP kernels on the caller's stream.

The functions keep the C names and argument order.  Device arguments are torch CUDA tensors on the
current device; errors raise EmbError (the library's checks) or TypeError/ValueError (the tensors').
"""
from __future__ import annotations

import ctypes as C
import struct
from operator import attrgetter
from typing import Optional

import torch

from .emb import EMB_F16, EMB_F32, _check, _stream as _emb_stream, lib as _emb_lib

EMB_BF16 = 2
ATTN_MAX_SINKS = 32
ADAMW_BLOCK = 128
GATE_NONE, GATE_VECTOR, GATE_ROWS = 0, 1, 2

_VP, _I32, _I64, _F = C.c_void_p, C.c_int32, C.c_int64, C.c_float
_D = C.c_double
_DTYPE = {torch.float32: EMB_F32, torch.float16: EMB_F16, torch.bfloat16: EMB_BF16}


class EmbAttn(C.Structure):
    _fields_ = [("dtype", _I32), ("q_heads", _I32), ("kv_heads", _I32), ("dim", _I32),
                ("window", _I32), ("sinks", _I32), ("scale", _F)]


class EmbHeads(C.Structure):
    _fields_ = [("p", _VP), ("seq", _I64), ("tok", _I64), ("head", _I64)]


# The same as bytes, which the calls take as well: a Structure costs 0.3 us more, of which a call has up to nine.
_pack_attn, _pack_heads = struct.Struct("6if").pack, struct.Struct("P3q").pack

_LIB = None
_A = _H = _VP
_SZ = C.POINTER(C.c_size_t)
_SIG = {
    "attn_window_fwd": [_A, _H, _H, _H, _VP, _I64, _I64, _H, _VP, _VP],
    "attn_window_bwd_workspace_bytes": [_A, _I64, _I64, _SZ],
    "attn_window_bwd": [_A, _H, _H, _H, _VP, _I64, _I64, _H, _VP, _H, _H, _H, _H, _VP, C.c_size_t,
                        _VP],
    "attn_window_decode_workspace_bytes": [_A, _I64, _I64, _SZ],
    "attn_window_decode": [_A, _H, _H, _H, _VP, _I64, _I64, _H, _VP, C.c_size_t, _VP],
    "norm_gate_residual_fwd": [_VP, _VP, _VP, _I32, _VP, _VP, _I64, _I32, _I32, _F, _F, _VP, _VP,
                               _VP],
    "norm_gate_residual_bwd_workspace_bytes": [_I64, _I32, _SZ],
    "norm_gate_residual_bwd": [_VP, _VP, _VP, _I32, _VP, _VP, _I64, _I32, _I32, _F, _F, _VP, _VP,
                               _VP, _VP, _VP, _VP, _VP, _VP, C.c_size_t, _VP],
    "adamw_state_elems": [_VP, _I32, C.POINTER(_I64)],
    "adamw_step": [_I32, _VP, _VP, _VP, _I32, _VP, _I32, _VP, _VP, _I64, _I64, _D, _D, _D, _D, _VP,
                   _VP, _VP],
    "adamw_step_q8": [_I32, _VP, _VP, _VP, _I32, _VP, _I32, _VP, _VP, _VP, _VP, _I64, _I64, _D, _D,
                      _D, _D, _VP, _VP, C.c_uint64, _VP],
    "adamw_q8_values": [_VP, _VP, _I64, _VP, _I32, _VP],
}


def exported_symbols():
    """Names include/emb_dense.h declares (used by the load test)."""
    return list(_SIG)


def lib() -> C.CDLL:
    """The HIP library with this module's signatures set."""
    global _LIB
    if _LIB is None:
        L = _emb_lib()
        for name, args in _SIG.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = C.c_int
        _LIB = L
    return _LIB


# the current stream's handle without the Stream object around it, which costs 3 us, and the device's
# number without a look at whether there is a device, which a CUDA tensor has answered
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
# The device that a call runs on is asked for once, where one of its tensors is on some GPU; each has to be there.
_NONE = -2


def _stream(dev: int, stream):
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _emb_stream(stream)


def _ptr(dev: int, t, name: str, dtype=None, shape=None, optional: bool = False) -> Optional[int]:
    """Device pointer of a contiguous tensor of this type and shape."""
    if t is None:
        if optional:
            return None
        raise TypeError(f"{name}: expected a tensor")
    if t.get_device() != dev or not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous CUDA tensor of the current device, got one on {t.device} "
                        f"with strides {t.stride()}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _ws(dev: int, ws):
    """Pointer and size of a workspace (None where none is needed)."""
    return (None, 0) if ws is None else (_ptr(dev, ws, "workspace"), ws.numel() * ws.element_size())


# ------------------------------------------------------------------ attention
def _heads(dev: int, t, name: str, dtype, shape) -> bytes:
    """EmbHeads of [tokens, heads, dim], or [sequences, tokens, heads, dim] of a cache: any strides
    but the last, which is 1."""
    if t.dtype is not dtype or t.get_device() != dev:
        raise TypeError(f"{name}: expected a CUDA tensor of {dtype} on the current device, got {t.dtype} on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1 and t.numel() > 0:
        raise ValueError(f"{name}: the last dimension's stride must be 1")
    if 1 in shape:
        # the strides of dimensions of one element are never used: 0 passes the library's check of them
        st = [s if n > 1 else 0 for s, n in zip(st, shape)]
    if len(st) == 3:
        return _pack_heads(t.data_ptr(), 0, st[0], st[1])
    return _pack_heads(t.data_ptr(), st[0], st[1], st[2])


def _attn(dtype, shape, kv_heads: int, window: int, sinks: int, scale: float) -> bytes:
    if dtype is not torch.float16 and dtype is not torch.bfloat16:
        raise TypeError(f"q: expected float16 or bfloat16, got {dtype}")
    try:
        # no window past the longest sequence differs from one of 2^31 - 1
        return _pack_attn(_DTYPE[dtype], shape[1], kv_heads, shape[2], min(int(window), 2**31 - 1),
                          int(sinks), float(scale))
    except struct.error:
        raise ValueError("window, sinks: a value that 32 bits do not hold") from None


def _shapes(q, k):
    """q's, and that of keys and values."""
    shape = q.shape
    if len(shape) != 3 or k.dim() != 3:
        raise ValueError("q, k: expected [tokens, heads, dim]")
    return shape, (shape[0], k.shape[1], shape[2])


def _offsets(dev: int, offsets):
    p = _ptr(dev, offsets, "offsets", torch.int32)
    n = offsets.numel()
    if offsets.dim() != 1 or n < 1:
        raise ValueError("offsets: expected one dimension of n_seq + 1 elements")
    return p, n - 1


def attn_window_fwd(q, k, v, offsets, window: int, sinks: int, scale: float, out, lse=None,
                    stream=None):
    """out [tokens, q_heads, dim] and lse [q_heads, tokens] (fp32, optional) of q [tokens, q_heads,
    dim] and k, v [tokens, kv_heads, dim]; sequence s holds tokens offsets[s] to offsets[s + 1] - 1."""
    t, (qs, kv) = q.dtype, _shapes(q, k)
    a = _attn(t, qs, kv[1], window, sinks, scale)
    dev = _device() if q.is_cuda else _NONE
    off, n_seq = _offsets(dev, offsets)
    _check(lib().attn_window_fwd(
        a, _heads(dev, q, "q", t, qs), _heads(dev, k, "k", t, kv), _heads(dev, v, "v", t, kv), off, n_seq, qs[0],
        _heads(dev, out, "out", t, qs),
        _ptr(dev, lse, "lse", torch.float32, (qs[1], qs[0]), optional=True),
        _stream(dev, stream)))


def attn_window_bwd_workspace_bytes(n_tok: int, n_seq: int, q_heads: int, kv_heads: int, dim: int,
                                    sinks: int) -> int:
    a, n = _attn(torch.float16, (n_tok, q_heads, dim), kv_heads, 1, sinks, 1.0), C.c_size_t()
    _check(lib().attn_window_bwd_workspace_bytes(a, n_seq, n_tok, C.byref(n)))
    return n.value


def attn_window_bwd(q, k, v, offsets, window: int, sinks: int, scale: float, out, lse, dout, dq,
                    dk, dv, ws, stream=None):
    """dq, dk and dv from the forward's inputs and results and the gradient of out."""
    t, (qs, kv) = q.dtype, _shapes(q, k)
    a = _attn(t, qs, kv[1], window, sinks, scale)
    dev = _device() if q.is_cuda else _NONE
    off, n_seq = _offsets(dev, offsets)
    wp, wb = _ws(dev, ws)
    _check(lib().attn_window_bwd(
        a, _heads(dev, q, "q", t, qs), _heads(dev, k, "k", t, kv), _heads(dev, v, "v", t, kv), off, n_seq, qs[0],
        _heads(dev, out, "out", t, qs),
        _ptr(dev, lse, "lse", torch.float32, (qs[1], qs[0])),
        _heads(dev, dout, "dout", t, qs), _heads(dev, dq, "dq", t, qs),
        _heads(dev, dk, "dk", t, kv), _heads(dev, dv, "dv", t, kv), wp, wb,
        _stream(dev, stream)))


def attn_window_decode_workspace_bytes(n_seq: int, capacity: int, q_heads: int, kv_heads: int,
                                       dim: int, window: int, sinks: int) -> int:
    a, n = _attn(torch.float16, (n_seq, q_heads, dim), kv_heads, window, sinks, 1.0), C.c_size_t()
    _check(lib().attn_window_decode_workspace_bytes(a, n_seq, capacity, C.byref(n)))
    return n.value


def attn_window_decode(q, k_cache, v_cache, lens, window: int, sinks: int, scale: float, out, ws,
                       stream=None):
    """out [n_seq, q_heads, dim] of one query per sequence, q [n_seq, q_heads, dim], against caches
    [n_seq, capacity, kv_heads, dim] that hold lens [n_seq] events, the query's own among them."""
    t, qs = q.dtype, q.shape
    if len(qs) != 3 or k_cache.dim() != 4:
        raise ValueError("expected q [sequences, heads, dim], k_cache [sequences, capacity, heads, dim]")
    _, cap, kv_heads, _ = k_cache.shape
    a = _attn(t, qs, kv_heads, window, sinks, scale)
    cache, dev = (qs[0], cap, kv_heads, qs[2]), _device() if q.is_cuda else _NONE
    wp, wb = _ws(dev, ws)
    _check(lib().attn_window_decode(
        a, _heads(dev, q, "q", t, qs), _heads(dev, k_cache, "k_cache", t, cache),
        _heads(dev, v_cache, "v_cache", t, cache), _ptr(dev, lens, "lens", torch.int32, (qs[0],)), qs[0], cap,
        _heads(dev, out, "out", t, qs), wp, wb, _stream(dev, stream)))


# ------------------------------------------------------------------ norms
def _gate_kind(gate) -> int:
    if gate is None:
        return GATE_NONE
    return GATE_VECTOR if gate.dim() == 1 else GATE_ROWS


def _rows(t):
    dtype, shape = t.dtype, t.shape
    if len(shape) != 2:
        raise ValueError("expected rows [rows, dim]")
    if dtype not in _DTYPE:
        raise TypeError(f"expected float32, float16 or bfloat16, got {dtype}")
    return dtype, shape, shape[1:]


def norm_gate_residual_fwd(x, y, gate, w_post, w_pre, alpha: float, eps: float, r, h, stream=None):
    """r = alpha x + gate * (w_post * rms(y)), h = w_pre * rms(r).  x, y, r, h [rows, dim]; gate
    [dim] or [rows, dim]; w_post, w_pre fp32 [dim].  None where a part is left out."""
    t, s, d = _rows(x)
    kind, dev = _gate_kind(gate), _device() if x.is_cuda else _NONE
    _check(lib().norm_gate_residual_fwd(
        _ptr(dev, x, "x"), _ptr(dev, y, "y", t, s, True), _ptr(dev, gate, "gate", t, d if kind == 1 else s, True),
        kind, _ptr(dev, w_post, "w_post", torch.float32, d, True),
        _ptr(dev, w_pre, "w_pre", torch.float32, d, True), s[0], s[1], _DTYPE[t], float(alpha),
        float(eps), _ptr(dev, r, "r", t, s, True), _ptr(dev, h, "h", t, s, True), _stream(dev, stream)))


def norm_gate_residual_bwd_workspace_bytes(rows: int, dim: int) -> int:
    n = C.c_size_t()
    _check(lib().norm_gate_residual_bwd_workspace_bytes(rows, dim, C.byref(n)))
    return n.value


def norm_gate_residual_bwd(r, y, gate, w_post, w_pre, alpha: float, eps: float, dr, dh, dx, dy,
                           dgate, dw_post, dw_pre, ws, stream=None):
    """Gradients of norm_gate_residual_fwd from r as stored; None for an output that is not wanted.
    dgate: fp32 [dim] for a gate vector, like the rows for a gate of rows."""
    t, s, d = _rows(r)
    kind, dev = _gate_kind(gate), _device() if r.is_cuda else _NONE
    f, wp_wb = torch.float32, _ws(dev, ws)
    _check(lib().norm_gate_residual_bwd(
        _ptr(dev, r, "r"), _ptr(dev, y, "y", t, s, True), _ptr(dev, gate, "gate", t, d if kind == 1 else s, True),
        kind, _ptr(dev, w_post, "w_post", f, d, True), _ptr(dev, w_pre, "w_pre", f, d, True), s[0], s[1],
        _DTYPE[t], float(alpha), float(eps), _ptr(dev, dr, "dr", t, s, True), _ptr(dev, dh, "dh", t, s, True),
        _ptr(dev, dx, "dx", t, s, True), _ptr(dev, dy, "dy", t, s, True),
        _ptr(dev, dgate, "dgate", f if kind == 1 else t, d if kind == 1 else s, True),
        _ptr(dev, dw_post, "dw_post", f, d, True), _ptr(dev, dw_pre, "dw_pre", f, d, True), *wp_wb,
        _stream(dev, stream)))


# ------------------------------------------------------------------ AdamW
def adamw_state_elems(weights) -> int:
    """Elements of a state array for these weight tensors."""
    out = _I64()
    _check(lib().adamw_state_elems(struct.pack(f"{len(weights)}q", *map(_numel, weights)), len(weights),
                                   C.byref(out)))
    return out.value


# looked up once: a step of a hundred small tensors is bound by what is asked of each of them
_numel, _data_ptr, _contiguous = torch.Tensor.numel, torch.Tensor.data_ptr, torch.Tensor.is_contiguous
_dtype_of, _device_of = attrgetter("dtype"), torch.Tensor.get_device


def _tensors(dev: int, ts, name: str, dtype, sizes) -> bytes:
    """Host array of the device pointers of contiguous tensors of one type and these sizes."""
    if not (list(map(_numel, ts)) == sizes and set(map(_dtype_of, ts)) <= {dtype} and
            set(map(_device_of, ts)) <= {dev} and all(map(_contiguous, ts))):
        got = [(t.dtype, tuple(t.shape), str(t.device)) for t, n in zip(ts, sizes) if t.numel() != n or
               t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous()]
        raise TypeError(f"{name}: expected contiguous CUDA tensors of {dtype} on the current device with the "
                        f"weights' sizes, got {got[0]}")
    return struct.pack(f"{len(ts)}P", *map(_data_ptr, ts))


def _adamw_args(dev: int, weights, grads, copies, weight_decay):
    sizes = list(map(_numel, weights))
    k = len(sizes)
    if len(grads) != k or (copies is not None and len(copies) != k):
        raise ValueError(f"expected {k} tensors in grads and copies")
    g_dtype = grads[0].dtype if k else torch.float32
    c_dtype = copies[0].dtype if k and copies else torch.bfloat16
    if g_dtype not in _DTYPE or c_dtype not in _DTYPE:
        raise TypeError(f"unexpected tensor dtype {g_dtype}, {c_dtype}")
    if isinstance(weight_decay, (int, float)):
        weight_decay = [weight_decay] * k
    elif len(weight_decay) != k:
        raise ValueError(f"weight_decay: expected {k} values, got {len(weight_decay)}")
    return (k, struct.pack(f"{k}q", *sizes), _tensors(dev, weights, "weights", torch.float32, sizes),
            _tensors(dev, grads, "grads", g_dtype, sizes), _DTYPE[g_dtype],
            None if copies is None else _tensors(dev, copies, "copies", c_dtype, sizes),
            _DTYPE[c_dtype]), struct.pack(f"{k}f", *weight_decay)


def _scalar(t):
    if t is not None and t.numel() != 1:
        raise ValueError(f"grad_scale: expected one element, got {t.numel()}")


def adamw_step(weights, grads, m, v, step: int, lr: float, beta1: float, beta2: float, eps: float,
               weight_decay, copies=None, grad_scale=None, stream=None):
    """One AdamW step over lists of tensors, in place.  weights fp32; grads of one type; m, v fp32
    [adamw_state_elems(weights)]; weight_decay: a number or one per tensor; copies: float16 or
    bfloat16 tensors that receive the new weights; grad_scale: fp32 device scalar."""
    dev = _device() if m.is_cuda else _NONE
    args, wd = _adamw_args(dev, weights, grads, copies, weight_decay)
    f = torch.float32
    _scalar(grad_scale)
    _check(lib().adamw_step(
        *args, _ptr(dev, m, "m", f), _ptr(dev, v, "v", f, m.shape), m.numel(), int(step), lr, beta1, beta2,
        eps, wd, _ptr(dev, grad_scale, "grad_scale", f, optional=True), _stream(dev, stream)))


def _codes(dev: int, t, name: str, n: int):
    if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError(f"{name}: expected uint8 or float8_e4m3fn, got {t.dtype}")
    return _ptr(dev, t, name, shape=(n,))


def adamw_step_q8(weights, grads, m, m_exp, v, v_exp, step: int, lr: float, beta1: float,
                  beta2: float, eps: float, weight_decay, seed: int, copies=None, grad_scale=None,
                  stream=None):
    """adamw_step with states in 8 bits: m, v codes [adamw_state_elems(weights)] (uint8 or
    float8_e4m3fn), m_exp, v_exp uint8 [that / ADAMW_BLOCK], all zero at first.  `seed`: another one
    each step."""
    dev = _device() if m.is_cuda else _NONE
    args, wd = _adamw_args(dev, weights, grads, copies, weight_decay)
    _scalar(grad_scale)
    n = m.numel()
    e = (n // ADAMW_BLOCK,)
    _check(lib().adamw_step_q8(
        *args, _codes(dev, m, "m", n), _ptr(dev, m_exp, "m_exp", torch.uint8, e), _codes(dev, v, "v", n),
        _ptr(dev, v_exp, "v_exp", torch.uint8, e), n, int(step), lr, beta1, beta2, eps, wd,
        _ptr(dev, grad_scale, "grad_scale", torch.float32, optional=True), int(seed) & (2**64 - 1),
        _stream(dev, stream)))


def adamw_q8_values(codes, exp, out, stream=None):
    """The values that 8-bit state codes stand for, in bfloat16 or float32; v's are its roots."""
    n, dev = codes.numel(), _device() if codes.is_cuda else _NONE
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"out: expected bfloat16 or float32, got {out.dtype}")
    _check(lib().adamw_q8_values(
        _codes(dev, codes, "codes", n), _ptr(dev, exp, "exp", torch.uint8, (n // ADAMW_BLOCK,)), n,
        _ptr(dev, out, "out", shape=(n,)), _DTYPE[out.dtype], _stream(dev, stream)))
