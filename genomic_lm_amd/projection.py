"""The 8-bit projections of a block, the quantisation of their operands, and rotary positions.

Wrappers of the entry points of libhyena.so of the same names (include/hyena.h
states the formulas).  Like the package's other functions they check and
marshal torch tensors and pass the current HIP stream; every step runs in the
library's kernels.

An operand is a tensor of e4m3 codes (float8_e4m3fn, or uint8 of the same bits)
with fp32 scales: activations (..., K) with a scale per row or per 128 columns, as
add_rmsnorm_fp8, quantize_fp8 and gated_linear_fp8 give them, weights (N, K) with a scale
per block of 128 x 128, as quantize_weight_fp8 gives them.
"""
from __future__ import annotations

import functools
import math

import torch

from . import _ACT_DTYPES, BF16, F32, _check, _io, _stream, lib
from .serving import _FP8, NORM_GROUP, _heads, _like, _rows, _vec

__all__ = ["linear_fp8", "gated_linear_fp8", "gated_linear_fp8_workspace_size", "quantize_fp8",
           "quantize_weight_fp8", "rotary_inv_freq", "qk_norm_rope", "ACTS"]

ACTS = {"none": 0, "gelu": 1, "gelu_tanh": 2, "silu": 3}


def _one_stride(name, t):
    """Elements between two rows of t (..., D): the leading axes must be walked by one stride."""
    if t.is_contiguous():
        return t.shape[-1]
    axes = [(n, s) for n, s in zip(t.shape[:-1], t.stride()) if n != 1]
    if ((t.stride(-1) == 1 or t.shape[-1] <= 1)
            and all(s == s2 * n2 for (_, s), (n2, s2) in zip(axes, axes[1:]))):
        return axes[-1][1] if axes else t.shape[-1]
    raise ValueError(f"{name} must have a contiguous last axis and rows at one stride")


def _operand(x, x_scale):
    """x (..., K) and its scales as the entry points take them."""
    if not (isinstance(x, torch.Tensor) and x.dtype in _FP8):
        raise TypeError("x must be a float8_e4m3fn or uint8 tensor")
    if not x.is_cuda or x.dim() < 1:
        raise ValueError("x must be on a GPU device, with at least one axis")
    if not isinstance(x_scale, torch.Tensor) or x_scale.dtype != torch.float32:
        raise TypeError("x_scale must be a float32 tensor")
    if x_scale.get_device() != x.get_device():
        raise ValueError("x_scale must be on the device of x")
    rows, K = x.shape[:-1], x.shape[-1]
    runs = (K + NORM_GROUP - 1) // NORM_GROUP
    if x_scale.shape == (*rows, runs):
        step, group = runs if x_scale.is_contiguous() else _one_stride("x_scale", x_scale), NORM_GROUP
    elif x_scale.shape == rows:
        # one scale per row: rows at one stride
        step = 1 if x_scale.is_contiguous() else _one_stride("x_scale", x_scale[..., None])
        group = 0
    else:
        raise ValueError(f"x_scale must have shape {tuple(rows)} or {(*rows, runs)}, got {tuple(x_scale.shape)}")
    T = rows[0] if len(rows) == 1 else math.prod(rows)
    return (x.data_ptr(), K if x.is_contiguous() else _one_stride("x", x), x_scale.data_ptr(), step, group), T, K, rows


def _weight(name, w, scale, K, dev, N=None):
    if not (isinstance(w, torch.Tensor) and w.dtype in _FP8):
        raise TypeError(f"{name} must be a float8_e4m3fn or uint8 tensor")
    if w.dim() != 2 or w.shape[1] != K or (N is not None and w.shape[0] != N):
        raise ValueError(f"{name} must have shape ({'N' if N is None else N}, {K}), got {tuple(w.shape)}")
    n = w.shape[0]
    sshape = ((n + NORM_GROUP - 1) // NORM_GROUP, (K + NORM_GROUP - 1) // NORM_GROUP)
    return (_vec(name, w, w.dtype, None, dev), _vec(f"{name}'s scale", scale, torch.float32, sshape, dev)), n


def _out(name, out, x, rows, N, dtype):
    """out (..., N) of a type of the activations: pointer, row stride, io and the tensor."""
    if out is None:
        if dtype not in _ACT_DTYPES:
            raise TypeError("dtype must be bfloat16 or float32")
        out = x.new_empty((*rows, N), dtype=dtype)
        return out.data_ptr(), N, F32 if dtype is torch.float32 else BF16, out
    p, s = _rows(name, out)
    if tuple(out.shape) != (*rows, N) or out.get_device() != x.get_device():
        raise ValueError(f"{name} must have shape {(*rows, N)}, on the device of x")
    return p, s, _io(out), out


def linear_fp8(x, x_scale, w, w_scale, bias=None, out=None, dtype=torch.bfloat16):
    """y = x w^T + bias of 8-bit operands: x (..., K) with x_scale (...) or (..., ceil(K / 128)),
    w (N, K) with w_scale (ceil(N / 128), ceil(K / 128)), bias (N) fp32 or None.

    Returns y (..., N) in `dtype` (bfloat16 or float32), or in out and its type.  float32: exact products,
    fp32 sums; bfloat16 in calls of more than 16 rows: products of eight columns may be cut below 2^-13 of their
    largest, up to 2^-10 of sum |x| |w|."""
    head, T, K, rows = _operand(x, x_scale)
    dev = x.get_device()
    wp, N = _weight("w", w, w_scale, K, dev)
    bp = None if bias is None else _vec("bias", bias, torch.float32, (N,), dev)
    yp, ys, io, out = _out("out", out, x, rows, N, dtype)
    _check("hyena_linear_fp8", lib().hyena_linear_fp8(*head, *wp, bp, yp, ys, T, N, K, io, _stream(x)))
    return out


@functools.lru_cache(maxsize=1024)
def gated_linear_fp8_workspace_size(T: int, I: int, K: int) -> int:
    """Bytes of workspace of gated_linear_fp8 with an e4m3 output."""
    return int(lib().hyena_gated_linear_fp8_workspace_size(T, I, K))


def gated_linear_fp8(x, x_scale, w_gate, gate_scale, w_up, up_scale, act: str = "gelu", out=None, scale=None,
                     dtype=torch.bfloat16, workspace=None):
    """h = act(x w_gate^T) * (x w_up^T), operands as in linear_fp8; act "gelu", "gelu_tanh",
    "silu" or "none".

    dtype bfloat16 or float32: returns h (..., I) (out: written instead, in its type); sums as in linear_fp8.
    dtype float8_e4m3fn: returns (q (..., I), scale (..., ceil(I / 128))), the operand of
    the next linear_fp8, written to out and scale if given; workspace: gated_linear_fp8_workspace_size
    bytes, made here if not given."""
    if act not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}")
    head, T, K, rows = _operand(x, x_scale)
    dev = x.get_device()
    gp, N = _weight("w_gate", w_gate, gate_scale, K, dev)
    up, _ = _weight("w_up", w_up, up_scale, K, dev, N)
    if dtype in _FP8:
        sshape = (*rows, (N + NORM_GROUP - 1) // NORM_GROUP)
        if out is None:                    # what is made here needs no check
            out = x.new_empty((*rows, N), dtype=dtype)
            qp = out.data_ptr()
        else:
            qp = _vec("out", out, out.dtype if getattr(out, "dtype", None) in _FP8 else dtype, (*rows, N), dev)
        if scale is None:
            scale = x.new_empty(sshape, dtype=torch.float32)
            sp = scale.data_ptr()
        else:
            sp = _vec("scale", scale, torch.float32, sshape, dev)
        wp, wn = None, 0
        if workspace is not None:
            if workspace.get_device() != dev or not workspace.is_contiguous():
                raise ValueError("workspace must be contiguous, on the device of x")
            wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        elif need := gated_linear_fp8_workspace_size(T, N, K):
            workspace = x.new_empty(need, dtype=torch.uint8)
            wp, wn = workspace.data_ptr(), need
        _check("hyena_gated_linear_fp8_quant", lib().hyena_gated_linear_fp8_quant(
            *head, *gp, *up, ACTS[act], qp, sp, T, N, K, wp, wn, _stream(x)))
        return out, scale
    if scale is not None:
        raise ValueError("scale goes with dtype float8_e4m3fn")
    hp, hs, io, out = _out("out", out, x, rows, N, dtype)
    _check("hyena_gated_linear_fp8", lib().hyena_gated_linear_fp8(
        *head, *gp, *up, ACTS[act], hp, hs, T, N, K, io, _stream(x)))
    return out


def quantize_fp8(x, group: int = 0, q=None, scale=None):
    """x (..., D) bf16 or fp32 to e4m3: x ~ q * scale, scale = max|x| / 448 per row (group 0,
    shape (...)) or per 128 columns (group 128, (..., ceil(D / 128))).

    Returns (q (..., D) float8_e4m3fn, scale fp32)."""
    xp, xs = _rows("x", x)
    if group not in (0, NORM_GROUP):
        raise ValueError(f"group must be 0 or {NORM_GROUP}")
    shape, dev = x.shape, x.get_device()
    D = shape[-1]
    sshape = shape[:-1] if group == 0 else (*shape[:-1], (D + group - 1) // group)
    if q is None:
        q = _like(x, torch.float8_e4m3fn)
        qp = q.data_ptr()
    else:
        qp = _vec("q", q, q.dtype if getattr(q, "dtype", None) in _FP8 else torch.float8_e4m3fn, shape, dev)
    if scale is None:
        scale = x.new_empty(sshape, dtype=torch.float32)
        sp = scale.data_ptr()
    else:
        sp = _vec("scale", scale, torch.float32, sshape, dev)
    T = x.numel() // D if D else math.prod(shape[:-1])
    _check("hyena_quantize_fp8", lib().hyena_quantize_fp8(xp, xs, qp, sp, group, T, D, _io(x), _stream(x)))
    return q, scale


def quantize_weight_fp8(w, q=None, scale=None):
    """w (N, K) bf16 or fp32 to e4m3 with a scale per block of 128 x 128.

    Returns (q (N, K) float8_e4m3fn, scale (ceil(N / 128), ceil(K / 128)) fp32)."""
    wp, ws = _rows("w", w)
    if w.dim() != 2:
        raise ValueError(f"w must be (N, K), got shape {tuple(w.shape)}")
    N, K = w.shape
    dev = w.get_device()
    sshape = ((N + NORM_GROUP - 1) // NORM_GROUP, (K + NORM_GROUP - 1) // NORM_GROUP)
    q = _like(w, torch.float8_e4m3fn) if q is None else q
    scale = w.new_empty(sshape, dtype=torch.float32) if scale is None else scale
    qp = _vec("q", q, q.dtype if getattr(q, "dtype", None) in _FP8 else torch.float8_e4m3fn, (N, K), dev)
    sp = _vec("scale", scale, torch.float32, sshape, dev)
    _check("hyena_quantize_weight_fp8", lib().hyena_quantize_weight_fp8(
        wp, ws, qp, sp, N, K, _io(w), _stream(w)))
    return q, scale


def rotary_inv_freq(rotary_dim: int, base: float = 10000.0, factor: float = 1.0, device="cuda"):
    """inv_freq (rotary_dim / 2) fp32: base^(-2i / rotary_dim) / factor, from 64 bits;
    factor: linear scaling of the positions (32 for a context of 262144 trained at 8192)."""
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even")
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    return (float(base) ** (-i / max(rotary_dim, 1)) / factor).float().to(device)


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=None, interleaved: bool = False,
                 q_out=None, k_out=None):
    """Queries (T, Hq, DH) and keys (T, Hk, DH), normed per head (eps given) and turned by
    position, in one pass; k may be None.

    positions (T) int32 (negative: the row is not written; q_out and k_out keep theirs, in tensors
    made here it holds no value); inv_freq (R / 2) fp32 turns the
    first R columns, pairs (i, i + R / 2), or (2i, 2i + 1) if interleaved; None: no rotation.
    q_weight, k_weight (DH) fp32 or None (1).  q_out may be q, k_out may be k.  Returns (q_out, k_out)."""
    qp = _heads("q", q)
    T, Hq, DH = q.shape
    dev = q.get_device()
    kp, Hk = (None, 0, 0), 0
    if k is not None:
        kp, Hk = _heads("k", k), k.shape[1]
        if k.shape[0] != T or k.shape[2] != DH or k.dtype != q.dtype or k.get_device() != dev:
            raise ValueError("k must match q in tokens, head dimension, dtype and device")
    elif k_out is not None:
        raise ValueError("k_out needs k")
    R = 0
    pp = fp = None
    if inv_freq is not None:
        fp = _vec("inv_freq", inv_freq, torch.float32, None, dev)
        if inv_freq.dim() != 1 or 2 * inv_freq.shape[0] > DH:
            raise ValueError("inv_freq must be (R / 2), R at most the head dimension")
        R = 2 * inv_freq.shape[0]
    if positions is not None:
        pp = _vec("positions", positions, torch.int32, (T,), dev)
    elif R:
        raise ValueError("inv_freq needs positions")
    if eps is None and (q_weight is not None or k_weight is not None):
        raise ValueError("q_weight and k_weight go with a norm: give eps")
    qw = None if q_weight is None else _vec("q_weight", q_weight, torch.float32, (DH,), dev)
    kw = None if k_weight is None else _vec("k_weight", k_weight, torch.float32, (DH,), dev)
    if q_out is None:                      # what is made here needs no check
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        qo = (q_out.data_ptr(), Hq * DH, DH)
    else:
        qo = _same("q_out", q_out, q)
    ko = (None, 0, 0)
    if k is not None:
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
            ko = (k_out.data_ptr(), Hk * DH, DH)
        else:
            ko = _same("k_out", k_out, k)
    _check("hyena_qk_norm_rope", lib().hyena_qk_norm_rope(
        *qp, *kp, pp, fp, R, int(interleaved), int(eps is not None), 0.0 if eps is None else float(eps), qw, kw,
        *qo, *ko, T, Hq, Hk, DH, _io(q), _stream(q)))
    return q_out, k_out


def _same(name, t, like):
    p = _heads(name, t)
    if t.shape != like.shape or t.dtype != like.dtype or t.get_device() != like.get_device():
        raise ValueError(f"{name} must match its input in shape, dtype and device")
    return p
