"""The serving step around the Hyena mixers: norm, page map, 8-bit K/V cache, attention.

Wrappers of the entry points of libhyena.so of the same names (include/hyena.h
states the formulas).  Like the package's other functions they check and
marshal torch tensors and pass the current HIP stream; every step runs in the
library's kernels.

The cache of an attention layer is four tensors:
    k_cache (pages, heads, page_size, DH)   float8_e4m3fn (or uint8)
    v_cache (pages, heads, DH, page_size)   float8_e4m3fn (or uint8)
    k_scale, v_scale (pages, heads)         float32, powers of two
new_cache() allocates them.  A step of a model maps its new tokens to slots once
(page_map), then appends and attends in every layer.
"""
from __future__ import annotations

import functools
import math

import torch

from . import _ACT_DTYPES, _check, _io, _stream, lib

__all__ = ["add_rmsnorm", "add_rmsnorm_fp8", "page_map", "kv_append_fp8", "attn_paged_fp8",
           "attn_paged_workspace_size", "new_cache", "NORM_GROUP"]

NORM_GROUP = 128
_FP8 = (torch.float8_e4m3fn, torch.uint8)


def _rows(name, t, like=None):
    """t (..., D) as (pointer, row stride): the leading axes must be walked by one stride."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in _ACT_DTYPES and t.dim() >= 1):
        if not isinstance(t, torch.Tensor) or t.dtype not in _ACT_DTYPES:
            raise TypeError(f"{name} must be a bfloat16 or float32 tensor")
        raise ValueError(f"{name} must be on a GPU device, with at least one axis")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype
                             or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must match x in shape, dtype and device")
    D = t.shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), D
    if t.dim() == 2:
        if t.stride(1) == 1 or D == 1:
            return t.data_ptr(), t.stride(0)
    elif D == 1 or t.stride(-1) == 1:
        # axes of one row have no say, such as the last token of each sequence, x[:, -1:]
        axes = [(n, s) for n, s in zip(t.shape[:-1], t.stride()) if n != 1]
        if all(s == s2 * n2 for (_, s), (n2, s2) in zip(axes, axes[1:])):
            return t.data_ptr(), axes[-1][1] if axes else D
    raise ValueError(f"{name} must have a contiguous last axis and rows at one stride")


def _vec(name, t, dtype, shape, dev):
    """A contiguous tensor of dtype, shape and device; its pointer."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev
            and (shape is None or t.shape == shape) and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {str(dtype)[6:]} tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the other arguments")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _like(x, dtype=None):
    """An uninitialised contiguous tensor of x's shape (the shortest path to one)."""
    if x.is_contiguous():
        return torch.empty_like(x, dtype=dtype)
    return torch.empty(x.shape, dtype=dtype or x.dtype, device=x.device)


def _norm_args(x, weight, residual, residual_out):
    xp, xs = _rows("x", x)
    D, dev = x.shape[-1], x.get_device()
    wp = None if weight is None else _vec("weight", weight, torch.float32, (D,), dev)
    rp = rop = None
    rs = ros = 0
    if residual is not None:
        rp, rs = _rows("residual", residual, x)
        if residual_out is None:           # what is made here needs no check
            residual_out = _like(x)
            rop, ros = residual_out.data_ptr(), D
        else:
            rop, ros = _rows("residual_out", residual_out, x)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    T = x.numel() // D if D else 0
    return (xp, xs, rp, rs, wp), (rop, ros, T, D, _io(x), _stream(x)), residual_out


def add_rmsnorm(x, weight=None, residual=None, eps: float = 1e-6, out=None, residual_out=None):
    """y = s / sqrt(mean(s^2) + eps) * weight over the last axis, s = x + residual.

    x, residual (..., D) bf16 or fp32, weight (D) fp32 or None (1).  Returns (y,
    residual_out): s rounded to x's dtype, None without a residual.  out may be
    x, residual_out may be residual or x."""
    head, tail, residual_out = _norm_args(x, weight, residual, residual_out)
    if out is None:
        out = _like(x)
        yp, ys = out.data_ptr(), x.shape[-1]
    else:
        yp, ys = _rows("out", out, x)
    _check("hyena_add_rmsnorm", lib().hyena_add_rmsnorm(*head, eps, yp, ys, *tail))
    return out, residual_out


def add_rmsnorm_fp8(x, weight=None, residual=None, eps: float = 1e-6, group: int = 0, q=None,
                    scale=None, residual_out=None):
    """add_rmsnorm with y in e4m3: y ~ q * scale, scale = max|y| / 448 per row
    (group 0, shape (...)) or per 128 columns (group 128, (..., ceil(D / 128))).

    Returns (q (..., D) float8_e4m3fn, scale fp32, residual_out)."""
    head, tail, residual_out = _norm_args(x, weight, residual, residual_out)
    if group not in (0, NORM_GROUP):
        raise ValueError(f"group must be 0 or {NORM_GROUP}")
    shape = x.shape
    sshape = shape[:-1] if group == 0 else (*shape[:-1], (shape[-1] + group - 1) // group)
    if q is None:
        q = _like(x, torch.float8_e4m3fn)
        qp = q.data_ptr()
    else:
        qp = _vec("q", q, q.dtype if getattr(q, "dtype", None) in _FP8 else torch.float8_e4m3fn, shape,
                  x.get_device())
    if scale is None:
        scale = x.new_empty(sshape, dtype=torch.float32)
        sp = scale.data_ptr()
    else:
        sp = _vec("scale", scale, torch.float32, sshape, x.get_device())
    _check("hyena_add_rmsnorm_fp8", lib().hyena_add_rmsnorm_fp8(*head, eps, qp, sp, group, *tail))
    return q, scale, residual_out


def _table(t):
    """block_table (R, max_pages) as (pointer, row stride, R, max_pages)."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32:
        raise TypeError("block_table must be an int32 tensor")
    if not t.is_cuda or t.dim() != 2:
        raise ValueError("block_table must be (R, max_pages) on a GPU device")
    R, width = t.shape
    if t.is_contiguous() or R <= 1 and (width <= 1 or t.stride(1) == 1):
        return t.data_ptr(), width, R, width
    if width > 1 and t.stride(1) != 1:
        raise ValueError("block_table must have contiguous rows")
    return t.data_ptr(), t.stride(0), R, width


def page_map(old_lens, new_lens, block_table, free_pages, free_head, page_size: int, T: int,
             cu=None, lens=None, positions=None, slots=None, status=None):
    """The tables of one step from request lengths.

    old_lens, new_lens (R) int32; block_table (R, max_pages) int32, whose entries
    of new pages are written; free_pages (F) int32 from index free_head[0] on (free_head
    (1) int32, or None: 0).  Returns cu (R + 1) int32, lens (R) int32, positions
    (T) int32, slots (T) int64 and status (2) int32: the free list's new head and
    the number of new tokens without a page."""
    tp, step, R, width = _table(block_table)
    dev = block_table.get_device()
    i32 = torch.int32
    op = _vec("old_lens", old_lens, i32, (R,), dev)
    np_ = _vec("new_lens", new_lens, i32, (R,), dev)
    fp = _vec("free_pages", free_pages, i32, None, dev)
    hp = None if free_head is None else _vec("free_head", free_head, i32, (1,), dev)
    T = int(T)
    if cu is lens is positions is slots is status is None:
        # one allocation for all outputs but the 64-bit one; what is made here needs no check
        cu, lens, positions, status = block_table.new_empty(2 * R + T + 3).split_with_sizes((R + 1, R, T, 2))
        slots = block_table.new_empty(T, dtype=torch.int64)
        cp, lp, pp, slp, stp = (t.data_ptr() for t in (cu, lens, positions, slots, status))
    else:
        new = block_table.new_empty
        cu = new(R + 1) if cu is None else cu
        lens = new(R) if lens is None else lens
        positions = new(T) if positions is None else positions
        slots = new(T, dtype=torch.int64) if slots is None else slots
        status = new(2) if status is None else status
        cp, lp = _vec("cu", cu, i32, (R + 1,), dev), _vec("lens", lens, i32, (R,), dev)
        pp, slp = _vec("positions", positions, i32, (T,), dev), _vec("slots", slots, torch.int64, (T,), dev)
        stp = _vec("status", status, i32, (2,), dev)
    _check("hyena_page_map", lib().hyena_page_map(
        op, np_, R, tp, step, width, fp, free_pages.numel(), hp, page_size, cp, lp, pp, slp, T, stp,
        _stream(block_table)))
    return cu, lens, positions, slots, status


def new_cache(num_pages: int, heads: int, page_size: int, head_dim: int, device="cuda"):
    """(k_cache, v_cache, k_scale, v_scale) of one layer, contents undefined: no
    page is read before tokens are appended to it."""
    f8 = torch.float8_e4m3fn
    return (torch.empty((num_pages, heads, page_size, head_dim), dtype=f8, device=device),
            torch.empty((num_pages, heads, head_dim, page_size), dtype=f8, device=device),
            torch.empty((num_pages, heads), device=device), torch.empty((num_pages, heads), device=device))


def _cache(k_cache, v_cache, k_scale, v_scale, H, DH, dev):
    """Pointers of a cache, its pages and their size."""
    if not (isinstance(k_cache, torch.Tensor) and k_cache.dtype in _FP8 and k_cache.dim() == 4):
        raise TypeError("k_cache must be a (pages, heads, page_size, DH) float8_e4m3fn or uint8 tensor")
    N, h, P, d = k_cache.shape
    if h != H or d != DH:
        raise ValueError(f"k_cache must have {H} heads of {DH}, got {tuple(k_cache.shape)}")
    return (_vec("k_cache", k_cache, k_cache.dtype, None, dev),
            _vec("v_cache", v_cache, k_cache.dtype, (N, H, DH, P), dev),
            _vec("k_scale", k_scale, torch.float32, (N, H), dev),
            _vec("v_scale", v_scale, torch.float32, (N, H), dev), N, P)


def _heads(name, t, like=None):
    """t (T, heads, DH) as (pointer, token stride, head stride)."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _ACT_DTYPES:
        raise TypeError(f"{name} must be a bfloat16 or float32 tensor")
    if not t.is_cuda or t.dim() != 3:
        raise ValueError(f"{name} must be (T, heads, DH) on a GPU device")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype
                             or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must match k in shape, dtype and device")
    s = t.stride()
    if s[2] != 1 and t.shape[2] > 1 and t.numel():
        raise ValueError(f"{name} must have a contiguous last axis")
    return t.data_ptr(), s[0], s[1]


def kv_append_fp8(k, v, slots, k_cache, v_cache, k_scale, v_scale) -> None:
    """k, v (T, H, DH) into the cache at slots (T) int64, in place: block scales
    grow as needed, and a block's older codes move with them."""
    kp = _heads("k", k)
    vp = _heads("v", v, k)
    T, H, DH = k.shape
    dev = k.get_device()
    sp = _vec("slots", slots, torch.int64, (T,), dev)
    kc, vc, ks, vs, N, P = _cache(k_cache, v_cache, k_scale, v_scale, H, DH, dev)
    _check("hyena_kv_append_fp8", lib().hyena_kv_append_fp8(
        *kp, *vp, sp, kc, vc, ks, vs, N, P, T, H, DH, _io(k), _stream(k)))


@functools.lru_cache(maxsize=1024)
def attn_paged_workspace_size(R: int, T: int, max_q: int, max_pages: int, page_size: int, Hq: int,
                              Hkv: int, DH: int) -> int:
    return int(lib().hyena_attn_paged_workspace_size(R, T, max_q, max_pages, page_size, Hq, Hkv, DH))


def attn_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, cu, max_q: int,
                   scale=None, out=None, workspace=None):
    """Causal attention of q (T, Hq, DH) over the paged cache, ragged requests:
    request r has query tokens cu[r] .. cu[r + 1] - 1 and lens[r] cached tokens,
    the last of which are the queries' own; cu may run past T (the queries there are
    left out), and rows of out past cu[R] are not written.  max_q: no request has
    more queries.  scale defaults to 1 / sqrt(DH).  Returns out (T, Hq, DH)."""
    qp, qt, qh = _heads("q", q)
    T, Hq, DH = q.shape
    dev = q.get_device()
    Hkv = k_cache.shape[1] if isinstance(k_cache, torch.Tensor) and k_cache.dim() == 4 else 0
    kc, vc, ks, vs, N, P = _cache(k_cache, v_cache, k_scale, v_scale, Hkv, DH, dev)
    tp, step, R, width = _table(block_table)
    if block_table.get_device() != dev:
        raise ValueError("block_table must be on the device of q")
    lp = _vec("lens", lens, torch.int32, (R,), dev)
    cp = _vec("cu", cu, torch.int32, (R + 1,), dev)
    if out is None:
        out = _like(q)
        op = out.data_ptr()
    else:
        op = _vec("out", out, q.dtype, q.shape, dev)
    max_q = int(max_q)
    if workspace is None:
        need = attn_paged_workspace_size(R, T, max_q, width, P, Hq, Hkv, DH)
        if need:
            workspace = q.new_empty(need, dtype=torch.uint8)
    wp, wn = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                  workspace.numel() * workspace.element_size())
    _check("hyena_attn_paged_fp8", lib().hyena_attn_paged_fp8(
        qp, qt, qh, kc, vc, ks, vs, N, P, tp, step, width, lp, cp, R, T, max_q, Hq, Hkv, DH,
        1.0 / math.sqrt(DH) if scale is None else float(scale), op, _io(q), wp, wn, _stream(q)))
    return out
