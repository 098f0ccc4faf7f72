"""Python binding of the operators between an adapted layer's projections (include/lora_layer.h):
argument marshalling only; every step runs in the library.

    h = x + residual;  y = h (mean(h^2) + eps)^(-1/2) (weight + weight_offset)     add_rms_norm
    new keys and values into a paged cache, queries and keys turned by position    kv_append
    o_t = sum_j softmax_j(scale q_t . k_j) v_j over the tokens that row t sees     PagedAttention

``q_offsets`` is the host list that ``LoraLinear.forward`` takes as ``seg_offsets``; ``kv_lens``
and ``block_table`` are int32 tensors on the device, read when the call runs, so that a captured
decode step can be replayed as the caches grow.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib as L
from .lora_linear import LoraError, _check  # noqa: F401

FP8 = torch.float8_e4m3fn
BF16 = torch.bfloat16

# The calls below serve steps of a few microseconds, so their checks read each property of a tensor once.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream, device: torch.device) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _dev(t: torch.Tensor, dtype: torch.dtype, device: torch.device, name: str) -> int:
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, is on {t.device}")
    return t.data_ptr()


def _cuda(t: torch.Tensor, name: str) -> torch.device:
    d = t.device
    if d.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    return d


def _rows(t: torch.Tensor, shape, dtype: torch.dtype, device: torch.device, name: str):
    """(pointer, row stride) of a [rows, width] tensor whose rows are contiguous."""
    if t.dtype is not dtype or t.device != device:
        _dev(t, dtype, device, name)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")
    s, i = t.stride()
    if i != 1 and shape[1] > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return t.data_ptr(), s if shape[0] > 1 else shape[1]


def _heads(t: torch.Tensor, n_heads: int, dim: int, device: torch.device, name: str):
    """(pointer, row stride, head stride) of a [rows, heads, dim] tensor with contiguous features."""
    if t.dtype is not BF16 or t.device != device:
        _dev(t, BF16, device, name)
    shape = t.shape
    if len(shape) != 3 or shape[1] != n_heads or shape[2] != dim:
        raise ValueError(f"{name} must have shape [rows, {n_heads}, {dim}], has {tuple(shape)}")
    st, sh, si = t.stride()
    if si != 1:
        raise ValueError(f"{name}'s features must be contiguous")
    if n_heads == 1:
        sh = dim
    return t.data_ptr(), st if shape[0] > 1 else max(st, dim) // 8 * 8, sh


def _on(device: torch.device, fn, *args) -> int:
    """fn(*args) with `device` current, for the calls that take no handle."""
    prev = _device() if _device is not None else torch.cuda.current_device()
    if prev == device.index:
        return fn(*args)
    torch.cuda.set_device(device)
    try:
        return fn(*args)
    finally:
        torch.cuda.set_device(prev)


def _norm(x, weight, residual, eps, weight_offset, h_out, y, q8, scales, group, stream):
    dev = _cuda(x, "x")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must have shape [rows, width]")
    xp, xs = _rows(x, shape, BF16, dev, "x")
    wp = _dev(weight, BF16, dev, "weight")
    if weight.shape != shape[1:] or (weight.stride(0) != 1 and shape[1] > 1):
        raise ValueError(f"weight must be contiguous with shape ({shape[1]},)")
    rp = hp = yp = qp = sp = None
    rs = hs = ys = qs = 0
    if residual is not None:
        rp, rs = _rows(residual, shape, BF16, dev, "residual")
    if h_out is not None:
        hp, hs = _rows(h_out, shape, BF16, dev, "h_out")
    if y is not None:
        yp, ys = _rows(y, shape, BF16, dev, "out")
    if q8 is not None:
        qp, qs = _rows(q8, shape, FP8, dev, "out")
        sp = _dev(scales, torch.float32, dev, "scales")
    rc = _on(dev, L.load().lora_linear_add_rms_norm, xp, xs, rp, rs, wp, weight_offset, eps, shape[0], shape[1], hp, hs,
             yp, ys, qp, qs, sp, group, _stream(stream, dev))
    if rc:
        _check(rc, "lora_linear_add_rms_norm")


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *, eps: float = 1e-6,
                 weight_offset: float = 0.0, out: torch.Tensor | None = None, h_out: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None):
    """(y, h) of the rows x [rows, width]: h = x + residual (bf16) and its norm y (bf16). Without a
    residual h is x itself and nothing is written for it. ``h_out`` may be ``residual`` or ``x``."""
    if out is None:
        out = torch.empty_like(x)
    if residual is not None and h_out is None:
        h_out = torch.empty_like(x)
    _norm(x, weight, residual, eps, weight_offset, h_out, out, None, None, 0, stream)
    return out, (h_out if h_out is not None else x)


def add_rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *, eps: float = 1e-6,
                     weight_offset: float = 0.0, group: int = 0, out: torch.Tensor | None = None,
                     scales: torch.Tensor | None = None, h_out: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None):
    """(q, scales, h): the norm in 8 bits (e4m3), y = q * scales, with one fp32 scale per row (group 0) or
    per ``group`` features (32, 64, 128 or 256) of a row; h as ``add_rms_norm``."""
    if group not in (0, 32, 64, 128, 256):
        raise ValueError("group must be 0, 32, 64, 128 or 256")
    n = 1 if group == 0 else -(-x.shape[1] // group)
    if out is None:
        out = torch.empty_like(x, dtype=FP8)
    if scales is None:
        scales = torch.empty((x.shape[0], n), dtype=torch.float32, device=x.device)
    elif scales.shape != (x.shape[0], n) or not scales.is_contiguous():
        raise ValueError(f"scales must be contiguous with shape {(x.shape[0], n)}")
    if residual is not None and h_out is None:
        h_out = torch.empty_like(x)
    _norm(x, weight, residual, eps, weight_offset, h_out, None, out, scales, group, stream)
    return out, scales, (h_out if h_out is not None else x)


def _cache(k_cache, v_cache, q_offsets, kv_lens, block_table, device):
    """The ``lora_kv_cache`` of these tensors; the caches are [n_pages, page_size, n_kv_heads, head_dim]."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must both have shape [n_pages, page_size, n_kv_heads, head_dim]")
    n_pages, page, n_kv, dim = shape
    kp, vp = _dev(k_cache, BF16, device, "k_cache"), _dev(v_cache, BF16, device, "v_cache")
    ks, vs = k_cache.stride(), v_cache.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("the caches' features must be contiguous")
    if n_pages == 1 or n_kv == 1:        # an axis of one has no stride of its own
        ks = (ks[0] if n_pages > 1 else dim, ks[1], ks[2] if n_kv > 1 else dim)
        vs = (vs[0] if n_pages > 1 else dim, vs[1], vs[2] if n_kv > 1 else dim)
    tp = _dev(block_table, torch.int32, device, "block_table")
    if block_table.dim() != 2:
        raise ValueError("block_table must have shape [n_seqs, pages_per_seq] with contiguous rows")
    n, per = block_table.shape
    ts, ti = block_table.stride()
    if ti != 1 and per > 1:
        raise ValueError("block_table must have shape [n_seqs, pages_per_seq] with contiguous rows")
    lp = _dev(kv_lens, torch.int32, device, "kv_lens")
    if kv_lens.shape != (n,) or (n > 1 and kv_lens.stride(0) != 1):
        raise ValueError(f"kv_lens must be contiguous with shape ({n},)")
    if len(q_offsets) != n + 1:
        raise ValueError("q_offsets must hold one more entry than there are sequences")
    return L.KvCache(kp, vp, ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], n_pages, page, n_kv, dim, tp,
                     ts if n > 1 else per, per, n, lp, (C.c_int32 * (n + 1))(*q_offsets))


def kv_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, q_offsets, kv_lens: torch.Tensor,
              block_table: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, cos: torch.Tensor | None = None,
              sin: torch.Tensor | None = None, *, q_out: torch.Tensor | None = None,
              stream: torch.cuda.Stream | None = None):
    """Writes the rows' keys and values k, v [T, n_kv_heads, head_dim] to their places in the paged cache and
    returns the turned queries (q [T, n_heads, head_dim]; ``q_out`` may be q itself). ``cos``, ``sin``: fp32
    [n_positions, rot / 2], or None for no rotary turn (q is then returned as it is, unless ``q_out`` is
    given). ``kv_lens`` counts the new rows."""
    dev = _cuda(k, "k")
    c = _cache(k_cache, v_cache, q_offsets, kv_lens, block_table, dev)
    T = q_offsets[-1]
    rot = n_pos = 0
    cp = sp = None
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        if cos.dim() != 2 or cos.shape != sin.shape or not cos.is_contiguous() or not sin.is_contiguous():
            raise ValueError("cos and sin must be contiguous and have one shape [n_positions, rot / 2]")
        n_pos, rot = cos.shape[0], 2 * cos.shape[1]
        cp, sp = _dev(cos, torch.float32, dev, "cos"), _dev(sin, torch.float32, dev, "sin")
    n_kv, dim = c.n_kv_heads, c.head_dim
    kp, ks, kh = _heads(k, n_kv, dim, dev, "k")
    vp, vs, vh = _heads(v, n_kv, dim, dev, "v")
    if k.shape[0] != T or v.shape[0] != T or (q is not None and q.shape[0] != T):
        raise ValueError("q, k and v must have q_offsets[-1] rows")
    qp = op = None
    qs = qh = os_ = oh = n_heads = 0
    if q is None:
        q_out = None
    elif rot or q_out is not None:
        n_heads = q.shape[1]
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        elif q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
        qp, qs, qh = _heads(q, n_heads, dim, dev, "q")
        op, os_, oh = _heads(q_out, n_heads, dim, dev, "q_out")
    else:
        q_out = q
    rc = _on(dev, L.load().lora_linear_kv_append, c, qp, qs, qh, op, os_, oh, n_heads, kp, ks, kh, vp, vs, vh, cp, sp, rot,
             n_pos, _stream(stream, dev))
    if rc:
        _check(rc, "lora_linear_kv_append")
    return q_out


class PagedAttention:
    """One handle: attention of n_heads query heads over a paged cache with n_kv_heads heads."""

    def __init__(self, n_heads: int, n_kv_heads: int, head_dim: int, page_size: int, max_tokens: int,
                 max_seqs: int = 64, device: int | torch.device | None = None):
        self._lib = L.load()
        self._forward = self._lib.lora_linear_attn_forward
        if device is None:
            device = torch.cuda.current_device()
        if isinstance(device, torch.device):
            device = device.index if device.index is not None else torch.cuda.current_device()
        self.device = torch.device("cuda", int(device))
        self.n_heads, self.n_kv_heads, self.head_dim, self.page_size = n_heads, n_kv_heads, head_dim, page_size
        self.max_tokens, self.max_seqs = max_tokens, max_seqs
        h = C.c_void_p()
        _check(self._lib.lora_linear_attn_create(C.byref(h), n_heads, n_kv_heads, head_dim, page_size, max_tokens,
                                                 max_seqs, int(device)), "lora_linear_attn_create")
        self._h = h

    def close(self) -> None:
        if getattr(self, "_h", None):
            self._lib.lora_linear_attn_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def forward(self, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, q_offsets,
                kv_lens: torch.Tensor, block_table: torch.Tensor, *, scale: float | None = None, window: int = 0,
                sinks: int = 0, out: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None) -> torch.Tensor:
        """o [T, n_heads, head_dim] of the new rows q over the cache; a row sees the tokens up to its own, or
        (window > 0) the last ``window`` of them and the first ``sinks`` tokens. scale: 1 / sqrt(head_dim)."""
        dev = self.device
        c = _cache(k_cache, v_cache, q_offsets, kv_lens, block_table, dev)
        if q.shape[0] != q_offsets[-1]:
            raise ValueError("q must have q_offsets[-1] rows")
        qp, qs, qh = _heads(q, self.n_heads, self.head_dim, dev, "q")
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        elif out.shape != q.shape:
            raise ValueError("out must have q's shape")
        op, os_, oh = _heads(out, self.n_heads, self.head_dim, dev, "out")
        if scale is None:
            scale = self.head_dim ** -0.5
        rc = self._forward(self._h, c, qp, qs, qh, op, os_, oh, scale, window, sinks, _stream(stream, dev))
        if rc:
            _check(rc, "lora_linear_attn_forward")
        return out

    def status(self, reset: bool = False) -> int:
        return self._lib.lora_linear_attn_status(self._h, 1 if reset else 0)
