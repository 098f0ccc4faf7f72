"""Python entry points of the operators between an adapted layer's projections (include/lora_layer.h).
Arguments are checked and marshalled by ``csrc/layer_bind.cpp``; every step runs in the library.

    h = x + residual;  y = h (mean(h^2) + eps)^(-1/2) (weight + weight_offset)     add_rms_norm
    new keys and values into a paged cache, queries and keys turned by position    kv_append
    o_t = sum_j softmax_j(scale q_t . k_j) v_j over the tokens that row t sees     PagedAttention

``q_offsets`` is the host list that ``LoraLinear.forward`` takes as ``seg_offsets``; ``kv_lens``
and ``block_table`` are int32 tensors on the device, read when the call runs, so that a captured
decode step can be replayed as the caches grow.

The operators serve: no gradient passes through them, whatever their inputs require. A tensor that a
call writes counts as modified in place.

``stream``: a call runs on it as under ``torch.cuda.stream(stream)``. What it allocates belongs to that
stream; that the inputs are ready there, and that another stream waits before it uses the outputs, is the
caller's to see to.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib as L
from .build import bind_for
from .lora_linear import LoraError, _check  # noqa: F401

_bind = None


def _load():
    """The native binding, bound to the library (once per process)."""
    global _bind
    lib = L.load()
    try:
        from . import _layer_bind
        built_for = getattr(_layer_bind, "built_for", "unknown")
    except ImportError as e:
        built_for = str(e)
    if built_for != bind_for():
        raise RuntimeError(f"_layer_bind.so is not built for this PyTorch ({built_for}): run __graft_entry__.build() "
                           "(or python -m mixed_lora_projection_gb300.build)")
    _layer_bind.bind(*(C.cast(f, C.c_void_p).value for f in (
        lib.lora_linear_add_rms_norm, lib.lora_linear_kv_append, lib.lora_linear_attn_forward)), _check)
    _bind = _layer_bind
    return _bind


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *, eps: float = 1e-6,
                 weight_offset: float = 0.0, out: torch.Tensor | None = None, h_out: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None):
    """(y, h) of the rows x [rows, width]: h = x + residual (bf16) and its norm y (bf16). Without a
    residual h is x itself and nothing is written for it (a copy of x, where ``out`` is x). ``h_out`` may be
    ``residual`` or ``x``."""
    return (_bind or _load()).norm(x, weight, residual, eps, weight_offset, out, h_out, None, -1, stream)


def add_rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *, eps: float = 1e-6,
                     weight_offset: float = 0.0, group: int = 0, out: torch.Tensor | None = None,
                     scales: torch.Tensor | None = None, h_out: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None):
    """(q, scales, h): the norm in 8 bits (e4m3), y = q * scales, with one fp32 scale per row (group 0) or
    per ``group`` features (32, 64, 128 or 256) of a row; h as ``add_rms_norm``."""
    if group < 0:
        raise ValueError("group must be 0, 32, 64, 128 or 256")
    return (_bind or _load()).norm(x, weight, residual, eps, weight_offset, out, h_out, scales, group, stream)


def kv_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, q_offsets, kv_lens: torch.Tensor,
              block_table: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, cos: torch.Tensor | None = None,
              sin: torch.Tensor | None = None, *, q_out: torch.Tensor | None = None,
              stream: torch.cuda.Stream | None = None):
    """Writes the rows' keys and values k, v [T, n_kv_heads, head_dim] to their places in the paged cache
    (k_cache, v_cache [n_pages, page_size, n_kv_heads, head_dim]) and returns the turned queries (q [T, n_heads,
    head_dim]; ``q_out`` may be q itself). ``cos``, ``sin``: fp32 [n_positions, rot / 2] (positions past either end
    use the row at that end), or None for no rotary turn (q is then returned as it is, unless ``q_out`` is given).
    ``kv_lens`` counts the new rows."""
    return (_bind or _load()).append(q, k, v, q_offsets, kv_lens, block_table, k_cache, v_cache, cos, sin, q_out, stream)


class PagedAttention:
    """One handle: attention of n_heads query heads over a paged cache with n_kv_heads heads. Its calls share a
    workspace, so they go one after another: on one stream, or on streams that wait for each other."""

    def __init__(self, n_heads: int, n_kv_heads: int, head_dim: int, page_size: int, max_tokens: int,
                 max_seqs: int = 64, device: int | torch.device | None = None):
        self._lib = L.load()
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
        self._ptr = h.value

    def close(self) -> None:
        if getattr(self, "_h", None):
            self._lib.lora_linear_attn_destroy(self._h)
            self._h = self._ptr = None

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
        (window > 0) the last ``window`` of them and the first ``sinks`` tokens. scale: 1 / sqrt(head_dim). The sums' order goes by
        the batch: a row's last bit may differ in another one."""
        return (_bind or _load()).attend(self._ptr, self.n_heads, self.head_dim, self.device.index, q, k_cache, v_cache,
                                         q_offsets, kv_lens, block_table, scale, window, sinks, out, stream)

    def set_option(self, option: int, value: int) -> None:
        _check(self._lib.lora_linear_attn_set_option(self._h, option, int(value)), "lora_linear_attn_set_option")

    def status(self, reset: bool = False) -> int:
        return self._lib.lora_linear_attn_status(self._h, 1 if reset else 0)
