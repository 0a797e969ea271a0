"""Binding of the operators around the products: residual RMS norm, rotary cache write, tree attention
and the 8-bit block product.  Argument marshalling only, as in ``_lib``: every call checks that its
tensors are on one GPU, before it allocates or enqueues anything, and that they have the shapes and types of
the C ABI (include/w12.h), enqueues on the current stream (or ``stream``) and returns; pitches and alignment
are checked by the library."""
from __future__ import annotations

import contextlib
import ctypes

import torch

from ._lib import _AttentionArgs, _KVCache, _NormArgs, _RopeArgs, _c_u64, _check, _ptr, lib

DTYPE_BF16, DTYPE_F32, DTYPE_E4M3 = 0, 1, 2
QUANT_BLOCK = 128
_COUNTER_BYTES = 16384      # the counters at the start of a product's workspace; the partial sums behind them hold anything

_BF16, _F32, _E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_FLOATS = {_BF16: DTYPE_BF16, _F32: DTYPE_F32}
_MASKS = (torch.int64, torch.uint64)


def _device(*ts) -> int:
    """The one GPU that every tensor is on; it has to be the current one, whose streams the call uses."""
    d = None
    for t in ts:
        if t is None:
            continue
        i = t.get_device()
        if i != d:
            if i < 0:
                raise ValueError("tensors must live on the GPU (libw12 has no CPU path)")
            if d is not None:
                raise ValueError("tensors are on different GPUs")
            d = i
    if d != torch.cuda.current_device():
        raise ValueError("the tensors' GPU is not the current one (use torch.cuda.device)")
    return d


# The current stream's handle without the Stream object (0.2 against 2 us, a fifth of a small call).
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _raw_stream(stream) -> int:
    return _current_raw_stream(torch.cuda.current_device()) if stream is None else stream.cuda_stream


def _on(stream):
    """Where a call allocates: on the stream that it was given, else where torch is (entering the current stream
    again costs as much as a small call)."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _rows(t: torch.Tensor, what: str, shape: tuple, dtypes, step: int) -> int:
    """Checks a matrix with contiguous rows; its pitch in elements.  A single row is never stepped
    by its pitch, and torch may report any stride for it, so it gets its padded width."""
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {shape}, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: expected {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{what}: rows must be contiguous")
    return ld if shape[0] != 1 else -(-shape[1] // step) * step


def _vector(t: torch.Tensor, what: str, n: int, dtype) -> None:
    if t.shape != (n,):
        raise ValueError(f"{what}: expected shape {(n,)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{what}: must be contiguous")


def _matrix2(t, what):
    if t.dim() != 2:
        raise ValueError(f"{what}: expected a 2-D tensor")
    return t.shape


def add_rmsnorm(residual: torch.Tensor, weight: torch.Tensor, delta: torch.Tensor | None = None, eps: float = 1e-6,
                residual_out: torch.Tensor | None = None, y: torch.Tensor | None = None, yq: torch.Tensor | None = None,
                yq_scale: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """r = residual + delta, stored to residual_out (which may be residual itself); y = r's RMS norm times
    weight.  residual and delta: BF16 or FP32 [M, N], rows of whole 16-byte steps; weight: BF16 [N].

    y (BF16, what gemm() takes) and yq with yq_scale (E4M3 and a scale per row and 128 columns, what
    gemm_e4m3() takes) are the outputs that are wanted; with none given, y is allocated here, on the
    stream.  Returns y (None when only yq is wanted)."""
    m, n = _matrix2(residual, "residual")
    _device(residual, weight, delta, residual_out, y, yq, yq_scale)
    if y is None and yq is None:
        with _on(stream):
            y = torch.empty(m, (n + 7) // 8 * 8, dtype=_BF16, device=residual.device)[:, :n]
    shape = (m, n)
    rt = residual.dtype
    step = 4 if rt == _F32 else 8
    ld_r = _rows(residual, "residual", shape, _FLOATS, step)
    _vector(weight, "weight", n, _BF16)
    dt = ld_d = ld_o = ld_y = ld_q = ld_s = 0
    if delta is not None:
        ld_d = _rows(delta, "delta", shape, _FLOATS, 4 if delta.dtype == _F32 else 8)
        dt = _FLOATS[delta.dtype]
    if residual_out is not None:
        ld_o = _rows(residual_out, "residual_out", shape, (rt,), step)
    if y is not None:
        ld_y = _rows(y, "y", shape, (_BF16,), 8)
    if (yq is None) != (yq_scale is None):
        raise ValueError("yq and yq_scale go together")
    if yq is not None:
        ld_q = _rows(yq, "yq", shape, (_E4M3,), 16)
        ld_s = _rows(yq_scale, "yq_scale", (m, -(-n // QUANT_BLOCK)), (_F32,), 1)
    a = _NormArgs(m, n, _FLOATS[rt], dt, residual.data_ptr(), ld_r, _ptr(delta), ld_d, weight.data_ptr(),
                  _ptr(residual_out), ld_o, _ptr(y), ld_y, _ptr(yq), ld_q, _ptr(yq_scale), ld_s, eps, 0)
    _check("w12_add_rmsnorm", lib().w12_add_rmsnorm(ctypes.byref(a), _raw_stream(stream)))
    return y


class KVCache:
    """A paged key / value cache: K and V [pages, page_size, heads, dim] (BF16, or E4M3 with a scale per head;
    views with other orders of the axes are fine as long as dim is contiguous).  The object keeps the
    tensors and their C descriptor; the cache's contents belong to the caller."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must have one shape [pages, page_size, heads, dim]")
        if k.dtype != v.dtype or k.dtype not in (_BF16, _E4M3):
            raise TypeError("k and v must both be bfloat16 or both float8_e4m3fn")
        if k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must have the same strides, with dim contiguous")
        pages, page, heads, dim = k.shape
        if (k.dtype == _E4M3) != (k_scale is not None) or (k_scale is None) != (v_scale is None):
            raise ValueError("an E4M3 cache has k_scale and v_scale, a BF16 cache has none")
        if k_scale is not None:
            _vector(k_scale, "k_scale", heads, _F32)
            _vector(v_scale, "v_scale", heads, _F32)
        for t in (k, v, k_scale, v_scale):
            if t is not None and not t.is_cuda:
                raise ValueError("tensors must live on the GPU (libw12 has no CPU path)")
            if t is not None and t.device != k.device:
                raise ValueError("tensors are on different GPUs")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.page_size, self.heads, self.dim = pages, page, heads, dim
        d = self.desc = _KVCache()
        d.dtype = DTYPE_BF16 if k.dtype == _BF16 else DTYPE_E4M3
        d.pages, d.page_size, d.heads, d.dim = pages, page, heads, dim
        d.page_stride, d.token_stride, d.head_stride = (0 if s == 1 else k.stride(i) for i, s in enumerate(k.shape[:3]))
        d.k, d.v = k.data_ptr(), v.data_ptr()
        if k_scale is not None:
            d.k_scale, d.v_scale = k_scale.data_ptr(), v_scale.data_ptr()


def rope_append(qkv: torch.Tensor, cache: KVCache, positions: torch.Tensor, slots: torch.Tensor, inv_freq: torch.Tensor,
                q_heads: int, axis: torch.Tensor | None = None, adjacent: bool = False, q: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """Rows [T, (q_heads + 2 heads) * dim] of a QKV product (FP32 or BF16) -> Q (BF16 [T, q_heads * dim],
    returned), and K, V put into the cache at slots (int64 [T]: page * page_size + token of the page;
    a negative slot is not put).  Q and K are turned by positions (int32 [axes, T]) times inv_freq
    (float64 [rot_dim / 2]); axis (uint8 [rot_dim / 2]) names the axis of every pair."""
    t, width = _matrix2(qkv, "qkv")
    dim = cache.dim
    if width != (q_heads + 2 * cache.heads) * dim:
        raise ValueError(f"qkv: expected {(q_heads + 2 * cache.heads) * dim} columns, got {width}")
    _device(qkv, cache.k, positions, slots, inv_freq, axis, q)
    if q is None:
        with _on(stream):
            q = torch.empty(t, q_heads * dim, dtype=_BF16, device=qkv.device)
    ld_x = _rows(qkv, "qkv", (t, width), _FLOATS, 8)
    axes = _matrix2(positions, "positions")[0]
    ld_p = _rows(positions, "positions", (axes, t), (torch.int32,), 1)
    _vector(slots, "slots", t, torch.int64)
    pairs = inv_freq.numel()
    _vector(inv_freq, "inv_freq", pairs, torch.float64)
    if axis is not None:
        _vector(axis, "axis", pairs, torch.uint8)
    ld_q = _rows(q, "q", (t, q_heads * dim), (_BF16,), 8)
    # a single row of positions is stepped by its pitch no more than a single row of anything: T will do
    a = _RopeArgs(t, q_heads, _FLOATS[qkv.dtype], 2 * pairs, axes, int(adjacent), qkv.data_ptr(), ld_x,
                  positions.data_ptr(), ld_p, slots.data_ptr(), inv_freq.data_ptr(), _ptr(axis), q.data_ptr(), ld_q)
    _check("w12_rope_append", lib().w12_rope_append(ctypes.byref(a), ctypes.byref(cache.desc), _raw_stream(stream)))
    return q


def tree_attention_workspace_size(rows: int, requests: int, q_heads: int, cache: KVCache) -> int:
    b = _c_u64()
    _check("w12_tree_attention_workspace_size",
           lib().w12_tree_attention_workspace_size(rows, requests, q_heads, ctypes.byref(cache.desc), ctypes.byref(b)))
    return b.value


def tree_attention_workspace(rows: int, requests: int, q_heads: int, cache: KVCache) -> torch.Tensor | None:
    """A workspace for tree_attention() of at most this many rows and requests over this cache, or None."""
    need = tree_attention_workspace_size(rows, requests, q_heads, cache)
    return torch.empty(need, dtype=torch.uint8, device=cache.k.device) if need else None


def tree_attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, ctx_len: torch.Tensor,
                   node_ptr: torch.Tensor, tree_mask: torch.Tensor | None = None, scale: float | None = None,
                   out: torch.Tensor | None = None, lse: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Attention of drafted tokens over a paged cache (w12_tree_attention): q BF16 [T, q_heads * dim] ->
    out BF16 [T, q_heads * dim], and lse FP32 [T, q_heads] if given.

    Request b has rows node_ptr[b] .. node_ptr[b + 1] - 1 (int32 [B + 1]) and ctx_len[b] (int32 [B]) tokens in
    the cache; its node i is token ctx_len[b] + i.  page_table: int32 [B, max_pages].  tree_mask: int64
    [T, words], bit j % 64 of word j / 64 set where the row's node attends node j of its request; None: a chain.
    scale: 1 / sqrt(dim) by default.  ws: tree_attention_workspace(); allocated here when omitted."""
    t, width = _matrix2(q, "q")
    dim = cache.dim
    q_heads = width // dim
    if q_heads * dim != width or q_heads == 0:
        raise ValueError(f"q: {width} columns are not whole heads of {dim}")
    _device(q, cache.k, page_table, ctx_len, node_ptr, tree_mask, out, lse, ws)
    if out is None or ws is None:
        with _on(stream):
            if out is None:
                out = torch.empty(t, width, dtype=_BF16, device=q.device)
            if ws is None:
                ws = tree_attention_workspace(t, ctx_len.numel(), q_heads, cache)
    requests = ctx_len.numel()
    _vector(ctx_len, "ctx_len", requests, torch.int32)
    _vector(node_ptr, "node_ptr", requests + 1, torch.int32)
    ld_q = _rows(q, "q", (t, width), (_BF16,), 8)
    max_pages = _matrix2(page_table, "page_table")[1]
    ld_t = _rows(page_table, "page_table", (requests, max_pages), (torch.int32,), 1)
    words = ld_m = ld_l = 0
    if tree_mask is not None:
        words = _matrix2(tree_mask, "tree_mask")[1]
        ld_m = _rows(tree_mask, "tree_mask", (t, words), _MASKS, 1)
    ld_o = _rows(out, "out", (t, width), (_BF16,), 8)
    if lse is not None:
        ld_l = _rows(lse, "lse", (t, q_heads), (_F32,), 1)
    a = _AttentionArgs(t, requests, q_heads, max_pages, words, dim ** -0.5 if scale is None else scale, q.data_ptr(), ld_q,
                       node_ptr.data_ptr(), ctx_len.data_ptr(), page_table.data_ptr(), ld_t, _ptr(tree_mask), ld_m,
                       out.data_ptr(), ld_o, _ptr(lse), ld_l)
    wsp, wsb = (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())
    _check("w12_tree_attention", lib().w12_tree_attention(ctypes.byref(a), ctypes.byref(cache.desc), wsp, wsb,
                                                          _raw_stream(stream)))
    return out


def gemm_e4m3_workspace_size(m: int, n: int, k: int) -> int:
    b = _c_u64()
    _check("w12_gemm_e4m3_workspace_size", lib().w12_gemm_e4m3_workspace_size(m, n, k, ctypes.byref(b)))
    return b.value


def gemm_e4m3_workspace(m: int, n: int, k: int, device="cuda", stream=None) -> torch.Tensor | None:
    """A ready-to-use workspace (its counters are zero) for gemm_e4m3() of up to m rows on W[n][k], or None.
    With a stream, it belongs to that stream."""
    d = torch.device(device)
    if d.type != "cuda":
        raise ValueError("tensors must live on the GPU (libw12 has no CPU path)")
    if d.index is not None and d.index != torch.cuda.current_device():
        raise ValueError("the tensors' GPU is not the current one (use torch.cuda.device)")
    need = gemm_e4m3_workspace_size(m, n, k)
    if not need:
        return None
    with _on(stream):
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    _check("w12_gemm_workspace_init",
           lib().w12_gemm_workspace_init(ws.data_ptr(), min(need, _COUNTER_BYTES), _raw_stream(stream)))
    return ws


def gemm_e4m3(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
              y: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y[M, N] (FP32) = (X x_scale) (W w_scale)^T with E4M3 X [M, K] and W [N, K], x_scale FP32 [M, ceil(K / 128)] and
    w_scale FP32 [ceil(N / 128), ceil(K / 128)].  ws: gemm_e4m3_workspace(); allocated here when omitted."""
    m, k = _matrix2(x, "x")
    n = _matrix2(w, "w")[0]
    kb = -(-k // QUANT_BLOCK)
    _device(x, x_scale, w, w_scale, y, ws)
    if y is None or ws is None:
        with _on(stream):
            if y is None:
                y = torch.empty(m, n, dtype=_F32, device=x.device)
            if ws is None:
                ws = gemm_e4m3_workspace(m, n, k, x.device)
    wsp, wsb = (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())
    _check("w12_gemm_e4m3", lib().w12_gemm_e4m3(
        x.data_ptr(), m, _rows(x, "x", (m, k), (_E4M3,), 16),
        x_scale.data_ptr(), _rows(x_scale, "x_scale", (m, kb), (_F32,), 1),
        w.data_ptr(), n, k, _rows(w, "w", (n, k), (_E4M3,), 16),
        w_scale.data_ptr(), _rows(w_scale, "w_scale", (-(-n // QUANT_BLOCK), kb), (_F32,), 1),
        y.data_ptr(), _rows(y, "y", (m, n), (_F32,), 1), wsp, wsb, _raw_stream(stream)))
    return y

