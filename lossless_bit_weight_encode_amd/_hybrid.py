"""Binding of a hybrid target's operators in speculative decoding: short convolution, gated delta rule and the
verification of drafted tokens.  Argument marshalling only, as in ``_ops``: every call checks that its tensors are on
one GPU, before it allocates or enqueues anything, and that they have the shapes and types of the C ABI
(include/w12.h), enqueues on the current stream (or ``stream``) and returns."""
from __future__ import annotations

import ctypes

import torch

from ._lib import _ConvArgs, _DeltaArgs, _Sequences, _VerifyDraftArgs, _c_u64, _check, _ptr, lib
from ._ops import _BF16, _F32, _FLOATS, _MASKS, _device, _matrix2, _on, _raw_stream, _rows, _vector

TREE_NODES = 64         # nodes of a tree for short_conv() and gated_delta()
VERIFY_NODES = 4096     # nodes of a request for verify_draft()
DELTA_CHUNK_FROM, DELTA_CHUNK_FROM_LENS = 12, 65      # rows a sequence from which gated_delta() needs its workspace, without and with lens
DELTA_CHUNK_LONG = 64   # rows past one a sequence from which it has use for one, without lens

_I32 = torch.int32


def _sequences(t: int, slots: int, seq_ptr, src, dst, tree_mask, lens, rows) -> _Sequences:
    """The descriptor of a call's sequences, for t rows and a state array of this many slots."""
    count = src.numel()
    _vector(src, "src", count, _I32)
    _vector(seq_ptr, "seq_ptr", count + 1, _I32)
    if dst is not None:
        _vector(dst, "dst", count, _I32)
    if lens is not None:
        _vector(lens, "lens", count, _I32)
    if rows is not None:
        _vector(rows, "rows", t, _I32)
    words = ld_m = 0
    if tree_mask is not None:
        words = _matrix2(tree_mask, "tree_mask")[1]
        ld_m = _rows(tree_mask, "tree_mask", (t, words), _MASKS, 1)
    return _Sequences(t, count, seq_ptr.data_ptr(), _ptr(lens), _ptr(rows), src.data_ptr(), _ptr(dst), _ptr(tree_mask), ld_m,
                      words, slots)


def short_conv(x: torch.Tensor, weight: torch.Tensor, state: torch.Tensor, seq_ptr: torch.Tensor, src: torch.Tensor,
               dst: torch.Tensor | None = None, bias: torch.Tensor | None = None, silu: bool = True,
               tree_mask: torch.Tensor | None = None, lens: torch.Tensor | None = None, rows: torch.Tensor | None = None,
               y: torch.Tensor | None = None, outputs: bool = True, stream=None) -> torch.Tensor | None:
    """Short causal convolution of every channel (w12_short_conv): x [T, channels] (FP32 or BF16), weight BF16
    [channels, width], bias BF16 [channels] -> y BF16 [T, channels], with SiLU unless silu is false.

    Sequence b has rows seq_ptr[b] .. seq_ptr[b + 1] - 1 (int32 [B + 1]) and starts from state[src[b]], the width - 1
    rows of x before its first; with dst, its last ones go to state[dst[b]].  state: [slots, width - 1, channels] of x's type.
    src, dst: int32 [B]; a slot outside the array stands for zeros, or for a state that is not kept.
    tree_mask (int64 [T, words], as for tree_attention()) makes every range a tree of up to 64 drafted tokens.
    rows (int32 [T]) names the rows that a sequence's tokens are, lens (int32 [B]) how many count: verify_draft()'s path
    and count.  With outputs false only the states move on.  Returns y (None without outputs)."""
    t, c = _matrix2(x, "x")
    width = _matrix2(weight, "weight")[1]
    _device(x, weight, state, seq_ptr, src, dst, bias, tree_mask, lens, rows, y)
    if y is not None and not outputs:
        raise ValueError("y without outputs")
    if outputs and y is None:
        with _on(stream):
            y = torch.empty(t, (c + 7) // 8 * 8, dtype=_BF16, device=x.device)[:, :c]
    step = 4 if x.dtype == _F32 else 8
    ld_x = _rows(x, "x", (t, c), _FLOATS, step)
    if weight.shape != (c, width) or weight.dtype != _BF16 or not weight.is_contiguous():
        raise ValueError(f"weight: expected a contiguous bfloat16 matrix of {c} rows")
    if bias is not None:
        _vector(bias, "bias", c, _BF16)
    if state.dim() != 3 or state.shape[1:] != (width - 1, c):
        raise ValueError(f"state: expected shape (slots, {width - 1}, {c}), got {tuple(state.shape)}")
    if state.dtype != x.dtype:
        raise TypeError(f"state: expected x's type, {x.dtype}, got {state.dtype}")
    padded = -(-c // step) * step
    slot, tap, one = state.stride()
    if one != 1 and c > 1:
        raise ValueError("state: channels must be contiguous")
    tap = tap if width > 2 else padded            # a single tap or slot is never stepped
    slot = slot if state.shape[0] > 1 else (width - 1) * max(tap, padded)
    ld_y = 0 if y is None else _rows(y, "y", (t, c), (_BF16,), 8)
    s = _sequences(t, state.shape[0], seq_ptr, src, dst, tree_mask, lens, rows)
    a = _ConvArgs(c, width, _FLOATS[x.dtype], int(silu), x.data_ptr(), ld_x, weight.data_ptr(), _ptr(bias), state.data_ptr(),
                  slot, tap, _ptr(y), ld_y)
    _check("w12_short_conv", lib().w12_short_conv(ctypes.byref(a), ctypes.byref(s), _raw_stream(stream)))
    return y


def _delta_state(state) -> tuple:
    if state.dim() != 4:
        raise ValueError("state: expected shape (slots, v_heads, dv, dk)")
    if state.dtype != _F32:
        raise TypeError(f"state: expected torch.float32, got {state.dtype}")
    return state.shape


def gated_delta_workspace_size(t: int, count: int, v_heads: int, dk: int, dv: int) -> int:
    b = _c_u64()
    _check("w12_gated_delta_workspace_size", lib().w12_gated_delta_workspace_size(t, count, v_heads, dk, dv, ctypes.byref(b)))
    return b.value


def gated_delta_workspace(t: int, count: int, state: torch.Tensor) -> torch.Tensor | None:
    """A workspace for gated_delta() of at most t rows in this many sequences over these states, or None."""
    _, h, dv, dk = _delta_state(state)
    need = gated_delta_workspace_size(t, count, h, dk, dv)
    return torch.empty(need, dtype=torch.uint8, device=state.device) if need else None


def gated_delta(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                state: torch.Tensor, seq_ptr: torch.Tensor, src: torch.Tensor, dst: torch.Tensor | None = None,
                scale: float | None = None, l2norm: bool = True, eps: float = 1e-6, tree_mask: torch.Tensor | None = None,
                lens: torch.Tensor | None = None, rows: torch.Tensor | None = None, out: torch.Tensor | None = None,
                outputs: bool = True, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """The gated delta rule (w12_gated_delta): q, k BF16 [T, k_heads * dk], v BF16 [T, v_heads * dv], log decays g and
    strengths beta FP32 [T, v_heads] -> out BF16 [T, v_heads * dv].  state: FP32 [slots, v_heads, dv, dk], a slot's
    values contiguous; a token turns S (the transpose of a head's dv x dk) into exp(g) S + k (beta (v - exp(g) S^T k))^T and
    gives scale S^T q (scale: 1 / sqrt(dk) by default), q and k divided by their norms first unless l2norm is false.

    seq_ptr, src, dst, tree_mask, lens, rows: as for short_conv(); prompts, single tokens and accepted paths move the
    states from src to dst, chains and trees of drafted tokens leave them (no dst).  With outputs false only the states move on,
    and q may be None.  ws: gated_delta_workspace(); allocated here when omitted and of use (for trees, from DELTA_CHUNK_FROM rows a
    sequence on, or where a long sequence can share the call with short ones; an empty one, with fewer rows, takes all tokens one by one).
    A sequence's result does not depend on those that share its call.  Returns out (None without outputs)."""
    slots, h, dv, dk = _delta_state(state)
    t, kw = _matrix2(k, "k")
    _device(q, k, v, g, beta, state, seq_ptr, src, dst, tree_mask, lens, rows, out, ws)
    if out is not None and not outputs:
        raise ValueError("out without outputs")
    if outputs and q is None:
        raise ValueError("outputs need q")
    hk = kw // dk
    if hk * dk != kw or hk == 0 or h % hk:
        raise ValueError(f"k: {kw} columns are not whole heads of {dk} that {h} value heads can share")
    if not outputs:
        q = None
    b = src.numel()
    chunks = (tree_mask is not None or t >= b * (DELTA_CHUNK_FROM if lens is None else DELTA_CHUNK_FROM_LENS) or
              (lens is None and t - b + 1 >= DELTA_CHUNK_LONG))
    if (outputs and out is None) or (chunks and ws is None):
        with _on(stream):
            if outputs and out is None:
                out = torch.empty(t, h * dv, dtype=_BF16, device=k.device)
            if chunks and ws is None:
                ws = gated_delta_workspace(t, b, state)
    ld_k = _rows(k, "k", (t, kw), (_BF16,), 8)
    ld_v = _rows(v, "v", (t, h * dv), (_BF16,), 8)
    ld_g = _rows(g, "g", (t, h), (_F32,), 1)
    ld_b = _rows(beta, "beta", (t, h), (_F32,), 1)
    ld_q = ld_o = 0
    if outputs:
        ld_q = _rows(q, "q", (t, kw), (_BF16,), 8)
        ld_o = _rows(out, "out", (t, h * dv), (_BF16,), 8)
    slot, head, column, one = state.stride()
    if one != 1 or column != dk or (head != dv * dk and h > 1):
        raise ValueError("state: a slot's values must be contiguous")
    if slots == 1:
        slot = h * dv * dk                        # a single slot is never stepped
    s = _sequences(t, slots, seq_ptr, src, dst, tree_mask, lens, rows)
    a = _DeltaArgs(hk, h, dk, dv, int(l2norm), eps, dk ** -0.5 if scale is None else scale, 0, _ptr(q), ld_q,
                   k.data_ptr(), ld_k, v.data_ptr(), ld_v, g.data_ptr(), ld_g, beta.data_ptr(), ld_b, state.data_ptr(), slot,
                   _ptr(out), ld_o)
    wsp, wsb = (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())
    _check("w12_gated_delta", lib().w12_gated_delta(ctypes.byref(a), ctypes.byref(s), wsp, wsb, _raw_stream(stream)))
    return out


def verify_draft_workspace_size(t: int, requests: int, vocab: int) -> int:
    b = _c_u64()
    _check("w12_verify_draft_workspace_size", lib().w12_verify_draft_workspace_size(t, requests, vocab, ctypes.byref(b)))
    return b.value


def verify_draft_workspace(t: int, requests: int, vocab: int, device="cuda") -> torch.Tensor:
    """A workspace for verify_draft() of at most t rows of this many requests over this vocabulary."""
    if torch.device(device).type != "cuda":
        raise ValueError("tensors must live on the GPU (libw12 has no CPU path)")
    return torch.empty(verify_draft_workspace_size(t, requests, vocab), dtype=torch.uint8, device=device)


def verify_draft(logits: torch.Tensor, tokens: torch.Tensor, u: torch.Tensor, node_ptr: torch.Tensor,
                 tree_mask: torch.Tensor | None = None, q: torch.Tensor | None = None, accept_u: torch.Tensor | None = None,
                 temperature: torch.Tensor | None = None, path: torch.Tensor | None = None, count: torch.Tensor | None = None,
                 next_token: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None) -> tuple:
    """Verification of drafted tokens against the target's probabilities (w12_verify_draft): logits [T, vocab]
    (FP32 or BF16), the rows' tokens int32 [T] and random numbers u FP32 [T] in [0, 1) -> (path, count, next_token).

    Request b has the nodes node_ptr[b] .. node_ptr[b + 1] - 1 (int32 [B + 1]), node 0 its last known token; tree_mask
    (int64 [T, words]) as for tree_attention(), None: chains.  temperature: FP32 [B], 0 for the largest logit; 1 when omitted.
    Without q, every row takes a token by its u, and the walk follows the children that have it.  With q (FP32 [T, vocab], the
    distributions that the rows' tokens were drawn from, chains only) and accept_u (FP32 [T]), nodes are accepted or rejected
    one after another, and next_token comes from what the target has over the draft.
    path (int32 [T], a request's accepted rows from its node_ptr on, then -1) and count (int32 [B]) are what short_conv() and
    gated_delta() take as rows and lens; next_token: int32 [B].  ws: verify_draft_workspace(); allocated here when omitted."""
    t, v = _matrix2(logits, "logits")
    _device(logits, tokens, u, node_ptr, tree_mask, q, accept_u, temperature, path, count, next_token, ws)
    b = node_ptr.numel() - 1
    if b < 1:
        raise ValueError("node_ptr: expected at least two values")
    if path is None or count is None or next_token is None or ws is None:
        with _on(stream):
            ints = dict(dtype=_I32, device=logits.device)
            path = torch.empty(t, **ints) if path is None else path
            count = torch.empty(b, **ints) if count is None else count
            next_token = torch.empty(b, **ints) if next_token is None else next_token
            ws = verify_draft_workspace(t, b, v, logits.device) if ws is None else ws
    ld_l = _rows(logits, "logits", (t, v), _FLOATS, 4 if logits.dtype == _F32 else 8)
    _vector(tokens, "tokens", t, _I32)
    _vector(node_ptr, "node_ptr", b + 1, _I32)
    _vector(u, "u", t, _F32)
    ld_q = words = ld_m = 0
    if q is not None:
        ld_q = _rows(q, "q", (t, v), (_F32,), 4)
    if accept_u is not None:
        _vector(accept_u, "accept_u", t, _F32)
    if temperature is not None:
        _vector(temperature, "temperature", b, _F32)
    if tree_mask is not None:
        words = _matrix2(tree_mask, "tree_mask")[1]
        ld_m = _rows(tree_mask, "tree_mask", (t, words), _MASKS, 1)
    _vector(path, "path", t, _I32)
    _vector(count, "count", b, _I32)
    _vector(next_token, "next_token", b, _I32)
    a = _VerifyDraftArgs(t, b, v, _FLOATS[logits.dtype], logits.data_ptr(), ld_l, _ptr(q), ld_q, tokens.data_ptr(),
                         node_ptr.data_ptr(), _ptr(tree_mask), ld_m, words, 0, u.data_ptr(), _ptr(accept_u), _ptr(temperature),
                         path.data_ptr(), count.data_ptr(), next_token.data_ptr())
    _check("w12_verify_draft", lib().w12_verify_draft(ctypes.byref(a), ws.data_ptr(), ws.numel() * ws.element_size(),
                                                      _raw_stream(stream)))
    return path, count, next_token
