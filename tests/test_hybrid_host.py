"""Host-side checks of the hybrid target's operators: bad arguments are refused before a GPU is touched.  The pointers
here are made up and never read."""
import contextlib
import ctypes
import os
import random
import re

import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from hybrid_util import delta_bounds, delta_steps, tree
from lossless_bit_weight_encode_amd import _lib as L

INVALID, SHAPE, SMALL, MISALIGNED = -1, -2, -3, -5


def _set(s, kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def seqs(**kw):
    s = L._Sequences()
    s.T, s.count, s.slots = 5, 2, 4
    s.ptr, s.src, s.dst = 0x1000, 0x1100, 0x1200
    return _set(s, kw)


TREE = dict(dst=None, tree_mask=0x2000, ld_mask=1, mask_words=1)
BAD_SEQS = [
    (SHAPE, dict(T=0)), (SHAPE, dict(T=(1 << 20) + 1)), (SHAPE, dict(count=0)), (SHAPE, dict(count=1025)),
    (SHAPE, dict(slots=0)), (SHAPE, dict(slots=(1 << 20) + 1)), (INVALID, dict(ptr=None)), (INVALID, dict(src=None)),
    (MISALIGNED, dict(ptr=0x1002)), (MISALIGNED, dict(src=0x1101)), (MISALIGNED, dict(dst=0x1202)),
    (MISALIGNED, dict(lens=0x1302)), (MISALIGNED, dict(rows=0x1303)), (INVALID, dict(mask_words=1)),
    (INVALID, dict(TREE, dst=0x1200)), (INVALID, dict(TREE, rows=0x1300)), (INVALID, dict(TREE, lens=0x1300)),
    (SHAPE, dict(TREE, mask_words=0)), (SHAPE, dict(TREE, mask_words=65, ld_mask=65)), (INVALID, dict(TREE, mask_words=2)),
    (MISALIGNED, dict(TREE, tree_mask=0x2004)),
]


def conv(s=None, **kw):
    a = L._ConvArgs()
    a.channels, a.width, a.dtype, a.silu = 100, 4, 1, 1
    a.x, a.ldx, a.weight, a.state, a.slot_stride, a.tap_stride = 0x10000, 100, 0x20000, 0x30000, 300, 100
    a.y, a.ldy = 0x40000, 104
    return w12.lib().w12_short_conv(ctypes.byref(_set(a, kw)), ctypes.byref(s or seqs()), None)


def delta(s=None, ws=0x900000, ws_bytes=1 << 40, **kw):
    a = L._DeltaArgs()
    a.k_heads, a.v_heads, a.dk, a.dv, a.l2norm, a.eps, a.scale = 2, 4, 64, 128, 1, 1e-6, 0.125
    a.q, a.ldq, a.k, a.ldk, a.v, a.ldv = 0x10000, 128, 0x20000, 128, 0x30000, 512
    a.g, a.ldg, a.beta, a.ldbeta = 0x40000, 4, 0x50000, 4
    a.state, a.slot_stride, a.out, a.ldo = 0x60000, 4 * 128 * 64, 0x70000, 512
    return w12.lib().w12_gated_delta(ctypes.byref(_set(a, kw)), ctypes.byref(s or seqs()), ws, ws_bytes, None)


@pytest.mark.parametrize("code,kw", BAD_SEQS)
@pytest.mark.parametrize("call", [conv, delta])
def test_sequences_are_refused(call, code, kw):
    assert call(seqs(**kw)) == code
    assert w12.lib().w12_last_error()


@pytest.mark.parametrize("code,kw", [
    (SHAPE, dict(channels=0)), (SHAPE, dict(channels=(1 << 17) + 1)), (SHAPE, dict(width=1)), (SHAPE, dict(width=5)),
    (INVALID, dict(dtype=2)), (INVALID, dict(x=None)), (INVALID, dict(ldx=96)), (MISALIGNED, dict(ldx=102)),
    (MISALIGNED, dict(x=0x10008)), (INVALID, dict(weight=None)), (MISALIGNED, dict(weight=0x20002)),
    (MISALIGNED, dict(bias=0x20001)), (INVALID, dict(state=None)), (MISALIGNED, dict(state=0x30008)),
    (INVALID, dict(tap_stride=96)), (MISALIGNED, dict(tap_stride=102)), (SHAPE, dict(tap_stride=1 << 41, slot_stride=1 << 43)),
    (INVALID, dict(slot_stride=296)), (MISALIGNED, dict(slot_stride=302)), (SHAPE, dict(slot_stride=1 << 42)),
    (MISALIGNED, dict(y=0x40008)), (INVALID, dict(ldy=96)), (MISALIGNED, dict(dtype=0, ldx=100, tap_stride=104, slot_stride=312)),
])
def test_conv_refusals(code, kw):
    assert conv(**kw) == code


def test_nothing_wanted_is_refused():
    assert conv(seqs(dst=None), y=None) == INVALID
    assert delta(seqs(dst=None), q=None, out=None) == INVALID


@pytest.mark.parametrize("code,kw", [
    (SHAPE, dict(v_heads=0)), (SHAPE, dict(v_heads=1025)), (SHAPE, dict(k_heads=0)), (SHAPE, dict(k_heads=3)),
    (SHAPE, dict(dk=96)), (SHAPE, dict(dk=256)), (SHAPE, dict(dv=96)), (INVALID, dict(reserved=1)),
    (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(scale=float("inf"))),
    (INVALID, dict(scale=float("nan"))), (INVALID, dict(q=None)), (INVALID, dict(out=None)), (INVALID, dict(k=None)),
    (INVALID, dict(v=None)), (INVALID, dict(g=None)), (INVALID, dict(beta=None)), (INVALID, dict(ldq=120)),
    (INVALID, dict(ldk=120)), (MISALIGNED, dict(ldk=130)), (INVALID, dict(ldv=504)), (MISALIGNED, dict(v=0x30008)),
    (INVALID, dict(ldg=3)), (INVALID, dict(ldbeta=3)), (MISALIGNED, dict(g=0x40002)), (MISALIGNED, dict(beta=0x50001)),
    (INVALID, dict(state=None)), (MISALIGNED, dict(state=0x60004)), (INVALID, dict(slot_stride=4 * 128 * 64 - 4)),
    (MISALIGNED, dict(slot_stride=4 * 128 * 64 + 2)), (SHAPE, dict(slot_stride=1 << 41)), (INVALID, dict(ldo=504)),
    (MISALIGNED, dict(out=0x70008)), (MISALIGNED, dict(ws=0x900004)),
])
def test_delta_refusals(code, kw):
    assert delta(**kw) == code


def verify(ws=0x900000, ws_bytes=1 << 50, **kw):
    a = L._VerifyDraftArgs()
    a.T, a.requests, a.vocab, a.logits_dtype, a.logits, a.ld_logits = 5, 2, 1000, 1, 0x10000, 1000
    a.tokens, a.node_ptr, a.u, a.path, a.count, a.next_token = 0x1000, 0x1100, 0x1200, 0x1300, 0x1400, 0x1500
    return w12.lib().w12_verify_draft(ctypes.byref(_set(a, kw)), ws, ws_bytes, None)


Q = dict(q=0x20000, ldq=1000, accept_u=0x1600)


@pytest.mark.parametrize("code,kw", [
    (SHAPE, dict(T=0)), (SHAPE, dict(T=(1 << 20) + 1)), (SHAPE, dict(requests=0)), (SHAPE, dict(requests=1025)),
    (SHAPE, dict(vocab=0)), (SHAPE, dict(vocab=(1 << 24) + 1)), (SHAPE, dict(T=1 << 20, vocab=1 << 20, ld_logits=1 << 20)),
    (INVALID, dict(reserved=1)), (INVALID, dict(logits_dtype=2)), (INVALID, dict(logits=None)), (INVALID, dict(ld_logits=996)),
    (MISALIGNED, dict(ld_logits=1002)), (MISALIGNED, dict(logits=0x10004)), (INVALID, dict(Q, ldq=996)),
    (MISALIGNED, dict(Q, q=0x20004)), (INVALID, dict(Q, accept_u=None)), (INVALID, dict(accept_u=0x1600)),
    (INVALID, dict(Q, tree_mask=0x2000, ld_mask=1, mask_words=1)), (INVALID, dict(mask_words=1)),
    (SHAPE, dict(tree_mask=0x2000, ld_mask=65, mask_words=65)), (MISALIGNED, dict(tree_mask=0x2004, ld_mask=1, mask_words=1)),
    (INVALID, dict(tokens=None)), (INVALID, dict(node_ptr=None)), (INVALID, dict(u=None)), (INVALID, dict(path=None)),
    (INVALID, dict(count=None)), (INVALID, dict(next_token=None)), (MISALIGNED, dict(u=0x1202)),
    (MISALIGNED, dict(Q, accept_u=0x1602)), (MISALIGNED, dict(temperature=0x1702)), (MISALIGNED, dict(path=0x1302)),
    (SMALL, dict(ws_bytes=16)), (INVALID, dict(ws=None)), (MISALIGNED, dict(ws=0x900008)),
])
def test_verify_refusals(code, kw):
    assert verify(**kw) == code


def test_workspaces_serve_fewer_rows():
    for h, dk, dv in ((48, 128, 128), (1, 64, 64)):
        sizes = [w12.gated_delta_workspace_size(t, c, h, dk, dv) for t, c in ((1, 1), (2, 1), (64, 1), (64, 8), (65, 64), (4096, 64), (4097, 1024))]
        assert sizes == sorted(sizes)
    sizes = [w12.verify_draft_workspace_size(t, b, 50257) for t, b in ((1, 1), (17, 1), (17, 4), (384, 16), (4096, 1024))]
    assert sizes == sorted(sizes) and sizes[0] > 0


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return getattr(L.lib(), name)
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def recorder(monkeypatch):
    """The bindings with neither library nor GPU behind them."""
    from lossless_bit_weight_encode_amd import _hybrid, _ops
    rec = _Recorder()
    monkeypatch.setattr(_hybrid, "lib", lambda: rec)
    monkeypatch.setattr(_ops, "_current_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    return rec


def _z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


CALLS = {
    "conv": lambda: w12.short_conv(_z(2, 8), _z(8, 4, dtype=torch.bfloat16), _z(1, 3, 8), _z(2, dtype=torch.int32), _z(1, dtype=torch.int32)),
    "delta": lambda: w12.gated_delta(*(_z(2, 64, dtype=torch.bfloat16) for _ in range(3)), _z(2, 1), _z(2, 1), _z(1, 1, 64, 64),
                                     _z(2, dtype=torch.int32), _z(1, dtype=torch.int32)),
    "verify": lambda: w12.verify_draft(_z(2, 100), _z(2, dtype=torch.int32), _z(2), _z(2, dtype=torch.int32)),
}


@pytest.mark.parametrize("name", CALLS)
def test_nothing_is_launched_before_the_tensors_are_checked(recorder, monkeypatch, name):
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(a) or empty(*a, **k))
    with pytest.raises(ValueError, match="GPU"):
        CALLS[name]()
    assert recorder.calls == [] and made == []


@pytest.fixture
def anywhere(recorder, monkeypatch):
    """As recorder, with tensors of any device taken for the current GPU's."""
    from lossless_bit_weight_encode_amd import _hybrid
    monkeypatch.setattr(_hybrid, "_device", lambda *a: 0)
    return recorder


I32, BF = torch.int32, torch.bfloat16


def _conv(x=None, weight=None, state=None, ptr=None, src=None, **kw):
    z = lambda t, *s, dtype=torch.float32: _z(*s, dtype=dtype) if t is None else t
    return w12.short_conv(z(x, 2, 8), z(weight, 8, 4, dtype=BF), z(state, 1, 3, 8), z(ptr, 2, dtype=I32), z(src, 1, dtype=I32), **kw)


def _delta(k=None, g=None, state=None, src=None, q="as k", **kw):
    z = lambda t, *s, dtype=torch.float32: _z(*s, dtype=dtype) if t is None else t
    k = z(k, 2, 64, dtype=BF)
    return w12.gated_delta(_z(2, 64, dtype=BF) if isinstance(q, str) else q, k, _z(2, 128, dtype=BF), z(g, 2, 2), _z(2, 2), z(state, 1, 2, 64, 64),
                           _z(2, dtype=I32), z(src, 1, dtype=I32), **kw)


def _verify(logits=None, tokens=None, **kw):
    return w12.verify_draft(_z(2, 100) if logits is None else logits, _z(2, dtype=I32) if tokens is None else tokens, _z(2),
                            _z(2, dtype=I32), ws=_z(1 << 16, dtype=torch.uint8), **kw)


@pytest.mark.parametrize("call", [
    lambda: _conv(x=_z(2, 8, dtype=torch.float16)), lambda: _conv(weight=_z(7, 4, dtype=BF)), lambda: _conv(weight=_z(8, 4)),
    lambda: _conv(state=_z(1, 2, 8)), lambda: _conv(state=_z(1, 3, 8, dtype=BF)), lambda: _conv(ptr=_z(3, dtype=I32)),
    lambda: _conv(src=_z(1, dtype=torch.int64)), lambda: _conv(bias=_z(7, dtype=BF)), lambda: _conv(lens=_z(2, dtype=I32)),
    lambda: _conv(rows=_z(1, dtype=I32)), lambda: _conv(y=_z(2, 8)), lambda: _conv(y=_z(2, 8, dtype=BF), outputs=False),
    lambda: _conv(tree_mask=_z(2, 1)), lambda: _conv(tree_mask=_z(3, 1, dtype=torch.int64)),
    lambda: _conv(state=_z(1, 8, 3).transpose(1, 2)),
    lambda: _delta(k=_z(2, 60, dtype=BF)), lambda: _delta(k=_z(2, 64)), lambda: _delta(k=_z(2, 192, dtype=BF)), lambda: _delta(g=_z(2, 3)),
    lambda: _delta(state=_z(1, 2, 64, 64, dtype=BF)), lambda: _delta(state=_z(2, 64, 64)), lambda: _delta(q=None),
    lambda: _delta(state=_z(1, 2, 64, 64).transpose(2, 3)), lambda: _delta(out=_z(2, 128)), lambda: _delta(src=_z(1)),
    lambda: _delta(out=_z(2, 128, dtype=BF), outputs=False), lambda: _delta(dst=_z(2, dtype=I32)),
    lambda: _verify(logits=_z(2, 100, dtype=torch.float16)), lambda: _verify(tokens=_z(2, dtype=torch.int64)),
    lambda: _verify(q=_z(2, 99), accept_u=_z(2)), lambda: _verify(q=_z(2, 100, dtype=BF), accept_u=_z(2)),
    lambda: _verify(temperature=_z(2)), lambda: _verify(path=_z(3, dtype=I32)), lambda: _verify(count=_z(2, dtype=I32)),
    lambda: _verify(next_token=_z(1, dtype=torch.int64)), lambda: _verify(tree_mask=_z(2, 1, dtype=I32)),
])
def test_binding_refuses(anywhere, call):
    with pytest.raises((ValueError, TypeError)):
        call()
    assert anywhere.calls == []


def test_binding_takes_what_is_right(anywhere):
    assert _conv().shape == (2, 8) and _delta().shape == (2, 128)
    _conv(outputs=False, dst=_z(1, dtype=I32), state=_z(1, 3, 16)[:, :, :8])
    _delta(q=None, outputs=False, dst=_z(1, dtype=I32))
    path, count, token = _verify(q=_z(2, 100), accept_u=_z(2))
    assert path.shape == (2,) and count.shape == (1,) and token.shape == (1,)
    assert anywhere.calls == ["w12_short_conv", "w12_gated_delta"] * 2 + ["w12_verify_draft"]


@pytest.mark.parametrize("n,parents", [(1, None), (150, None), (33, "tree")])
def test_bounds_cover_what_they_describe(n, parents):
    """The recurrence in 32 bits stays within the bounds that the kernels are held to."""
    gen = torch.Generator().manual_seed(n)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    parents = parents and tree(random.Random(n), n)
    q, k, v = (torch.nn.functional.silu(rnd(n, d)).bfloat16() for d in (64, 64, 32))
    args = [q, k, v, -torch.rand(n, generator=gen), torch.rand(n, generator=gen), rnd(64, 32)]
    wide = [x.double() for x in args] + [0.125, True, 1e-6]
    o, s = delta_steps(*wide, parents=parents)
    do, ds = delta_bounds(*wide, parents=parents)
    q, k = (x.float() / torch.sqrt((x.float() ** 2).sum(1, keepdim=True) + 1e-6) for x in (q, k))
    states = []
    for i in range(n):
        p = i - 1 if parents is None else parents[i]
        st = (args[5] if p < 0 else states[p]) * torch.exp(args[3][i])
        st = st + torch.outer(k[i], args[4][i] * (v[i].float() - st.t() @ k[i]))
        assert ((0.125 * (st.t() @ q[i])).bfloat16().double() - o[i]).abs().le(do[i]).all()
        states.append(st)
    if parents is None:
        assert (states[-1].double() - s).abs().le(ds).all()


def test_rows_from_which_gated_delta_needs_its_workspace():
    """The binding allocates where the library asks for it."""
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "w12.h")).read()
    for name in ("DELTA_CHUNK_FROM", "DELTA_CHUNK_FROM_LENS"):
        assert int(re.search(rf"#define W12_{name} (\d+)", text).group(1)) == getattr(w12, name)
