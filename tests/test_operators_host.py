"""Host-side checks of the operators around the products: bad arguments are refused before a GPU is touched.
The pointers here are made up and never read."""
import ctypes

import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from lossless_bit_weight_encode_amd import _lib as L

INVALID, SHAPE, SMALL, MISALIGNED = -1, -2, -3, -5


def _set(s, kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def norm(**kw):
    a = L._NormArgs()
    a.M, a.N, a.residual_dtype, a.delta_dtype, a.eps = 4, 100, 0, 1, 1e-6
    a.residual, a.ld_residual, a.delta, a.ld_delta, a.weight = 0x1000, 104, 0x2000, 100, 0x3000
    a.residual_out, a.ld_residual_out, a.y, a.ldy = 0x1000, 104, 0x4000, 104
    a.yq, a.ldyq, a.yq_scale, a.ld_scale = 0x5000, 112, 0x6000, 1
    return w12.lib().w12_add_rmsnorm(ctypes.byref(_set(a, kw)), None)


@pytest.mark.parametrize("code,kw", [
    (SHAPE, dict(M=0)), (SHAPE, dict(M=(1 << 20) + 1)), (SHAPE, dict(N=0)), (SHAPE, dict(N=65537, ld_residual=65544)),
    (INVALID, dict(residual=None)), (INVALID, dict(weight=None)), (INVALID, dict(residual_dtype=2)),
    (INVALID, dict(delta_dtype=7)), (INVALID, dict(ld_residual=96)), (INVALID, dict(ld_delta=96)),
    (MISALIGNED, dict(ld_residual=102)), (MISALIGNED, dict(ld_delta=102)), (MISALIGNED, dict(residual=0x1004)),
    (MISALIGNED, dict(delta=0x2008)), (MISALIGNED, dict(weight=0x3002)), (INVALID, dict(ld_residual_out=112)),
    (MISALIGNED, dict(y=0x4002)), (INVALID, dict(ldy=96)), (MISALIGNED, dict(ldyq=104)), (INVALID, dict(ldyq=96)),
    (INVALID, dict(ld_scale=0)), (MISALIGNED, dict(yq_scale=0x6002)), (INVALID, dict(yq_scale=None)),
    (INVALID, dict(yq=None)), (INVALID, dict(y=None, yq=None, yq_scale=None, delta=None)),
    (INVALID, dict(y=None, yq=None, yq_scale=None, residual_out=None)), (INVALID, dict(eps=-1.0)),
    (INVALID, dict(eps=float("nan"))), (INVALID, dict(reserved=1)), (SHAPE, dict(ld_delta=1 << 40)),
])
def test_norm_refusals(code, kw):
    assert norm(**kw) == code
    assert w12.lib().w12_last_error()


def cache(**kw):
    c = L._KVCache()
    c.dtype, c.pages, c.page_size, c.heads, c.dim = 0, 10, 16, 2, 64
    c.page_stride, c.token_stride, c.head_stride, c.k, c.v = 16 * 128, 128, 64, 0x10000, 0x20000
    return _set(c, kw)


BAD_CACHES = [
    (INVALID, dict(dtype=1)), (SHAPE, dict(pages=0)), (SHAPE, dict(page_size=24)), (SHAPE, dict(page_size=2048)),
    (SHAPE, dict(page_size=0)), (SHAPE, dict(heads=0)), (SHAPE, dict(dim=96)), (INVALID, dict(k=None)),
    (INVALID, dict(v=None)), (MISALIGNED, dict(k=0x10008)), (MISALIGNED, dict(token_stride=132)),
    (INVALID, dict(page_stride=-2048)), (SHAPE, dict(page_stride=1 << 45)), (INVALID, dict(dtype=2, k_scale=None)),
    (MISALIGNED, dict(dtype=2, token_stride=136, k_scale=0x100, v_scale=0x200)),
    (MISALIGNED, dict(dtype=2, k_scale=0x102, v_scale=0x200)), (INVALID, dict(reserved=3)),
]


def rope(c=None, **kw):
    a = L._RopeArgs()
    a.T, a.q_heads, a.src_dtype, a.rot_dim, a.axes, a.adjacent = 3, 4, 1, 64, 2, 0
    a.qkv, a.ld_qkv, a.positions, a.ld_positions, a.slots, a.inv_freq = 0x1000, 512, 0x2000, 3, 0x3000, 0x4000
    a.q, a.ldq = 0x5000, 256
    return w12.lib().w12_rope_append(ctypes.byref(_set(a, kw)), ctypes.byref(c or cache()), None)


@pytest.mark.parametrize("code,kw", BAD_CACHES)
def test_rope_refuses_bad_caches(code, kw):
    assert rope(cache(**kw)) == code


@pytest.mark.parametrize("code,kw", [
    (SHAPE, dict(T=0)), (SHAPE, dict(q_heads=0)), (INVALID, dict(src_dtype=2)), (SHAPE, dict(rot_dim=63)),
    (SHAPE, dict(rot_dim=66)), (SHAPE, dict(rot_dim=-2)), (SHAPE, dict(axes=0)), (SHAPE, dict(axes=9)),
    (INVALID, dict(ld_qkv=504)), (MISALIGNED, dict(ld_qkv=514)), (MISALIGNED, dict(qkv=0x1008)), (INVALID, dict(q=None)),
    (INVALID, dict(ldq=248)), (INVALID, dict(positions=None)), (INVALID, dict(ld_positions=2)),
    (INVALID, dict(inv_freq=None)), (MISALIGNED, dict(inv_freq=0x4004)), (INVALID, dict(slots=None)),
    (MISALIGNED, dict(slots=0x3004)),
])
def test_rope_refusals(code, kw):
    assert rope(**kw) == code


def attention(c=None, ws=0x100000, ws_bytes=1 << 40, **kw):
    a = L._AttentionArgs()
    a.T, a.requests, a.q_heads, a.max_pages, a.mask_words, a.scale = 5, 2, 4, 8, 1, 0.125
    a.q, a.ldq, a.node_ptr, a.ctx_len, a.page_table, a.ld_table = 0x1000, 256, 0x2000, 0x3000, 0x4000, 8
    a.tree_mask, a.ld_mask, a.out, a.ldo, a.lse, a.ld_lse = 0x5000, 1, 0x6000, 256, 0x7000, 4
    return w12.lib().w12_tree_attention(ctypes.byref(_set(a, kw)), ctypes.byref(c or cache()), ws, ws_bytes, None)


@pytest.mark.parametrize("code,kw", BAD_CACHES)
def test_attention_refuses_bad_caches(code, kw):
    assert attention(cache(**kw)) == code


@pytest.mark.parametrize("code,kw", [
    (SHAPE, dict(T=0)), (SHAPE, dict(requests=0)), (SHAPE, dict(requests=1025)), (SHAPE, dict(q_heads=3)),
    (SHAPE, dict(q_heads=130)), (SHAPE, dict(max_pages=0)), (SHAPE, dict(max_pages=1 << 27, ld_table=1 << 27)),
    (INVALID, dict(q=None)), (INVALID, dict(ldq=248)), (MISALIGNED, dict(ldq=258)), (MISALIGNED, dict(out=0x6008)),
    (INVALID, dict(out=None)), (INVALID, dict(page_table=None)), (INVALID, dict(ld_table=7)),
    (MISALIGNED, dict(page_table=0x4002)), (INVALID, dict(node_ptr=None)), (INVALID, dict(ctx_len=None)),
    (MISALIGNED, dict(node_ptr=0x2002)), (SHAPE, dict(mask_words=0)), (SHAPE, dict(mask_words=65, ld_mask=65)),
    (INVALID, dict(mask_words=2)), (MISALIGNED, dict(tree_mask=0x5004)), (INVALID, dict(tree_mask=None)),
    (INVALID, dict(ld_lse=3)), (MISALIGNED, dict(lse=0x7002)), (INVALID, dict(scale=0.0)),
    (INVALID, dict(scale=float("nan"))), (INVALID, dict(scale=float("inf"))), (MISALIGNED, dict(ws=0x100004)),
])
def test_attention_refusals(code, kw):
    assert attention(**kw) == code


def test_attention_workspace_checks():
    need = ctypes.c_uint64()
    size = w12.lib().w12_tree_attention_workspace_size
    assert size(5, 2, 4, ctypes.byref(cache()), ctypes.byref(need)) == 0
    assert size(5, 2, 4, ctypes.byref(cache()), None) == INVALID
    assert size(0, 2, 4, ctypes.byref(cache()), ctypes.byref(need)) == SHAPE
    if need.value:
        assert attention(ws_bytes=need.value - 1) == SMALL
        assert attention(ws=None) == INVALID


def gemm(**kw):
    p = dict(X=0x1000, M=4, ldx=208, xs=0x2000, ldxs=2, W=0x3000, N=70, K=200, ldw=208, wsc=0x4000, ldws=2, Y=0x5000,
             ldy=70, ws=0x100000, ws_bytes=1 << 40)
    p.update(kw)
    return w12.lib().w12_gemm_e4m3(*p.values(), None)


@pytest.mark.parametrize("code,kw", [
    (SHAPE, dict(M=0)), (SHAPE, dict(M=4097)), (SHAPE, dict(N=0)), (SHAPE, dict(K=0)), (SHAPE, dict(K=65537)),
    (INVALID, dict(X=None)), (INVALID, dict(W=None)), (INVALID, dict(xs=None)), (INVALID, dict(wsc=None)),
    (INVALID, dict(Y=None)), (INVALID, dict(ldx=192)), (MISALIGNED, dict(ldx=200)), (MISALIGNED, dict(ldw=204)),
    (MISALIGNED, dict(X=0x1008)), (MISALIGNED, dict(W=0x3004)), (INVALID, dict(ldxs=1)), (INVALID, dict(ldws=1)),
    (MISALIGNED, dict(xs=0x2002)), (INVALID, dict(ldy=69)), (MISALIGNED, dict(Y=0x5002)), (SHAPE, dict(ldx=1 << 30)),
    (SHAPE, dict(ldw=1 << 26)), (SHAPE, dict(ldy=1 << 28)), (MISALIGNED, dict(ws=0x100008)),
])
def test_gemm_e4m3_refusals(code, kw):
    assert gemm(**kw) == code


def test_gemm_e4m3_workspace_checks():
    need = w12.gemm_e4m3_workspace_size(4, 70, 200)
    with pytest.raises(w12.W12Error):
        w12.gemm_e4m3_workspace_size(0, 70, 200)
    if need:
        assert gemm(ws_bytes=need - 1) == SMALL
        assert gemm(ws=None) == INVALID


def test_binding_refuses_cpu_tensors():
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    with pytest.raises(ValueError, match="GPU"):
        w12.add_rmsnorm(torch.zeros(2, 64, dtype=bf), torch.ones(64, dtype=bf), y=torch.zeros(2, 64, dtype=bf))
    with pytest.raises(ValueError, match="GPU"):
        w12.KVCache(torch.zeros(2, 16, 1, 64, dtype=bf), torch.zeros(2, 16, 1, 64, dtype=bf))
    with pytest.raises(ValueError, match="GPU"):
        w12.gemm_e4m3(torch.zeros(2, 128).to(f8), torch.ones(2, 1), torch.zeros(8, 128).to(f8), torch.ones(1, 1),
                      y=torch.zeros(2, 8), ws=torch.zeros(16))


def test_cache_handle_refusals():
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    k = torch.zeros(2, 16, 1, 64, dtype=bf)
    with pytest.raises(ValueError, match="shape"):
        w12.KVCache(k, k[:1])
    with pytest.raises(TypeError):
        w12.KVCache(k, k.float())
    with pytest.raises(ValueError, match="strides"):
        w12.KVCache(k, torch.zeros(2, 16, 1, 128, dtype=bf)[..., ::2])
    with pytest.raises(ValueError, match="k_scale"):
        w12.KVCache(k.to(f8), k.to(f8))
    with pytest.raises(ValueError, match="k_scale"):
        w12.KVCache(k, k, torch.ones(1), torch.ones(1))
    with pytest.raises(ValueError, match="k_scale"):
        w12.KVCache(k.to(f8), k.to(f8), torch.ones(2), torch.ones(2))
