"""GPU tests of the operators around the products at the ends of their ranges, against their formulas in 64 bits."""
import pytest
import torch

import lossless_bit_weight_encode_amd as w12

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
E24, Q4 = 2.0 ** -24, 2.0 ** -4


def rnd(seed, *shape, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale


@pytest.mark.parametrize("rt", [F32, BF])
def test_norm_blocks_whose_scale_is_subnormal_or_rounds_to_zero(rt):
    """Blocks of 128 with largest magnitudes from 1e-45 to 1e-36 beside zeros, in rows with one large value: finite
    outputs that stand for the values.  The scale is off by half the smallest FP32 step, 2^-150, which its largest
    multiple, 448, carries into a value (cut off, or lost with a scale of 0); y itself has such steps."""
    n, m = 640, 12
    r = torch.zeros(m, n)
    r[:, 0] = 1000.0
    for i in range(m):
        r[i, 128:180] = rnd(i, 52).clamp(-1, 1) * 10.0 ** (-43.5 + 0.75 * i)      # y: 0.0253 times that
    r = r.to(rt)
    w = torch.ones(n)
    w[256:384] = 1e-40                  # tiny weights, over zeros and over the values set next
    w[384:512] = 0
    r[:, 300:310] = 0.01
    w = w.to(BF)
    y = torch.empty(m, n, dtype=BF, device="cuda")
    yq = torch.empty(m, n, dtype=F8, device="cuda")
    sc = torch.empty(m, 5, device="cuda")
    w12.add_rmsnorm(r.cuda(), w.cuda(), y=y, yq=yq, yq_scale=sc, eps=1e-6)
    assert y.isfinite().all() and yq.float().isfinite().all(), "NaN from finite rows"
    x = r.double()
    ref = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6) * w.double()
    sc, yq = sc.cpu().double(), yq.cpu().double()
    least = ref.view(m, 5, 128).abs().amax(2) / 448
    assert (sc > 0).all() and sc.isfinite().all()
    assert (sc[(least == 0)] == 1).all()
    got = yq * sc.repeat_interleave(128, 1)
    tol = (Q4 + 4 * (n + 12) * E24) * ref.abs() + 2.0 ** -10 * least.repeat_interleave(128, 1) + 450 * 2.0 ** -149
    assert ((got - ref).abs() <= tol).all()
    assert (yq[ref == 0] == 0).all()
    # and a product of these rows is finite
    w8 = rnd(99, 128, n, scale=50.0).clamp(-448, 448).to(F8).cuda()
    out = w12.gemm_e4m3(yq.to(F8).cuda(), sc.float().cuda(), w8, torch.full((1, 5), 1e-3, device="cuda"))
    assert out.isfinite().all()


def test_attention_with_decreasing_ranges_stays_inside_its_workspace():
    """Ranges 0..T, T..0, 0..T ... overlap: 16000 items of short requests and 450 of a long one whose chunks leave
    partial results, where the workspace has 10080 places.  What the rows get is open; nothing behind the
    workspace, the output and lse is touched, and the next call is right."""
    t, requests, heads, d, page, long = 512, 1000, 8, 64, 64, 910
    k, v = (torch.randn(4, page, heads, d, dtype=BF, device="cuda") for _ in range(2))
    cache = w12.KVCache(k, v)
    q = torch.randn(t, heads * d, dtype=BF, device="cuda")
    ptr = torch.zeros(requests + 1, dtype=torch.int32, device="cuda")
    ptr[1::2] = t
    ctx = torch.zeros(requests, dtype=torch.int32, device="cuda")
    ctx[long] = 3000 * page
    table = torch.zeros(requests, 3010, dtype=torch.int32, device="cuda")
    need = w12.tree_attention_workspace_size(t, requests, heads, cache)
    guard = 8 << 20
    ws = torch.full((need + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.empty(2 * t, heads * d, dtype=BF, device="cuda").fill_(7.0)
    lse = torch.full((2 * t, heads), 7.0, device="cuda")
    torch.cuda.synchronize()
    w12.tree_attention(q, cache, table, ctx, ptr, out=out[:t], lse=lse[:t], ws=ws[:need])
    torch.cuda.synchronize()
    assert (ws[need:] == 0x5A).all() and (out[t:] == 7).all() and (lse[t:] == 7).all()
    # one request of all rows over the first page, as a chain behind 64 tokens
    p1, c1 = torch.tensor([0, t], dtype=torch.int32, device="cuda"), torch.tensor([64], dtype=torch.int32, device="cuda")
    t1 = (torch.arange(9, dtype=torch.int32, device="cuda") % 4)[None].contiguous()
    got = w12.tree_attention(q, cache, t1, c1, p1).cpu().double().view(t, heads, d)
    kk, vv = (x.cpu().double()[t1[0].long().cpu()].reshape(-1, heads, d)[:64 + t] for x in (k, v))
    for row in (0, 1, 255, 511):
        s = torch.einsum("hd,thd->ht", q[row].cpu().double().view(heads, d), kk[:65 + row]) * d ** -0.5
        p = torch.softmax(s, 1)
        ref, mag = torch.einsum("ht,thd->hd", p, vv[:65 + row]), torch.einsum("ht,thd->hd", p, vv[:65 + row].abs())
        # the result and p rounded to BF16 (2^-8 each); scores and sums of hundreds of terms in FP32
        assert ((got[row] - ref).abs() <= ref.abs() * 2.0 ** -8 + mag * (2.0 ** -8 * 1.01 + 4 * 1024 * E24)).all()


def test_one_workspace_serves_fewer_rows():
    """A workspace for the most rows, used by calls of other paths and tilings one after another: the bits of a call
    with its own."""
    n, k = 5120, 4352
    w = rnd(1, n, k, scale=50.0).clamp(-448, 448).to(F8).cuda()
    x = rnd(2, 600, k, scale=50.0).clamp(-448, 448).to(F8).cuda()
    xs, wsc = torch.rand(600, 34, device="cuda") * 1e-2, torch.rand(40, 34, device="cuda") * 1e-2
    ws = w12.gemm_e4m3_workspace(600, n, k)
    for m in (600, 1, 512, 64, 4, 65, 5, 300, 1):
        a = w12.gemm_e4m3(x[:m], xs[:m], w, wsc, ws=ws)
        assert torch.equal(a, w12.gemm_e4m3(x[:m], xs[:m], w, wsc)), m
        assert (ws[:16384] == 0).all(), "counters are left at zero"


def test_a_workspace_belongs_to_its_stream():
    """The clearing kernel runs on the given stream, so the memory has to be that stream's: what the current stream
    freed may still be in use by kernels that it has in flight."""
    s = torch.cuda.Stream()
    ws = w12.gemm_e4m3_workspace(1, 5120, 17408, stream=s)
    owners = [g["stream"] for g in torch.cuda.memory_snapshot()
              if g["address"] <= ws.data_ptr() < g["address"] + g["total_size"]]
    assert owners == [s.cuda_stream]
