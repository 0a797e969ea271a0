"""GPU tests of the schedules that real sizes take: long shares of the 8-bit product, chunks and joins of the attention.
References are plain 64-bit computations on the GPU.

Tolerances count roundings, half a step each: 2^-8 of the value (BF16), 2^-24 (FP32); sums of n FP32 terms are off by
at most n 2^-24 of the sum of magnitudes, twice that where matrix instructions cut off."""
import math

import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from test_gpu_operators import ancestors, mask_tensor

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
B8, E24 = 2.0 ** -8, 2.0 ** -24


# ------------------------------------------------------------------------------------------ 8-bit product

def _e4m3(gen, rows, k):
    ld = (k + 15) // 16 * 16 + 16
    out = torch.empty(rows, ld, dtype=torch.uint8, device="cuda")
    for i in range(0, rows, 8192):
        part = torch.randn(min(8192, rows - i), ld, generator=gen, device="cuda") * 60
        out[i:i + 8192] = part.clamp_(-448, 448).to(F8).view(torch.uint8)
    out[:, k:] = 0x7F                   # NaN between the rows
    return out.view(F8)[:, :k]


# On 256 compute units: shares of 85, 85, 22, 22, 44, 67, 8, 7, 20, 8 steps over tiles of 40, 40, 40, 40, 71, 33, 136, 133, 9, 5
# (whole tiles, partial ones before and behind them, scales renewed inside a share, a last step that k ends in).
@pytest.mark.parametrize("m,n,k", [(512, 34816, 5120), (500, 34816, 5000), (63, 34816, 5120), (63, 34816, 5000), (40, 40000, 9000),
                                   (64, 131109, 4200), (1, 5120, 17408), (3, 5001, 17001), (130, 70000, 1100), (20, 100003, 600)])
def test_gemm_e4m3_long_shares(m, n, k):
    gen = torch.Generator("cuda").manual_seed(m + n + k)
    x, w = _e4m3(gen, m, k), _e4m3(gen, n, k)
    kb, nb = -(-k // 128), -(-n // 128)
    xs = torch.rand(m, kb, generator=gen, device="cuda") * 0.02 + 1e-3
    ws = torch.exp(torch.randn(nb, kb, generator=gen, device="cuda")) * 1e-3
    y = torch.full((m, n), float("nan"), device="cuda")
    wk = w12.gemm_e4m3_workspace(m, n, k)
    w12.gemm_e4m3(x, xs, w, ws, y=y, ws=wk)
    a = x.double() * xs.double().repeat_interleave(128, 1)[:, :k]
    for n0 in range(0, n, 16384):
        n1 = min(n, n0 + 16384)
        b = w[n0:n1].double() * ws[n0 // 128:-(-n1 // 128)].double().repeat_interleave(128, 1)[:, :k].repeat_interleave(128, 0)[:n1 - n0]
        tol = (a.abs() @ b.abs().t()) * (2 * (128 + kb + 8) * E24)
        over = (y[:, n0:n1].double() - a @ b.t()).abs() - tol
        assert not over.isnan().any() and over.max() <= 0, f"channels {n0}..{n1}: {int((over > 0).sum())} values"
    for _ in range(3):
        assert torch.equal(w12.gemm_e4m3(x, xs, w, ws, ws=wk), y), "not the same from run to run"


# -------------------------------------------------------------------------------------------------- attention

class Batch:
    """Requests over a paged cache on the GPU whose unused places are NaN, with a workspace of exactly the size asked for
    and a guard behind it."""

    def __init__(self, ctxs, nodes, hq, hkv, d, page=64, f8=False, tree=True, seed=0, qscale=1.5):
        gen = torch.Generator("cuda").manual_seed(seed)
        cpu = torch.Generator().manual_seed(seed)
        self.ctxs, self.nodes, self.hq, self.hkv, self.d, self.page = ctxs, nodes, hq, hkv, d, page
        need = [-(-(c + n) // page) for c, n in zip(ctxs, nodes)]
        order = torch.randperm(sum(need) + 2, generator=gen, device="cuda").int()
        self.table = torch.full((len(ctxs), max(need) + 1), -1, dtype=torch.int32, device="cuda")
        used = torch.zeros(sum(need) + 2, page, dtype=torch.bool, device="cuda")
        at = 0
        for b, p in enumerate(need):
            self.table[b, :p] = order[at:at + p]
            at += p
            tok = torch.arange(ctxs[b] + nodes[b], device="cuda")
            used[self.table[b].long()[tok // page], tok % page] = True
        kv, scales = [], []
        for _ in range(2):
            x = torch.randn(sum(need) + 2, page, hkv, d, generator=gen, device="cuda")
            if f8:
                s = 0.01 + 0.004 * torch.rand(hkv, generator=gen, device="cuda")
                x = (x / s[:, None]).clamp_(-448, 448)
                scales.append(s)
            x[~used] = float("nan")
            kv.append(x.to(F8 if f8 else BF))
        self.cache = w12.KVCache(*kv, *scales)
        self.ptr = [0]
        for n in nodes:
            self.ptr.append(self.ptr[-1] + n)
        self.q = (torch.randn(self.ptr[-1], hq * d, generator=gen, device="cuda") * qscale).to(BF)
        self.bits = self.mask = None
        if tree:
            self.bits = []
            for n in nodes:
                parents = [-1] + [int(torch.randint(max(0, i - 9), i, (1,), generator=cpu)) for i in range(1, n)]
                self.bits += ancestors(parents[:n])
            self.mask = mask_tensor(self.bits, -(-max(nodes) // 64)).cuda()

    def run(self):
        t = self.q.shape[0]
        need = w12.tree_attention_workspace_size(t, len(self.ctxs), self.hq, self.cache)
        ws = torch.full((need + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
        lse = torch.full((t, self.hq), float("nan"), device="cuda")
        ints = dict(dtype=torch.int32, device="cuda")
        out = w12.tree_attention(self.q, self.cache, self.table, torch.tensor(self.ctxs, **ints), torch.tensor(self.ptr, **ints),
                                 tree_mask=self.mask, lse=lse, ws=ws[:need])
        torch.cuda.synchronize()
        assert (ws[need:] == 0x5A).all(), "write behind the workspace"
        return out, lse

    def check(self, out, lse, per_request=5):
        d, g = self.d, self.hq // self.hkv
        pick = torch.Generator().manual_seed(1)
        assert out.isfinite().all() and lse.isfinite().all()
        for b, (ctx, n) in enumerate(zip(self.ctxs, self.nodes)):
            some = sorted({0, n - 1, *torch.randint(0, n, (per_request,), generator=pick).tolist()})
            rows = torch.tensor([self.ptr[b] + i for i in some], device="cuda")
            tok = torch.arange(ctx + n, device="cuda")
            page = self.table[b].long()[tok // self.page]
            see = torch.ones(len(some), ctx + n, dtype=torch.bool)
            for r, i in enumerate(some):
                m = self.bits[self.ptr[b] + i] if self.bits else (1 << (i + 1)) - 1
                see[r, ctx:] = torch.tensor([(m >> j) & 1 for j in range(n)], dtype=torch.bool)
            hide = ~see.cuda().repeat_interleave(g, 0)
            terms = (~hide).sum(1, keepdim=True)
            for h in range(self.hkv):
                k, v = ((x.view(torch.uint8)[page, tok % self.page, h].view(F8) if x.dtype == F8 else x[page, tok % self.page, h]).double()
                        for x in (self.cache.k, self.cache.v))
                if self.cache.k_scale is not None:
                    k, v = k * self.cache.k_scale[h].double(), v * self.cache.v_scale[h].double()
                q = self.q[rows].double().view(-1, self.hkv, g, d)[:, h].reshape(-1, d)
                s = (q @ k.t() * d ** -0.5).masked_fill_(hide, -math.inf)
                l = torch.logsumexp(s, 1, keepdim=True)
                p = torch.exp(s - l)
                ref, mag = p @ v, p @ v.abs()
                # a score: d products summed; its exponent: scale, base and their difference; the sum: all the terms
                amag = (q.abs() @ k.abs().t()).amax(1, keepdim=True) * d ** -0.5
                top = s.masked_fill(hide, 0).abs().amax(1, keepdim=True)
                rel = 2 * (2 * d * E24 * amag + 8 * E24 * (top + 1)) + 2 * terms * E24 + 16 * E24
                got = out[rows].double().view(-1, self.hkv, g, d)[:, h].reshape(-1, d)
                got_l = lse[rows].double().view(-1, self.hkv, g)[:, h].reshape(-1, 1)
                # p is rounded to BF16 for the product with v, not for its sum
                assert ((got - ref).abs() <= ref.abs() * B8 + mag * (B8 * 1.01 + rel)).all(), f"request {b} head {h}: out"
                assert ((got_l - l).abs() <= rel + 4 * E24 * l.abs()).all(), f"request {b} head {h}: lse"


def _unequal(n, low, high, seed):
    return torch.randint(low, high + 1, (n,), generator=torch.Generator().manual_seed(seed)).tolist()


@pytest.mark.parametrize("d,f8,page", [(128, False, 64), (128, True, 64), (64, False, 16), (64, True, 128), (256, False, 64),
                                       (256, True, 16)])
def test_attention_batch_in_one_round(d, f8, page):
    """16 requests of 13 to 24 nodes over 500 to 4000 tokens: chunks of several tiles, joined by waves with elements of
    their own."""
    b = Batch(_unequal(16, 500, 4000, 1), _unequal(16, 13, 24, 2), 40, 8, d, page=page, f8=f8, seed=d + f8)
    out, lse = b.run()
    b.check(out, lse)
    for _ in range(3):
        again = b.run()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1]), "not the same from run to run"


@pytest.mark.parametrize("n,hq,hkv,d,f8,top", [(48, 16, 8, 128, False, 6000), (70, 40, 8, 64, True, 3000), (300, 8, 8, 64, False, 2500)])
def test_attention_many_requests_of_several_chunks(n, hq, hkv, d, f8, top):
    """More requests than make one round: chunks by the cost of all tiles, of one request many and of others none."""
    ctxs = _unequal(n, 0, 200, 3)
    ctxs[5], ctxs[n // 2], ctxs[n - 1] = top, top - 77, top // 2
    b = Batch(ctxs, _unequal(n, 1, 9, 4), hq, hkv, d, f8=f8, seed=n)
    b.check(*b.run(), per_request=2)
    even = Batch([top // 2 + 3 * i for i in range(n)], [3] * n, hq, hkv, d, f8=f8, tree=False, seed=n + 1)
    even.check(*even.run(), per_request=1)


@pytest.mark.parametrize("ctx,n,hq,hkv,d,f8,page", [(60000, 64, 40, 8, 128, False, 64), (40001, 63, 10, 2, 128, True, 64),
                                                    (30011, 40, 8, 2, 256, False, 64), (20000, 13, 6, 1, 64, False, 16)])
def test_attention_one_request_with_long_chunks(ctx, n, hq, hkv, d, f8, page):
    """Chunks of many tiles, over and over through both buffers."""
    b = Batch([ctx], [n], hq, hkv, d, page=page, f8=f8, seed=ctx)
    b.check(*b.run(), per_request=10)


@pytest.mark.parametrize("ctx,n,hq,hkv,d,f8", [(3000, 960, 40, 8, 128, False), (0, 4096, 10, 2, 128, False), (100, 2500, 16, 4, 64, True),
                                              (7, 1500, 8, 2, 256, False)])
def test_attention_prompt(ctx, n, hq, hkv, d, f8):
    """Chains of hundreds to thousands of nodes: more than a round of items, or one chunk a block."""
    b = Batch([ctx], [n], hq, hkv, d, f8=f8, tree=False, seed=n)
    b.check(*b.run(), per_request=20)
