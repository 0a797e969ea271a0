"""GPU tests of the operators around the products against plain 64-bit implementations on the CPU.

Tolerances.  A rounding is off by at most half a step: relative to the value 2^-8 (BF16), 2^-24 (FP32), 2^-4
(E4M3, plus half its smallest step, 2^-10, near zero).  Sums of n FP32 terms are off by at most n 2^-24 of the
sum of magnitudes; matrix instructions may cut off where they could round, which doubles that.
"""
import math

import pytest
import torch

import lossless_bit_weight_encode_amd as w12

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
B8, E24, Q4 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4
NAN = float("nan")


def rnd(seed, *shape, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale


def pitched(x, ld, fill=NAN):
    """x [R, C] on the GPU with pitch ld, the gap filled with NaN, after a guard of 64 values and before one."""
    r, c = x.shape
    buf = torch.full((64 + r * ld + 64,), fill, dtype=torch.float32).to(x.dtype)
    v = buf[64:64 + r * ld].view(r, ld)
    v[:, :c] = x
    buf = buf.cuda()
    return buf[64:64 + r * ld].view(r, ld)[:, :c], buf


def out_buf(r, c, ld, dtype):
    """An output [r, c] of pitch ld inside a buffer of a pattern, and a check that nothing else was written."""
    size = 64 + r * ld + 64
    raw = {BF: torch.int16, F32: torch.int32, F8: torch.uint8}[dtype]
    buf = torch.full((size,), 0x55, dtype=raw, device="cuda")

    def untouched():
        b = buf.clone().cpu()
        b[64:64 + r * ld].view(r, ld)[:, :c] = 0x55
        return bool((b == 0x55).all())

    return buf.view(dtype)[64:64 + r * ld].view(r, ld)[:, :c], untouched


def assert_close(got, ref, tol, what):
    got = got.detach().cpu().double()
    assert torch.equal(got.isnan(), ref.isnan()), f"{what}: NaN at other places"
    fin = ref.isfinite()
    assert torch.equal(got[~fin & ~ref.isnan()], ref[~fin & ~ref.isnan()]), f"{what}: infinities differ"
    over = ((got - ref).abs() - tol)[fin]
    assert over.numel() == 0 or over.max() <= 0, f"{what}: {int((over > 0).sum())} values off by up to {over.max():.3g} too much"


# ---------------------------------------------------------------------------------------------- norm

def norm_ref(r, d, w, eps):
    x = r.double() + (0 if d is None else d.double())
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * w.double()
    return x, y


def check_quant(yq, scale, y, n, rel):
    nb = -(-n // 128)
    yp = torch.nn.functional.pad(y, (0, nb * 128 - n)).view(y.shape[0], nb, 128)
    amax = yp.abs().amax(2)
    s_ref = torch.where(amax == 0, torch.ones_like(amax), amax / 448)
    assert_close(scale, s_ref, rel * s_ref + 2.0 ** -149, "scale")
    s = s_ref[:, :, None].expand(-1, -1, 128).reshape(y.shape[0], -1)[:, :n]
    got = yq.cpu().double() * s
    assert_close(got, y, (Q4 + 4 * rel) * y.abs() + 2.0 ** -10 * s, "yq")


@pytest.mark.parametrize("m,n", [(1, 1), (1, 5120), (3, 7), (2, 127), (5, 129), (2, 1000), (1, 8193), (3, 17408), (2, 65536),
                                 (67, 136), (300, 64), (1100, 2056), (1, 16), (2, 40001), (33, 4095)])
@pytest.mark.parametrize("rt,dt", [(BF, F32), (F32, F32), (F32, BF), (BF, BF), (BF, None)])
def test_norm(m, n, rt, dt):
    r = rnd(1, m, n, scale=3.0).to(rt)
    d = None if dt is None else rnd(2, m, n).to(dt)
    w = (1 + rnd(3, n, scale=0.2)).to(BF)
    ld = (n + 15) // 16 * 16 + 16
    rd, _ = pitched(r, ld)
    dd = None if d is None else pitched(d, ld)[0]
    wd = pitched(w[None], ld)[0][0]
    ro, ok_r = out_buf(m, n, ld, rt)
    y, ok_y = out_buf(m, n, ld, BF)
    yq, ok_q = out_buf(m, n, ld, F8)
    sc, ok_s = out_buf(m, -(-n // 128), -(-n // 128) + 1, F32)
    got = w12.add_rmsnorm(rd, wd, dd, eps=1e-5, residual_out=ro, y=y, yq=yq, yq_scale=sc)
    torch.cuda.synchronize()
    assert got is y and ok_r() and ok_y() and ok_q() and ok_s(), "write outside an output"
    x, ref = norm_ref(r, d, w, 1e-5)
    half = {BF: B8, F32: E24}[rt]
    assert_close(ro, x, x.abs() * (half + (0 if dt is None else E24 * 1.01)), "residual_out")
    # r: one rounding; the mean square: n terms, each squared from a rounded r; square root, quotient, two products
    rel = (n + 12) * E24
    if d is not None:
        # a sum that cancels has the rounding of the sum, relative to itself: nothing more
        rel += E24
    assert_close(y, ref, ref.abs() * (B8 + 1.01 * rel), "y")
    check_quant(yq, sc, ref, n, rel)


def test_norm_in_place_and_each_output_alone():
    r, d, w = rnd(4, 9, 264).to(BF), rnd(5, 9, 264), (1 + rnd(6, 264, scale=0.1)).to(BF)
    rd, dd, wd = r.cuda(), d.cuda(), w.cuda()
    y = w12.add_rmsnorm(rd, wd, dd, residual_out=rd)
    x, ref = norm_ref(r, d, w, 1e-6)
    assert_close(rd, x, x.abs() * (B8 + 2 * E24), "in place")
    assert_close(y, ref, ref.abs() * (B8 + 300 * E24), "y")
    y2 = torch.empty_like(y)
    w12.add_rmsnorm(r.cuda(), wd, dd, y=y2)                       # nothing stored but y
    assert torch.equal(y, y2)
    yq = torch.empty(9, 272, dtype=F8, device="cuda")[:, :264]
    sc = torch.empty(9, 3, device="cuda")
    assert w12.add_rmsnorm(r.cuda(), wd, dd, yq=yq, yq_scale=sc) is None
    check_quant(yq, sc, ref, 264, 300 * E24)


def test_norm_zero_rows_nan_and_infinity():
    n = 400
    r = rnd(7, 6, n)
    r[0] = 0
    r[1, 130:300] = 0
    r[2, 5] = NAN
    r[3, 399] = float("inf")
    r[4] *= 1e-25                    # squares below the normal range
    w = torch.ones(n)
    w[128:256] = 0
    y = torch.empty(6, n, dtype=BF, device="cuda")
    yq = torch.empty(6, n, dtype=F8, device="cuda")
    sc = torch.empty(6, 4, device="cuda")
    w12.add_rmsnorm(r.cuda(), w.to(BF).cuda(), y=y, yq=yq, yq_scale=sc, eps=1e-6)
    y, yq, sc = y.cpu().double(), yq.cpu().double(), sc.cpu()
    assert (y[0] == 0).all() and (yq[0] == 0).all() and (sc[0] == 1).all()
    assert (sc[:2, 1] == 1).all() and (yq[:2, 128:256] == 0).all()
    assert y[2].isnan().all() and sc[2].isnan().all() and yq[2].isnan().all()
    assert y[3, 399].isnan() and (y[3, :399] == 0).all()          # inf / inf, x / inf
    ref = norm_ref(r[4:], None, w, 1e-6)[1]
    assert_close(y[4:], ref, ref.abs() * B8 * 1.01 + 1e-38, "tiny row")


# ---------------------------------------------------------------------------------------------- rope

def make_cache(pages, page, heads, dim, f8, heads_first=False, seed=0):
    shape = (pages, heads, page, dim) if heads_first else (pages, page, heads, dim)
    kv, scales = [], []
    for i in range(2):
        x = rnd(seed + i, *shape)
        if f8:
            s = 0.01 + 0.005 * torch.rand(heads, generator=torch.Generator().manual_seed(seed + 7 + i))
            sb = s[None, :, None, None] if heads_first else s[None, None, :, None]
            x = (x / sb).clamp(-448, 448).to(F8)
            scales.append(s.cuda())
        else:
            x = x.to(BF)
        x = x.cuda()
        kv.append(x.transpose(1, 2) if heads_first else x)
    return w12.KVCache(*kv, *scales)


def values(cache):
    """K and V of a cache in 64 bits on the CPU."""
    k, v = cache.k.cpu().double(), cache.v.cpu().double()
    if cache.k_scale is not None:
        k = k * cache.k_scale.cpu().double()[:, None]
        v = v * cache.v_scale.cpu().double()[:, None]
    return k, v


@pytest.mark.parametrize("t,hq,hkv,d,rot,axes,adjacent,src,f8,page,hf,far", [
    (1, 1, 1, 64, 64, 1, False, F32, False, 16, False, 10),
    (1, 40, 8, 128, 128, 1, False, F32, False, 64, False, 131071),
    (7, 5, 1, 128, 64, 2, False, BF, False, 1, True, 999),
    (33, 4, 4, 256, 256, 3, False, F32, True, 32, False, 1 << 20),
    (65, 6, 2, 64, 32, 3, True, F32, False, 8, False, 5000),
    (12, 8, 2, 128, 10, 2, False, F32, True, 64, True, 77),      # a part that no vector divides
    (12, 8, 2, 128, 10, 2, True, BF, True, 128, False, 77),
    (300, 2, 1, 128, 128, 8, False, F32, False, 16, False, (1 << 31) - 1),
    (3, 64, 1, 64, 48, 1, False, F32, True, 16, False, 12345),
    (5, 3, 3, 128, 0, 1, False, F32, False, 16, False, 5),        # nothing turns
    (600, 10, 2, 128, 128, 3, False, BF, True, 64, False, 300000),
    (20, 4, 2, 256, 24, 2, True, F32, False, 16, False, 4000),
])
def test_rope(t, hq, hkv, d, rot, axes, adjacent, src, f8, page, hf, far):
    pages = -(-(t + 40) // page)
    cache = make_cache(pages, page, hkv, d, f8, hf, seed=20)
    old_k, old_v = cache.k.cpu().clone(), cache.v.cpu().clone()
    width = (hq + 2 * hkv) * d
    qkv = rnd(21, t, width, scale=2.0).to(src)
    gen = torch.Generator().manual_seed(22)
    pos = torch.randint(max(0, far - 50000), far + 1, (axes, t), generator=gen, dtype=torch.int64)
    pos[0, 0] = far
    if t > 3:
        pos[axes - 1, 2] = -17
    pos = pos.to(torch.int32)
    slots = torch.randperm(pages * page, generator=gen)[:t]
    if t > 4:
        slots[1], slots[3] = -1, pages * page + 5          # rows that are not put
    inv = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1)))
    axis = torch.randint(0, axes, (rot // 2,), generator=gen).to(torch.uint8)
    qd = pitched(qkv, width + 16)[0]
    q, ok = out_buf(t, hq * d, hq * d + 8, BF)
    posd = torch.zeros(axes, t + 3, dtype=torch.int32, device="cuda")[:, :t]
    posd.copy_(pos)
    w12.rope_append(qd, cache, posd, slots.cuda(), inv.cuda(), hq, axis=axis.cuda() if axes > 1 else None, adjacent=adjacent, q=q)
    torch.cuda.synchronize()
    assert ok(), "write outside q"
    x = qkv.double().view(t, hq + 2 * hkv, d)
    ref, mag = x.clone(), x.abs()
    for i in range(rot // 2):
        th = pos[int(axis[i])].double() * inv[i]
        th = torch.remainder(th, 2 * math.pi)[:, None]
        lo, hi = (2 * i, 2 * i + 1) if adjacent else (i, i + rot // 2)
        a, b = x[:, :hq + hkv, lo], x[:, :hq + hkv, hi]
        ref[:, :hq + hkv, lo], ref[:, :hq + hkv, hi] = a * th.cos() - b * th.sin(), a * th.sin() + b * th.cos()
        both = a.abs() + b.abs()
        mag[:, :hq + hkv, lo], mag[:, :hq + hkv, hi] = both, both
    # angle: FP64 to 2^-52 of up to 2^31 radians, kept to FP32 (2^-24 of a half turn), sine and cosine within 4 steps,
    # then two products and a sum
    err = mag * (math.pi * E24 + 2.0 ** 31 * 2.0 ** -51 + 12 * E24)
    assert_close(q.reshape(t, hq, d), ref[:, :hq], ref[:, :hq].abs() * B8 + err[:, :hq] * 1.01, "q")
    got_k, got_v = cache.k.cpu(), cache.v.cpu()
    for got, old, sc, h0, what in ((got_k, old_k, cache.k_scale, hq, "k"), (got_v, old_v, cache.v_scale, hq + hkv, "v")):
        want, e = ref[:, h0:h0 + hkv], err[:, h0:h0 + hkv]
        old = old.clone()
        for i in range(t):
            s = int(slots[i])
            if s < 0 or s >= pages * page:
                continue
            g = got[s // page, s % page].double()
            if f8:
                scale = sc.cpu().double()[:, None]
                r = (want[i] / scale).clamp(-448, 448)
                assert_close(g, r, r.abs() * (Q4 + 4 * E24) + 2.0 ** -10 + e[i] / scale * 1.1, what)
            else:
                assert_close(g, want[i], want[i].abs() * B8 + e[i] * 1.01, what)
            old[s // page, s % page] = got[s // page, s % page]
        assert torch.equal(got.view(torch.uint8), old.view(torch.uint8)), f"{what}: a place that no row names was written"


def test_rope_keeps_nan_and_cuts_off():
    cache = make_cache(2, 16, 1, 64, True, seed=30)
    qkv = torch.zeros(2, 192)
    qkv[0, 64:68] = torch.tensor([NAN, float("inf"), -1e30, 1e30])
    qkv[1, 128:131] = torch.tensor([-float("inf"), NAN, 460 * float(cache.v_scale[0])])
    w12.rope_append(qkv.cuda(), cache, torch.zeros(1, 2, dtype=torch.int32, device="cuda"),
                    torch.tensor([3, 20], device="cuda"), torch.zeros(0, dtype=torch.float64, device="cuda"), 1)
    k, v = cache.k.cpu().float()[0, 3, 0], cache.v.cpu().float()[1, 4, 0]
    assert k[0].isnan() and k[1:4].tolist() == [448, -448, 448]
    assert v[0] == -448 and v[1].isnan() and v[2] == 448


# ----------------------------------------------------------------------------------------- attention

def ancestors(parents):
    bits = []
    for i, p in enumerate(parents):
        bits.append((1 << i) | (bits[p] if p >= 0 else 0))
    return bits


def mask_tensor(bits, words):
    rows = []
    for b in bits:
        row = []
        for w in range(words):
            v = (b >> (64 * w)) & ((1 << 64) - 1)
            row.append(v - (1 << 64) if v >> 63 else v)
        rows.append(row)
    return torch.tensor(rows, dtype=torch.int64)


class Problem:
    """A batch over a paged cache whose unused places (and the tails of its pages) are NaN."""

    def __init__(self, ctxs, nodes, hq, hkv, d, page=16, f8=False, hf=False, mask="tree", words=1, seed=0, qscale=1.0,
                 spare=3):
        gen = torch.Generator().manual_seed(seed)
        self.ctxs, self.nodes, self.hq, self.hkv, self.d, self.page = ctxs, nodes, hq, hkv, d, page
        b = len(ctxs)
        need = [-(-(c + n) // page) for c, n in zip(ctxs, nodes)]
        self.max_pages = max(1, max(need)) + 1
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=gen)
        shape = (pages, hkv, page, d) if hf else (pages, page, hkv, d)
        self.table = torch.full((b, self.max_pages), 0x7FFFFFFF, dtype=torch.int32)
        at = 0
        for i, p in enumerate(need):
            self.table[i, :p] = order[at:at + p].to(torch.int32)
            at += p
        used = torch.zeros(pages, page, dtype=torch.bool)
        for i in range(b):
            tok = torch.arange(ctxs[i] + nodes[i])
            used[self.table[i].long()[tok // page], tok % page] = True
        kv, self.scales = [], []
        for j in range(2):
            x = torch.randn(pages, page, hkv, d, generator=gen)
            if f8:
                s = 0.01 + 0.004 * torch.rand(hkv, generator=gen)
                x = (x / s[:, None]).clamp(-448, 448)
                self.scales.append(s)
            x[~used] = NAN
            x = x.to(F8 if f8 else BF)
            if hf:
                buf = torch.empty(shape, dtype=x.dtype)
                buf.view(torch.uint8).copy_(x.view(torch.uint8).transpose(1, 2)) if f8 else buf.copy_(x.transpose(1, 2))
                x = buf.cuda().transpose(1, 2)
            else:
                x = x.cuda()
            kv.append(x)
        self.cache = w12.KVCache(*kv, *[s.cuda() for s in self.scales])
        self.t = sum(nodes)
        self.q = (torch.randn(max(1, self.t), hq * d, generator=gen) * qscale).to(BF)
        self.ptr = [0]
        for n in nodes:
            self.ptr.append(self.ptr[-1] + n)
        self.mask = None
        if mask == "tree":
            bits = []
            for n in nodes:
                parents = [-1] + [int(torch.randint(max(0, i - 9), i, (1,), generator=gen)) for i in range(1, n)]
                bits += ancestors(parents[:n])
            self.mask = mask_tensor(bits, words)
        elif mask == "random":
            self.mask = torch.randint(-(1 << 62), 1 << 62, (max(1, self.t), words), generator=gen)
            self.mask[::3] = 0

    def run(self, lse=True, **kw):
        t = self.q.shape[0]
        out, ok = out_buf(t, self.hq * self.d, self.hq * self.d + 8, BF)
        ls, ok_l = out_buf(t, self.hq, self.hq + 1, F32)
        q, _ = pitched(self.q, self.hq * self.d + 16)
        mask = None if self.mask is None else self.mask.cuda()
        w12.tree_attention(q, self.cache, self.table.cuda(), torch.tensor(self.ctxs, dtype=torch.int32, device="cuda"),
                           torch.tensor(self.ptr, dtype=torch.int32, device="cuda"), tree_mask=mask, out=out,
                           lse=ls if lse else None, **kw)
        torch.cuda.synchronize()
        assert ok() and ok_l(), "write outside an output"
        return out.cpu(), ls.cpu()

    def sees(self, row, node, n):
        if self.mask is None:
            return [j <= node for j in range(n)]
        w = self.mask[row]
        return [j < 64 * len(w) and bool((int(w[j // 64]) >> (j % 64)) & 1) for j in range(n)]

    def check(self, out, lse, scale=None):
        k, v = values(self.cache)
        d, g = self.d, self.hq // self.hkv
        scale = d ** -0.5 if scale is None else scale
        for b, (ctx, n) in enumerate(zip(self.ctxs, self.nodes)):
            tok = torch.arange(ctx + n)
            page = self.table[b].long()[(tok // self.page).clamp(max=self.max_pages - 1)]
            here = (tok // self.page < self.max_pages) & (page >= 0) & (page < self.cache.pages)
            page = page.clamp(0, self.cache.pages - 1)
            kb, vb = k[page, tok % self.page], v[page, tok % self.page]          # [len, hkv, d]
            for i in range(n):
                row = self.ptr[b] + i
                see = torch.cat((torch.ones(ctx, dtype=torch.bool), torch.tensor(self.sees(row, i, n), dtype=torch.bool))) & here
                q = self.q[row].double().view(self.hkv, g, d)
                got, got_l = out[row].double().view(self.hkv, g, d), lse[row].double().view(self.hkv, g)
                if not see.any():
                    assert (got == 0).all() and (got_l == -math.inf).all(), f"row {row} attends nothing"
                    continue
                kk, vv = kb[see], vb[see]
                s = torch.einsum("hgd,thd->hgt", q, kk) * scale
                amag = torch.einsum("hgd,thd->hgt", q.abs(), kk.abs()).amax() * scale
                l = torch.logsumexp(s, 2)
                p = torch.exp(s - l[..., None])
                ref = torch.einsum("hgt,thd->hgd", p, vv)
                mag = torch.einsum("hgt,thd->hgd", p, vv.abs())
                # scores: d products summed, and the exponent's base and scale; p is rounded to BF16 for the
                # matrix product; sums of up to len terms, cut off or rounded
                ds = float(2 * d * E24 * amag + 8 * E24 * (s.abs().max() + 1))
                rel = ds * 2 + 2 * len(kk) * E24 + 16 * E24
                assert_close(got, ref, ref.abs() * B8 + mag * (B8 * 1.01 + rel), f"request {b} node {i} out")
                # the sum of the rounded p: each is off by up to 2^-8 of itself
                assert_close(got_l, l, torch.full_like(l, B8 * 1.01 + rel) + l.abs() * 4 * E24, f"request {b} node {i} lse")


CASES = [
    dict(ctxs=[0], nodes=[1], hq=1, hkv=1, d=64),
    dict(ctxs=[1], nodes=[1], hq=1, hkv=1, d=128, mask=None),
    dict(ctxs=[509], nodes=[1], hq=40, hkv=8, d=128, page=64, mask=None),
    dict(ctxs=[0], nodes=[64], hq=8, hkv=2, d=64),
    dict(ctxs=[1000], nodes=[63], hq=10, hkv=2, d=128, page=64),
    dict(ctxs=[777], nodes=[64], hq=8, hkv=1, d=256, page=32, f8=True),
    dict(ctxs=[31, 0, 64, 65, 300], nodes=[5, 17, 1, 33, 24], hq=6, hkv=2, d=128, page=16, hf=True),
    dict(ctxs=[31, 0, 200, 65], nodes=[5, 0, 0, 40], hq=4, hkv=4, d=64, page=1, f8=True, mask=None),
    dict(ctxs=[0, 0, 0], nodes=[3, 0, 2], hq=4, hkv=1, d=128, mask="random"),
    dict(ctxs=[0, 90], nodes=[64, 64], hq=2, hkv=1, d=128, mask="random", page=8),
    dict(ctxs=[130], nodes=[130], hq=2, hkv=1, d=64, mask="tree", words=3, page=128),
    dict(ctxs=[130], nodes=[100], hq=2, hkv=2, d=64, mask="tree", words=1, page=1024),    # nodes past the words
    dict(ctxs=[77], nodes=[300], hq=3, hkv=3, d=128, mask=None, page=4),
    dict(ctxs=[33], nodes=[2], hq=64, hkv=1, d=128, page=16),
    dict(ctxs=[33], nodes=[37], hq=7, hkv=7, d=64, page=2, f8=True, hf=True),
    dict(ctxs=[5000], nodes=[9], hq=5, hkv=1, d=128, page=64, qscale=6.0),
    dict(ctxs=[12345], nodes=[2], hq=2, hkv=1, d=64, page=64, qscale=0.05),
    dict(ctxs=[2000], nodes=[8], hq=4, hkv=1, d=256, page=64, qscale=3.0),
    dict(ctxs=list(range(0, 90, 3)), nodes=[(i % 5) for i in range(30)], hq=4, hkv=2, d=64, page=16, f8=True),
    dict(ctxs=[4000, 3, 1500], nodes=[1, 1, 1], hq=16, hkv=2, d=256, page=16, f8=True, mask=None),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention(i):
    p = Problem(**CASES[i], seed=40 + i)
    p.check(*p.run())


def test_attention_scale_and_no_lse_and_repeat():
    p = Problem([700, 40], [20, 64], 10, 2, 128, seed=70)
    out, lse = p.run(scale=0.3)
    p.check(out, lse, scale=0.3)
    for _ in range(5):
        again, _ = p.run(lse=False, scale=0.3)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "not the same from run to run"


@pytest.mark.parametrize("hq,d,f8", [(5, 128, False), (5, 64, True), (2, 256, False)])
def test_attention_masked_nodes_do_not_reach_a_row(hq, d, f8):
    """NaN and infinities in the keys and values of nodes that a row does not attend."""
    n, ctx = 40, 70
    p = Problem([ctx], [n], hq, 1, d, page=16, f8=f8, seed=80)
    clean, lse = p.run()
    bad = [3, 17, 30]
    tok = ctx + torch.tensor(bad)
    page, off = p.table[0].long()[tok // 16].cuda(), (tok % 16).cuda()
    for j in range(len(bad)):
        fill = NAN if f8 else [NAN, float("inf"), -float("inf")][j]
        code = torch.tensor([fill]).to(p.cache.k.dtype).view(torch.uint8 if f8 else torch.int16).item()
        for x in (p.cache.k, p.cache.v):
            x.view(torch.uint8 if f8 else torch.int16)[page[j], off[j]] = code
    out, _ = p.run()
    for i in range(n):
        hit = any((int(p.mask[i, 0]) >> b) & 1 for b in bad)
        if hit:
            assert out[i].isnan().any(), f"row {i} attends a NaN"
        else:
            assert torch.equal(out[i].view(torch.int16), clean[i].view(torch.int16)), f"row {i} does not attend the NaN"


def test_attention_value_infinity_reaches_its_element_alone():
    p = Problem([100], [4], 2, 1, 64, page=16, mask=None, seed=85)
    page, off = int(p.table[0, 2]), 5
    p.cache.v[page, off, 0, 7] = float("inf")
    out, _ = p.run()
    o = out.float().view(-1, 2, 64)
    assert (o[:, :, 7] == math.inf).all() and o[:, :, :7].isfinite().all() and o[:, :, 8:].isfinite().all()


def test_attention_absent_pages():
    """Page numbers outside the cache, and tokens past the table, count as absent."""
    p = Problem([200, 90], [6, 6], 4, 2, 64, page=16, seed=90)
    p.table[0, 3], p.table[0, 5], p.table[1, 0] = -1, p.cache.pages, -(1 << 31)
    p.check(*p.run())
    p.table[1, :] = -5                       # nothing left of the second request
    p.check(*p.run())
    # a table that is too short for its request: the drafted nodes lie past its end
    short = Problem([40], [8], 2, 1, 64, page=16, seed=91)
    short.table, short.max_pages = short.table[:, :2].contiguous(), 2
    short.check(*short.run())


def test_attention_rows_outside_requests_and_odd_ranges():
    p = Problem([50, 60], [7, 9], 4, 2, 64, seed=95)
    out, lse = p.run()
    p2 = Problem([50, 60], [7, 9], 4, 2, 64, seed=95)
    p2.ptr = [0, 7, 12]                      # the last rows belong to nobody
    o2, l2 = p2.run()
    raw = o2.view(torch.int16)
    assert (raw[12:] == 0x55).all() and (l2.view(torch.int32)[12:] == 0x55).all(), "rows outside every request were written"
    assert torch.equal(o2[:7].view(torch.int16), out[:7].view(torch.int16))
    p2.ptr = [-3, 7, 1000]                   # cut to 0..T
    o3, _ = p2.run()
    assert torch.equal(o3.view(torch.int16), out.view(torch.int16))
    p2.ptr, p2.ctxs = [0, 7, 16], [-4, 60]   # a negative length counts as 0
    o4, _ = p2.run()
    assert torch.equal(o4[7:].view(torch.int16), out[7:].view(torch.int16))
    p.ctxs = [0, 60]
    o5, _ = p.run()
    assert torch.equal(o4[:7].view(torch.int16), o5[:7].view(torch.int16))


def test_attention_many_requests():
    n = 700
    p = Problem([(i * 7) % 40 for i in range(n)], [1 + (i % 3 == 0) for i in range(n)], 2, 1, 64, page=16, seed=97)
    p.check(*p.run())


def test_attention_far_into_a_large_cache():
    """Page offsets past 2^32 elements."""
    pages, page, heads, d = 70000, 64, 8, 128
    k = torch.empty(pages, page, heads, d, dtype=BF, device="cuda")
    v = torch.empty(pages, page, heads, d, dtype=BF, device="cuda")
    small = Problem([100], [5], 8, 8, d, page=64, seed=98)
    k[-4:], v[-4:] = small.cache.k[:4], small.cache.v[:4]
    assert small.cache.pages <= 6
    used = small.table[0, :2]
    for i in range(2):
        k[pages - 10 + i], v[pages - 10 + i] = small.cache.k[int(used[i])], small.cache.v[int(used[i])]
    ref = small.run()
    small.table[0, 0], small.table[0, 1] = pages - 10, pages - 9
    small.cache = w12.KVCache(k, v)
    got = small.run()
    assert torch.equal(got[0].view(torch.int16), ref[0].view(torch.int16)) and torch.equal(got[1], ref[1])
    # the write goes to the same places
    qkv = torch.randn(1, 24 * d, device="cuda")
    w12.rope_append(qkv, small.cache, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                    torch.tensor([(pages - 1) * page + 63], device="cuda"), torch.zeros(0, dtype=torch.float64, device="cuda"), 8)
    assert torch.equal(k[-1, -1].flatten(), qkv[0, 8 * d:16 * d].to(BF))


# ------------------------------------------------------------------------------------------ 8-bit product

def gemm_inputs(m, n, k, seed, ld=0):
    x = rnd(seed, m, k, scale=60.0).clamp(-448, 448).to(F8)
    w = rnd(seed + 1, n, k, scale=60.0).clamp(-448, 448).to(F8)
    kb, nb = -(-k // 128), -(-n // 128)
    g = torch.Generator().manual_seed(seed + 2)
    xs = torch.rand(m, kb, generator=g) * 0.02 + 1e-3
    ws = torch.exp(torch.randn(nb, kb, generator=g)) * 1e-3
    return x, xs, w, ws


def gemm_ref(x, xs, w, ws):
    n, k = w.shape
    a = x.double() * xs.double().repeat_interleave(128, 1)[:, :k]
    b = w.double() * ws.double().repeat_interleave(128, 1)[:, :k].repeat_interleave(128, 0)[:n]
    return a @ b.t(), a.abs() @ b.abs().t()


GEMM = [(1, 1, 1), (1, 16, 128), (1, 70, 200), (2, 129, 1000), (3, 256, 4096), (7, 500, 127), (16, 130, 129), (17, 64, 384),
        (31, 300, 2064), (33, 1024, 512), (63, 513, 1040), (64, 128, 128), (65, 200, 300), (100, 257, 1111), (128, 384, 256),
        (130, 640, 700), (200, 100, 100), (256, 512, 2048), (257, 300, 640), (512, 260, 384), (1000, 130, 260),
        (4, 40, 20000), (48, 96, 12000), (300, 2100, 650), (4096, 33, 65)]


@pytest.mark.parametrize("m,n,k", GEMM)
def test_gemm_e4m3(m, n, k):
    x, xs, w, ws = gemm_inputs(m, n, k, 100 + m + n + k)
    ld = (k + 15) // 16 * 16 + 16
    kb, nb = -(-k // 128), -(-n // 128)
    xd, wd = pitched(x, ld)[0], pitched(w, ld)[0]
    xsd, wsd = pitched(xs, kb + 1)[0], pitched(ws, kb + 2)[0]
    y, ok = out_buf(m, n, n + 3, F32)
    wk = w12.gemm_e4m3_workspace(m, n, k)
    w12.gemm_e4m3(xd, xsd, wd, wsd, y=y, ws=wk)
    torch.cuda.synchronize()
    assert ok(), "write outside Y"
    ref, mag = gemm_ref(x, xs, w, ws)
    assert_close(y, ref, mag * 2 * (128 + kb + 8) * E24, "Y")
    for _ in range(3):
        y2 = w12.gemm_e4m3(xd, xsd, wd, wsd, ws=wk)
        assert torch.equal(y2, y), "not the same from run to run"


def test_gemm_e4m3_nan_stays_in_its_row_and_channel():
    m, n, k = 40, 300, 520
    x, xs, w, ws = gemm_inputs(m, n, k, 7)
    x.view(torch.uint8)[5, 519] = 0x7F
    w.view(torch.uint8)[200, 0] = 0xFF
    y = w12.gemm_e4m3(pitched(x, 528)[0], xs.cuda(), pitched(w, 528)[0], ws.cuda()).cpu()
    bad = torch.zeros(m, n, dtype=torch.bool)
    bad[5], bad[:, 200] = True, True
    assert torch.equal(y.isnan(), bad)


# --------------------------------------------------------------------------------------------- streams, graphs

def test_operators_on_another_stream():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        r, w = rnd(200, 8, 256).cuda(), torch.ones(256, dtype=BF, device="cuda")
    s.synchronize()
    y = w12.add_rmsnorm(r, w, stream=s)
    x, xs, ww, ws = (t.cuda() for t in gemm_inputs(20, 300, 512, 3))
    p = Problem([90], [12], 4, 2, 64, seed=201)
    args = (p.q.cuda(), p.cache, p.table.cuda(), torch.tensor([90], dtype=torch.int32, device="cuda"),
            torch.tensor([0, 12], dtype=torch.int32, device="cuda"), p.mask.cuda())
    torch.cuda.synchronize()
    g = w12.gemm_e4m3(x, xs, ww, ws, stream=s)
    o = w12.tree_attention(*args, stream=s)
    s.synchronize()
    assert torch.equal(y, w12.add_rmsnorm(r, w))
    assert torch.equal(g, w12.gemm_e4m3(x, xs, ww, ws))
    assert torch.equal(o, w12.tree_attention(*args))


def test_operators_in_a_graph():
    """A captured step follows the lengths, tables and inputs that change between replays."""
    p = Problem([300, 20], [8, 16], 8, 2, 128, page=16, seed=210)
    t, hq, hkv, d = 24, 8, 2, 128
    ctx = torch.tensor(p.ctxs, dtype=torch.int32, device="cuda")
    ptr = torch.tensor(p.ptr, dtype=torch.int32, device="cuda")
    table, mask = p.table.cuda(), p.mask.cuda()
    res, w = rnd(211, t, 512).to(BF).cuda(), torch.ones(512, dtype=BF, device="cuda")
    x8 = torch.empty(t, 512, dtype=F8, device="cuda")
    xs = torch.empty(t, 4, device="cuda")
    _, _, w8, ws8 = (v.cuda() for v in gemm_inputs(1, (hq + 2 * hkv) * d, 512, 212))
    qkv = torch.empty(t, (hq + 2 * hkv) * d, device="cuda")
    q, out = torch.empty(t, hq * d, dtype=BF, device="cuda"), torch.empty(t, hq * d, dtype=BF, device="cuda")
    inv = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    slots, pos = torch.empty(t, dtype=torch.int64, device="cuda"), torch.empty(1, t, dtype=torch.int32, device="cuda")
    gws = w12.gemm_e4m3_workspace(t, qkv.shape[1], 512)
    aws = w12.tree_attention_workspace(t, 2, hq, p.cache)

    def place():
        for b in range(2):
            for i in range(p.nodes[b]):
                tok = int(ctx[b]) + i
                slots[p.ptr[b] + i] = int(table[b, tok // 16]) * 16 + tok % 16
                pos[0, p.ptr[b] + i] = tok

    def step():
        w12.add_rmsnorm(res, w, yq=x8, yq_scale=xs)
        w12.gemm_e4m3(x8, xs, w8, ws8, y=qkv, ws=gws)
        w12.rope_append(qkv, p.cache, pos, slots, inv, hq, q=q)
        w12.tree_attention(q, p.cache, table, ctx, ptr, tree_mask=mask, out=out, ws=aws)

    place()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        res.copy_(rnd(220 + i, 24, 512).to(BF))
        ctx.copy_(torch.tensor([300 - 40 * i, 20 - i], dtype=torch.int32))
        place()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got, gq = out.clone(), qkv.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and torch.equal(gq, qkv), f"replay {i} differs from the eager step"
        assert got.isfinite().all() and got.abs().max() > 0


@pytest.mark.parametrize("ctx,n,hq,d,f8", [(0, 64, 5, 128, False), (100, 63, 5, 128, False), (40, 50, 1, 64, True), (7, 33, 3, 256, False)])
def test_attention_rows_that_attend_one_drafted_token(ctx, n, hq, d, f8):
    """Every place of a tile is some row's only drafted token (and with ctx 0 its only token)."""
    p = Problem([ctx], [n], hq, 1, d, page=64, f8=f8, seed=60 + n)
    p.mask = mask_tensor([1 << ((7 * i + 3) % n) for i in range(n)], 1)
    p.check(*p.run())
