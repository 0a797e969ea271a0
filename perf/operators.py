"""Timing cases of the operators around the W12 products in one step of speculative decoding: the residual
addition with RMS norm (``add_rmsnorm``), rotary positions with the write into the paged cache
(``rope_append``), attention of a tree of drafted tokens over that cache (``tree_attention``) and the 8-bit
product with block scales (``gemm_e4m3``).

``run`` computes a case either with the library (``own`` true) or in its plain form, elementary torch operations
in 32 bits; ``exact`` computes it in 64 bits from the definitions.  Sizes come from the layer that the benchmark
uses (hidden size 5120, QKV of 40 + 2 x 8 heads of 128, gate_up 34816, down 5120 x 17408) and its row counts
(1..64 drafted tokens of one request, 512 rows of a batch); the others are generic.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
BLOCK = 128


# --------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token through a layer: the delay of a single small launch is all there is
        dict(name="norm_one_token", op="norm", m=1, n=5120, res="bf16", delta="f32", out="bf16"),
        # a 63-node tree before a layer that is there in W12 and, for the drafter, in 8 bits
        dict(name="norm_tree", op="norm", m=63, n=5120, res="bf16", delta="f32", out="both"),
        # admission of a long prompt in front of an 8-bit layer, residual kept in 32 bits
        dict(name="norm_prompt_e4m3", op="norm", m=4096, n=5120, res="f32", delta="f32", out="e4m3"),
        # one token: positions and cache write
        dict(name="rope_one_token", op="rope", t=1, hq=40, hkv=8, d=128, rot=128, axes=1, adjacent=False, src="f32",
             cache="bf16", page=64, heads_first=False, cached=8192, far=8191),
        # 512 rows of a batch with images or video in it: three axes, 8-bit cache
        dict(name="rope_batch_axes", op="rope", t=512, hq=40, hkv=8, d=128, rot=128, axes=3, adjacent=False, src="f32",
             cache="e4m3", page=64, heads_first=False, cached=16384, far=262143),
        # one token after a short prompt
        dict(name="attn_one_token", op="attn", b=1, nodes=1, ctx=509, hq=40, hkv=8, d=128, cache="bf16", page=64,
             heads_first=False, tree=False),
        # one request's tree of 63 nodes over a cache of ordinary length
        dict(name="attn_tree", op="attn", b=1, nodes=63, ctx=8191, hq=40, hkv=8, d=128, cache="bf16", page=64,
             heads_first=False, tree=True),
        # 16 requests of unequal lengths share a step of 24-node trees, 8-bit cache
        dict(name="attn_batch_e4m3", op="attn", b=16, nodes=24, ctx=8000, hq=40, hkv=8, d=128, cache="e4m3", page=64,
             heads_first=True, tree=True),
        # the largest tree over a very long cache
        dict(name="attn_long", op="attn", b=1, nodes=64, ctx=131001, hq=40, hkv=8, d=128, cache="bf16", page=64,
             heads_first=False, tree=True),
        # one token through the drafter's down projection
        dict(name="e4m3_one_token", op="gemm", m=1, n=5120, k=17408),
        # a block of 63 rows through gate_up
        dict(name="e4m3_tree", op="gemm", m=63, n=34816, k=5120),
        # 512 rows of a batch through gate_up
        dict(name="e4m3_batch", op="gemm", m=512, n=34816, k=5120),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("norm", "rope", "attn", "attn", "gemm", "gemm"))
    if op == "norm":
        n = _log(rng, 64, 17408)
        if rng.random() < 0.6:
            n = max(64, n // 64 * 64)
        m = min(_log(rng, 1, 4096), 4096 * 5120 // n)
        return dict(op="norm", m=m, n=n, res=rng.choice(("bf16", "f32")), delta=rng.choice(("f32", "bf16", "none")),
                    out=rng.choice(("bf16", "e4m3", "both")))
    if op == "gemm":
        while True:
            m, n, k = _log(rng, 1, 512), _log(rng, 64, 34816), _log(rng, 64, 17408)
            if rng.random() < 0.6:
                n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
            if n * k <= 34816 * 5120:
                return dict(op="gemm", m=m, n=n, k=k)
    d = rng.choice((64, 128, 128, 256))
    hkv = rng.choice((1, 2, 4, 8))
    g = rng.choice((1, 2, 4, 5, 8))
    cache = rng.choice(("bf16", "e4m3"))
    page = rng.choice((16, 32, 64, 128))
    heads_first = rng.random() < 0.3
    if op == "rope":
        return dict(op="rope", t=_log(rng, 1, 512), hq=hkv * g, hkv=hkv, d=d, rot=rng.choice((d, d, d // 2)),
                    axes=rng.choice((1, 2, 3)), adjacent=rng.random() < 0.3, src=rng.choice(("f32", "bf16")),
                    cache=cache, page=page, heads_first=heads_first, cached=_log(rng, 64, 16384),
                    far=_log(rng, 1000, 1000000))
    while True:
        b, nodes, ctx = _log(rng, 1, 32), _log(rng, 1, 64), _log(rng, 1, 131072)
        if b * ctx * hkv * d <= 131072 * 1024 and b * ctx * nodes * hkv * g * d <= 131072 * 64 * 5120:
            return dict(op="attn", b=b, nodes=nodes, ctx=ctx, hq=hkv * g, hkv=hkv, d=d, cache=cache, page=page,
                        heads_first=heads_first, tree=rng.random() < 0.7)


def _lengths(case):
    """Cached tokens and drafted nodes of every request: unequal in a batch, the same in every run of a case."""
    b, ctx, nodes = case["b"], case["ctx"], case["nodes"]
    if b == 1:
        return [ctx], [nodes]
    r = random.Random(b * 1000003 + ctx * 101 + nodes)
    return ([ctx] + [r.randint(ctx // 8, ctx) for _ in range(b - 1)],
            [nodes] + [r.randint(max(1, nodes // 2), nodes) for _ in range(b - 1)])


def work(case):
    size = {"bf16": 2, "f32": 4, "none": 0, "e4m3": 1}
    if case["op"] == "norm":
        m, n = case["m"], case["n"]
        per = 2 * size[case["res"]] + size[case["delta"]] - (size[case["res"]] if case["delta"] == "none" else 0)
        per += 2 * (case["out"] in ("bf16", "both")) + 1 * (case["out"] in ("e4m3", "both"))
        scales = 4 * m * -(-n // BLOCK) * (case["out"] != "bf16")
        return {"bytes": m * n * per + 2 * n + scales, "flops": 6 * m * n}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        return {"bytes": n * k + m * k + 4 * m * n + 4 * m * kb + 4 * -(-n // BLOCK) * kb, "flops": 2 * m * n * k}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        t = case["t"]
        return {"bytes": t * d * ((hq + 2 * hkv) * size[case["src"]] + hq * 2 + 2 * hkv * size[case["cache"]]) + 8 * t
                + 4 * t * case["axes"], "flops": 3 * t * d * (hq + hkv)}
    ctxs, nodes = _lengths(case)
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctxs, nodes))
    toks = sum(c + n for c, n in zip(ctxs, nodes))
    return {"bytes": 2 * toks * hkv * d * size[case["cache"]] + 4 * sum(nodes) * hq * d + 8 * sum(nodes),
            "flops": 4 * pairs * hq * d}


# -------------------------------------------------------------------------------------------- inputs

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _cache_tensors(case, pages, gen):
    """K and V of a paged cache [pages, page, heads, dim], filled; e4m3 caches have a scale per head."""
    page, hkv, d = case["page"], case["hkv"], case["d"]
    shape = (pages, hkv, page, d) if case["heads_first"] else (pages, page, hkv, d)
    kv, scales = [], []
    for _ in range(2):
        x = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
        if case["cache"] == "e4m3":
            s = torch.empty(hkv, device=DEV).uniform_(0.008, 0.015, generator=gen)
            sb = s[None, :, None, None] if case["heads_first"] else s[None, None, :, None]
            x = _quantised(x, sb)
            scales.append(s)
        kv.append(x.transpose(1, 2) if case["heads_first"] else x)
    return kv[0], kv[1], (scales or [None, None])


def _quantised(x, sb):
    out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    step = max(1, x.shape[0] // 8)
    for i in range(0, x.shape[0], step):
        out[i:i + step] = (x[i:i + step].float() / sb).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)
    return out.view(E4M3)


def _inv_freq(rot):
    return (1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).to(DEV)


def _ancestors(r, n):
    """Bit sets of a random tree in drafting order: node 0 is the root, every node attends itself and its ancestors."""
    bits = [1]
    for i in range(1, n):
        bits.append(bits[r.randint(max(0, i - 12), i - 1)] | (1 << i))
    return bits


def prepare(case, seed):
    if own:
        import lossless_bit_weight_encode_amd as w12
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = random.Random(seed)
    s = dict(case=case)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.empty(shape, device=DEV).normal_(generator=gen) * scale).to(dtype)

    if case["op"] == "norm":
        m, n = case["m"], case["n"]
        ld = (n + 7) // 8 * 8                       # rows are padded to 16 bytes, as the products want them
        s["residual"] = randn(m, ld, dtype=DT[case["res"]], scale=2.0)[:, :n]
        s["delta"] = None if case["delta"] == "none" else randn(m, ld, dtype=DT[case["delta"]], scale=0.5)[:, :n]
        s["weight"] = (1 + randn(n, scale=0.1)).to(torch.bfloat16)
        s["residual_out"] = None if s["delta"] is None else torch.empty(m, ld, dtype=DT[case["res"]], device=DEV)[:, :n]
        s["y"] = torch.empty(m, ld, dtype=torch.bfloat16, device=DEV)[:, :n] if case["out"] != "e4m3" else None
        s["yq"] = s["yq_scale"] = None
        if case["out"] != "bf16":
            s["yq"] = torch.empty(m, (n + 15) // 16 * 16, dtype=E4M3, device=DEV)[:, :n]
            s["yq_scale"] = torch.empty(m, -(-n // BLOCK), device=DEV)
        return s
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        ld, kb = (k + 15) // 16 * 16, -(-k // BLOCK)
        s["x"] = randn(m, ld, scale=100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3)[:, :k]
        w = torch.empty(n, ld, dtype=torch.uint8, device=DEV)
        for i in range(0, n, 4096):
            w[i:i + 4096] = randn(min(4096, n - i), ld, scale=100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)
        s["w"] = w.view(E4M3)[:, :k]
        s["x_scale"] = torch.empty(m, kb, device=DEV).uniform_(0.005, 0.015, generator=gen)
        s["w_scale"] = torch.empty(-(-n // BLOCK), kb, device=DEV).uniform_(0.0001, 0.0003, generator=gen)
        s["y"] = torch.empty(m, n, device=DEV)
        s["ws"] = w12.gemm_e4m3_workspace(m, n, k, DEV) if own else None
        return s
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    if case["op"] == "rope":
        t = case["t"]
        pages = -(-(case["cached"] + t) // page)
        s["k"], s["v"], (s["k_scale"], s["v_scale"]) = _cache_tensors(case, pages, gen)
        s["qkv"] = randn(t, (hq + 2 * hkv) * d, dtype=DT[case["src"]])
        pos = torch.randint(0, case["far"] + 1, (case["axes"], t), generator=gen, device=DEV, dtype=torch.int32)
        pos[0] = case["far"] - t + 1 + torch.arange(t, device=DEV, dtype=torch.int32) if case["far"] >= t else pos[0]
        s["positions"] = pos
        # the rows' places: t different tokens of the cache
        s["slots"] = torch.randperm(pages * page, generator=gen, device=DEV)[:t].sort().values
        s["inv_freq"] = _inv_freq(case["rot"])
        s["axis"] = (torch.arange(case["rot"] // 2, device=DEV) * case["axes"] // (case["rot"] // 2)).to(torch.uint8)
        s["q"] = torch.empty(t, hq * d, dtype=torch.bfloat16, device=DEV)
    else:
        ctxs, nodes = _lengths(case)
        per = -(-max(c + n for c, n in zip(ctxs, nodes)) // page)
        need = [-(-(c + n) // page) for c, n in zip(ctxs, nodes)]
        s["k"], s["v"], (s["k_scale"], s["v_scale"]) = _cache_tensors(case, sum(need), gen)
        order = torch.randperm(sum(need), generator=gen, device=DEV).to(torch.int32)
        table = torch.zeros(case["b"], per, dtype=torch.int32, device=DEV)
        at = 0
        for i, p in enumerate(need):
            table[i, :p] = order[at:at + p]
            at += p
        s["page_table"] = table
        ptr = [0]
        for n in nodes:
            ptr.append(ptr[-1] + n)
        s["q"] = randn(ptr[-1], hq * d, dtype=torch.bfloat16, scale=2.0)
        s["ctx_len"] = torch.tensor(ctxs, dtype=torch.int32, device=DEV)
        s["node_ptr"] = torch.tensor(ptr, dtype=torch.int32, device=DEV)
        s["max_nodes"] = case["nodes"]
        s["tree_mask"] = None
        if case["tree"]:
            bits = [b for n in nodes for b in _ancestors(r, n)]
            s["tree_mask"] = torch.tensor([[b - (1 << 64) if b >> 63 else b] for b in bits], dtype=torch.int64, device=DEV)
        s["out"] = torch.empty(ptr[-1], hq * d, dtype=torch.bfloat16, device=DEV)
    # the handle of the cache and the workspace, which a program makes once beside its cache
    s["cache"] = s["ws"] = None
    if own:
        s["cache"] = w12.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if case["op"] == "attn":
            s["ws"] = w12.tree_attention_workspace(s["q"].shape[0], case["b"], hq, s["cache"])
    return s


# ----------------------------------------------------------------------------------------------- run

def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_norm(s):
    import lossless_bit_weight_encode_amd as w12
    w12.add_rmsnorm(s["residual"], s["weight"], s["delta"], eps=1e-6, residual_out=s["residual_out"], y=s["y"],
                    yq=s["yq"], yq_scale=s["yq_scale"])
    return {"residual": s["residual_out"], "y": s["y"], "yq": s["yq"], "yq_scale": s["yq_scale"]}


def _own_rope(s):
    import lossless_bit_weight_encode_amd as w12
    w12.rope_append(s["qkv"], s["cache"], s["positions"], s["slots"], s["inv_freq"], s["case"]["hq"], axis=s["axis"],
                    adjacent=s["case"]["adjacent"], q=s["q"])
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def _own_attn(s):
    import lossless_bit_weight_encode_amd as w12
    return w12.tree_attention(s["q"], s["cache"], s["page_table"], s["ctx_len"], s["node_ptr"], tree_mask=s["tree_mask"],
                              out=s["out"], ws=s["ws"])


def _own_gemm(s):
    import lossless_bit_weight_encode_amd as w12
    return w12.gemm_e4m3(s["x"], s["x_scale"], s["w"], s["w_scale"], y=s["y"], ws=s["ws"])


def _plain_norm(s):
    r = s["residual"].float()
    if s["delta"] is not None:
        r = r + s["delta"].float()
    y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-6) * s["weight"].float()
    yq = scale = None
    if s["yq"] is not None:
        m, n = y.shape
        nb = -(-n // BLOCK)
        yb = torch.nn.functional.pad(y, (0, nb * BLOCK - n)).view(m, nb, BLOCK)
        amax = yb.abs().amax(2)
        scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
        yq = (yb / scale[:, :, None]).reshape(m, nb * BLOCK)[:, :n].to(E4M3)
    return {"residual": None if s["delta"] is None else r.to(s["residual"].dtype),
            "y": None if s["y"] is None else y.to(torch.bfloat16), "yq": yq, "yq_scale": scale}


def _plain_rope(s):
    c = s["case"]
    t, hq, hkv, d, rot = c["t"], c["hq"], c["hkv"], c["d"], c["rot"]
    ang = s["positions"].double()[s["axis"].long()].t() * s["inv_freq"]            # [t, rot / 2]
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    x = s["qkv"].float().view(t, hq + 2 * hkv, d)
    qk, v = x[:, :hq + hkv], x[:, hq + hkv:]
    part = qk[..., :rot]
    if c["adjacent"]:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    qk = torch.cat((part, qk[..., rot:]), -1)
    k = qk[:, hq:]
    page, off = s["slots"] // c["page"], s["slots"] % c["page"]
    if c["cache"] == "e4m3":
        for dst, src, sc in ((s["k"], k, s["k_scale"]), (s["v"], v, s["v_scale"])):
            dst.view(torch.uint8)[page, off] = (src / sc[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3).view(torch.uint8)
    else:
        s["k"][page, off] = k.to(torch.bfloat16)
        s["v"][page, off] = v.to(torch.bfloat16)
    return {"q": qk[:, :hq].to(torch.bfloat16).reshape(t, hq * d), "k": s["k"], "v": s["v"]}


def _plain_attn(s):
    c = s["case"]
    b, n, hq, hkv, d = c["b"], s["max_nodes"], c["hq"], c["hkv"], c["d"]
    table = s["page_table"].long()
    length = table.shape[1] * c["page"]

    def gather(x, scale):
        x = x.view(torch.uint8)[table].view(E4M3).float() if c["cache"] == "e4m3" else x[table].float()
        x = x.reshape(b, length, hkv, d).transpose(1, 2)
        return x * scale[None, :, None, None] if scale is not None else x

    t = s["q"].shape[0]
    row = torch.arange(t, device=DEV)
    req = torch.searchsorted(s["node_ptr"][1:].contiguous(), row.int(), right=True)
    node = row - s["node_ptr"].long()[req]
    q = torch.zeros(b, n, hkv, hq // hkv, d, device=DEV)
    q[req, node] = s["q"].float().view(t, hkv, hq // hkv, d)
    # which drafted nodes a node attends: its ancestors, or in a chain all before it, and itself
    j = torch.arange(n, device=DEV)
    sees = torch.zeros(b, n, n, dtype=torch.bool, device=DEV)
    if s["tree_mask"] is not None:
        sees[req, node] = ((s["tree_mask"][:, j // 64] >> (j % 64)) & 1).bool()
    else:
        sees[req, node] = j[None, :] <= node[:, None]
    at = torch.arange(length, device=DEV)[None, :] - s["ctx_len"].long()[:, None]      # [b, length]
    keep = (at < 0)[:, None, :] | ((at >= 0) & (at < n))[:, None, :] & sees.gather(2, at.clamp(0, n - 1)[:, None, :].expand(b, n, length))
    q = q.permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)                                # [b, hkv, g n, d]
    p = torch.matmul(q, gather(s["k"], s["k_scale"]).transpose(2, 3)) / math.sqrt(d)
    p = p.view(b, hkv, hq // hkv, n, length).masked_fill_(~keep[:, None, None], -math.inf)
    top = p.amax(4, keepdim=True)
    p = (p - torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(4, keepdim=True)
    o = torch.matmul(p.view(b, hkv, -1, length), gather(s["v"], s["v_scale"])).view(b, hkv, hq // hkv, n, d)
    o = o / torch.where(total == 0, 1.0, total)
    return o.permute(0, 3, 1, 2, 4)[req, node].to(torch.bfloat16).reshape(t, hq * d)


def _plain_gemm(s):
    n, k = s["w"].shape
    x = s["x"].float() * s["x_scale"].repeat_interleave(BLOCK, 1)[:, :k]
    w = s["w"].float() * s["w_scale"].repeat_interleave(BLOCK, 1)[:, :k].repeat_interleave(BLOCK, 0)[:n]
    return x @ w.t()


_run_own = {"norm": _own_norm, "rope": _own_rope, "attn": _own_attn, "gemm": _own_gemm}
_run_plain = {"norm": _plain_norm, "rope": _plain_rope, "attn": _plain_attn, "gemm": _plain_gemm}


# --------------------------------------------------------------------------------------------- exact

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"norm": _exact_norm, "rope": _exact_rope, "attn": _exact_attn, "gemm": _exact_gemm}[case["op"]](s)


def _exact_norm(s):
    r = s["residual"].double()
    d = s["delta"]
    if d is not None:
        r += d.double()
    m, n = r.shape
    y = s["weight"].double() * r / torch.sqrt(torch.linalg.vector_norm(r, dim=1, keepdim=True) ** 2 / n + 1e-6)
    scale = yq = None
    if s["yq"] is not None:
        scale = torch.ones(m, -(-n // BLOCK), dtype=torch.float64, device=DEV)
        yq = torch.empty_like(y)
        for i in range(scale.shape[1]):
            blk = y[:, i * BLOCK:(i + 1) * BLOCK]
            top = blk.abs().max(1).values
            scale[:, i] = torch.where(top > 0, top / E4M3_MAX, scale[:, i])
            yq[:, i * BLOCK:(i + 1) * BLOCK] = blk / scale[:, i:i + 1]
    return {"residual": None if d is None else r, "y": None if s["y"] is None else y, "yq": yq, "yq_scale": scale}


def _exact_rope(s):
    c = s["case"]
    hq, hkv, d, half = c["hq"], c["hkv"], c["d"], c["rot"] // 2
    x = s["qkv"].double().reshape(c["t"], -1, d)
    out = x.clone()
    for i in range(half):
        th = s["positions"][int(s["axis"][i])].double() * s["inv_freq"][i]
        z = torch.polar(torch.ones_like(th), th)[:, None]
        lo, hi = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + half)
        w = torch.complex(x[:, :hq + hkv, lo], x[:, :hq + hkv, hi]) * z
        out[:, :hq + hkv, lo], out[:, :hq + hkv, hi] = w.real, w.imag
    k, v = s["k"].double(), s["v"].double()
    page, off = s["slots"] // c["page"], s["slots"] % c["page"]
    new_k, new_v = out[:, hq:hq + hkv], out[:, hq + hkv:]
    if c["cache"] == "e4m3":
        new_k = (new_k / s["k_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        new_v = (new_v / s["v_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    k[page, off] = new_k
    v[page, off] = new_v
    return {"q": out[:, :hq].reshape(c["t"], hq * d), "k": k, "v": v}


def _exact_attn(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    g = hq // hkv
    ctxs, nodes = _lengths(c)
    out = torch.empty(s["q"].shape[0], hq, d, dtype=torch.float64, device=DEV)
    row = 0
    for b, (ctx, n) in enumerate(zip(ctxs, nodes)):
        tok = torch.arange(ctx + n, device=DEV)
        page, off = s["page_table"][b].long()[tok // c["page"]], tok % c["page"]
        allow = torch.ones(n, ctx + n, dtype=torch.bool, device=DEV)
        if s["tree_mask"] is None:
            allow[:, ctx:] = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        else:
            for j in range(n):
                allow[:, ctx + j] = (s["tree_mask"][row:row + n, j // 64] >> (j % 64)) % 2 != 0
        for h in range(hkv):
            if c["cache"] == "bf16":
                kh, vh = s["k"][:, :, h][page, off].double(), s["v"][:, :, h][page, off].double()
            else:
                kh = s["k"].view(torch.uint8)[:, :, h][page, off].view(E4M3).double() * s["k_scale"][h].double()
                vh = s["v"].view(torch.uint8)[:, :, h][page, off].view(E4M3).double() * s["v_scale"][h].double()
            for i in range(g):
                q = s["q"][row:row + n, (h * g + i) * d:(h * g + i + 1) * d].double()
                sc = torch.where(allow, q @ kh.t() * d ** -0.5, -math.inf)
                out[row:row + n, h * g + i] = torch.exp(sc - torch.logsumexp(sc, 1, keepdim=True)) @ vh
        row += n
    return out.reshape(row, hq * d)


def _exact_gemm(s):
    m, k = s["x"].shape
    y = torch.zeros(m, s["w"].shape[0], dtype=torch.float64, device=DEV)
    for i in range(0, k, BLOCK):
        part = s["x"][:, i:i + BLOCK].double() @ s["w"][:, i:i + BLOCK].double().t()
        part *= s["x_scale"][:, i // BLOCK].double()[:, None]
        y += part * s["w_scale"][:, i // BLOCK].double().repeat_interleave(BLOCK)[None, :y.shape[1]]
    return y
