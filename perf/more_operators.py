"""Timing cases of the operators that a hybrid target needs in speculative decoding, beside those of ``operators.py``:
the gated delta rule of its recurrent layers (``gated_delta``: prompts in chunks, single tokens, chains and trees of
drafted tokens over a state that stays as it is, and the accepted path's way into the state), the short causal
convolution in front of it (``short_conv``), and the verification of the drafted tokens against the target's
probabilities (``verify_draft``).

``run`` computes a case either with the library (``own`` true) or in its plain form, elementary torch operations in
32 bits (64 for sums of log decays and for the borders of a cumulative distribution); ``exact`` computes it in 64 bits
from the definitions.  Row counts are the benchmark's (1..64 drafted tokens of one request, 16 x 24 of a batch); heads
of 128, 16 for keys and 48 for values, stand for a layer of the benchmark's hidden size, 10240 channels for its
queries, keys and values together; the other sizes are generic.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
CHUNK = 64
MAX_TREE = 64
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # plain decoding of one request: a token's update of every head's state, and its output
        dict(name="delta_one_token", op="delta", form="seq", b=1, n=1, hk=16, hv=48, dk=128, dv=128, l2=True),
        # the same for a full batch: states read and written are all there is
        dict(name="delta_decode_batch", op="delta", form="seq", b=64, n=1, hk=16, hv=48, dk=128, dv=128, l2=True),
        # one prompt, from the state of a cached prefix
        dict(name="delta_prompt", op="delta", form="seq", b=1, n=4096, hk=16, hv=48, dk=128, dv=128, l2=True),
        # prompts of unequal lengths that are admitted together
        dict(name="delta_prompts_ragged", op="delta", form="seq", b=7, n=5003, hk=16, hv=32, dk=128, dv=128, l2=True),
        # one request's tree of 63 nodes: outputs for every node, the state stays
        dict(name="delta_tree", op="delta", form="tree", b=1, n=63, hk=16, hv=48, dk=128, dv=128, l2=True),
        # 16 requests share a step of 24-node trees
        dict(name="delta_tree_batch", op="delta", form="tree", b=16, n=24, hk=16, hv=48, dk=128, dv=128, l2=True),
        # and their accepted paths move the states on
        dict(name="delta_accept_batch", op="delta", form="accept", b=16, n=24, hk=16, hv=48, dk=128, dv=128, l2=True),
        # a tree's rows of the product in front, every node on its own path
        dict(name="conv_tree", op="conv", form="tree", b=1, n=63, c=10240, w=4, src="f32", bias=False),
        # a prompt's
        dict(name="conv_prompt", op="conv", form="seq", b=1, n=4096, c=10240, w=4, src="f32", bias=False),
        # a chain of 16 drafted tokens with the drafter's probabilities, an odd vocabulary
        dict(name="verify_chain", op="verify", form="chain", b=1, n=17, v=50257, q=True, temps="one"),
        # one request's tree of 63 nodes
        dict(name="verify_tree", op="verify", form="tree", b=1, n=63, v=131072, q=False, temps="one"),
        # 16 requests, some greedy, some sampled at temperatures of their own
        dict(name="verify_batch", op="verify", form="tree", b=16, n=24, v=131072, q=False, temps="mixed"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("delta", "delta", "delta", "conv", "verify"))
    if op == "delta":
        form = rng.choice(("seq", "seq", "tree", "accept"))
        while True:
            hk = rng.choice((1, 2, 4, 8, 16))
            hv = hk * rng.choice((1, 2, 3, 4))
            dk, dv = rng.choice((64, 128, 128)), rng.choice((64, 128, 128, 256))
            b = _log(rng, 1, 64)
            n = _log(rng, 1, 5003 if form == "seq" else MAX_TREE)
            state = b * hv * dk * dv
            if b * n * hv * dk * dv <= 20000 * 32 * 128 * 128 and state <= 64 * 48 * 128 * 128:
                return dict(op="delta", form=form, b=b, n=n, hk=hk, hv=hv, dk=dk, dv=dv, l2=rng.random() < 0.8)
    if op == "conv":
        while True:
            form = rng.choice(("seq", "tree", "accept"))
            b, c = _log(rng, 1, 64), _log(rng, 64, 16384)
            if rng.random() < 0.7:
                c = max(64, c // 64 * 64)
            n = _log(rng, 1, 4096 if form == "seq" else MAX_TREE)
            if b * n * c <= 4096 * 10240:
                return dict(op="conv", form=form, b=b, n=n, c=c, w=rng.choice((2, 3, 4, 4)), src=rng.choice(("f32", "bf16")),
                            bias=rng.random() < 0.3)
    while True:
        form = rng.choice(("chain", "tree"))
        b, n, v = _log(rng, 1, 32), _log(rng, 1, 64), _log(rng, 1000, 160000)
        if b * n * v <= 384 * 131072:
            return dict(op="verify", form=form, b=b, n=n, v=v, q=form == "chain" and rng.random() < 0.6,
                        temps=rng.choice(("one", "mixed")))


def _lengths(case):
    """Rows of every sequence: unequal in a batch of more than single rows, the same in every run of a case."""
    b, n = case["b"], case["n"]
    r = random.Random(b * 1000003 + n)
    return [n] + [r.randint(max(1, n // 3), n) for _ in range(b - 1)]


def _accepted(case):
    """How many nodes of each request were accepted, the first among them: the same in every run of a case."""
    r = random.Random(case["b"] * 77 + case["n"])
    return [r.randint(1, min(n, 12)) for n in _lengths(case)]


def work(case):
    size = {"bf16": 2, "f32": 4}
    rows = sum(_lengths(case))
    if case["op"] == "delta":
        hk, hv, dk, dv, b = case["hk"], case["hv"], case["dk"], case["dv"], case["b"]
        used = sum(_accepted(case)) if case["form"] == "accept" else rows
        out = 0 if case["form"] == "accept" else 1
        per = 2 * (hk * dk * (1 + out) + hv * dv * (1 + out)) + 8 * hv
        states = 4 * b * hv * dk * dv
        return {"bytes": used * per + states * (1 if case["form"] == "tree" else 2),
                "flops": used * hv * dk * dv * (4 + 2 * out)}
    if case["op"] == "conv":
        c, w, b = case["c"], case["w"], case["b"]
        used = sum(_accepted(case)) if case["form"] == "accept" else rows
        x = size[case["src"]]
        states = b * (w - 1) * c * x
        out = 0 if case["form"] == "accept" else 2
        read = b * min(w - 1, case["n"]) * c * x if case["form"] == "accept" else used * c * x
        return {"bytes": read + used * c * out + states * (1 if case["form"] == "tree" else 2) + 2 * c * w,
                "flops": 2 * used * c * w if out else 0}
    v, b = case["v"], case["b"]
    return {"bytes": 4 * rows * v + (4 * b * v if case["q"] else 0) + 24 * rows, "flops": 4 * rows * v}


# -------------------------------------------------------------------------------------------- inputs

def _parents(r, n):
    """A random tree in drafting order: node 0 is the root."""
    return [-1] + [r.randint(max(0, i - 12), i - 1) for i in range(1, n)]


def _mask(parents):
    """Bit sets of the nodes: a node and its ancestors, as int64."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((1 << i) | (bits[p] if p >= 0 else 0))
    return [x - (1 << 64) if x >> 63 else x for x in bits]


def _ptr(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def _rows_of(s, r, form, lengths):
    """What every operator here is told of its rows: the ranges, the trees, the accepted paths."""
    ptr = _ptr(lengths)
    s["lengths"], s["seq_ptr"] = lengths, _ints(ptr)
    s["tree_mask"] = s["lens"] = s["rows"] = s["parents"] = None
    if form == "tree":
        s["parents"] = [_parents(r, n) for n in lengths]
        s["tree_mask"] = _ints([b for p in s["parents"] for b in _mask(p)], torch.int64).view(-1, 1)
    if form == "accept":
        s["taken"] = _accepted(s["case"])
        rows = [-1] * ptr[-1]
        for b, n in enumerate(lengths):
            path = [0] + sorted(r.sample(range(1, n), s["taken"][b] - 1))
            rows[ptr[b]:ptr[b] + len(path)] = [ptr[b] + i for i in path]
        s["lens"], s["rows"] = _ints(s["taken"]), _ints(rows)


def _slots(s, r, b, stores):
    """Places of the sequences' states: the new ones go to places of their own, so that a pass can be repeated."""
    order = list(range(2 * b if stores else b))
    r.shuffle(order)
    s["src"], s["dst"] = _ints(order[:b]), _ints(order[b:]) if stores else None
    s["places"] = (order[:b], order[b:])
    return len(order)


def prepare(case, seed):
    if own:
        import lossless_bit_weight_encode_amd as w12
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = random.Random(seed)
    s = dict(case=case)
    lengths = _lengths(case)
    t = sum(lengths)

    def randn(*shape, scale=1.0, dtype=torch.float32):
        return (torch.empty(shape, device=DEV).normal_(generator=gen) * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.empty(shape, device=DEV).uniform_(lo, hi, generator=gen)

    _rows_of(s, r, case["form"], lengths)
    if case["op"] == "conv":
        c, w, dt = case["c"], case["w"], DT[case["src"]]
        ld = (c + 7) // 8 * 8                          # rows are padded to 16 bytes, as the products want them
        s["x"] = randn(t, ld, dtype=dt)[:, :c]
        s["weight"] = randn(c, w, scale=w ** -0.5, dtype=torch.bfloat16)
        s["bias"] = randn(c, scale=0.1, dtype=torch.bfloat16) if case["bias"] else None
        slots = _slots(s, r, case["b"], case["form"] != "tree")
        s["state"] = randn(slots, w - 1, ld, dtype=dt)[:, :, :c]
        s["y"] = None if case["form"] == "accept" else torch.empty(t, ld, dtype=torch.bfloat16, device=DEV)[:, :c]
        return s
    if case["op"] == "delta":
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        # queries, keys and values lie side by side, as the convolution leaves them
        x = torch.nn.functional.silu(randn(t, 2 * hk * dk + hv * dv))
        if not case["l2"]:
            x[:, :2 * hk * dk] *= dk ** -0.5           # keys of norms under 1, as a layer without the norm has to see to
        x = x.to(torch.bfloat16)
        s["q"], s["k"], s["v"] = x.split((hk * dk, hk * dk, hv * dv), 1)
        # heads forget at rates from 1 in 1000 tokens to several a token
        rate = torch.exp(uniform(hv, lo=math.log(0.001), hi=math.log(2.0)))
        s["g"] = -rate * torch.nn.functional.softplus(randn(t, hv) + 0.5)
        s["beta"] = torch.sigmoid(randn(t, hv))
        slots = _slots(s, r, case["b"], case["form"] != "tree")
        s["state"] = randn(slots, hv, dv, dk, scale=0.3)
        s["out"] = None if case["form"] == "accept" else torch.empty(t, hv * dv, dtype=torch.bfloat16, device=DEV)
        s["ws"] = w12.gated_delta_workspace(t, case["b"], s["state"]) if own else None
        return s
    v, b = case["v"], case["b"]
    ld = (v + 7) // 8 * 8
    ptr = _ptr(lengths)
    parents = [[i - 1 for i in range(n)] for n in lengths] if case["form"] == "chain" else s["parents"]
    up = _ints([ptr[i] + max(p, 0) for i, ps in enumerate(parents) for p in ps], torch.int64)    # a row's parent row
    logits = randn(t, ld, scale=2.0)[:, :v]
    # most of a row's mass lies on a few tokens
    top = torch.randint(0, v, (t, 8), generator=gen, device=DEV)
    logits.scatter_(1, top, 13.0 - 0.5 * torch.arange(8, device=DEV) + randn(t, 8))
    s["logits"] = logits
    s["temperature"] = torch.ones(b, device=DEV)
    if case["temps"] == "mixed":
        s["temperature"] = torch.where(uniform(b) < 0.3, 0.0, uniform(b, lo=0.5, hi=1.5))
    s["q"] = None
    if case["q"]:
        s["q"] = torch.empty(t, ld, device=DEV)[:, :v]
        s["q"].copy_(torch.softmax(logits[up] + randn(t, v, scale=0.5), 1))
        s["tokens"] = torch.multinomial(s["q"], 1, generator=gen)[:, 0].to(torch.int32)
    else:
        # what a drafter proposes is often what the target would say after the node's parent
        kind = torch.randint(0, 4, (t,), generator=gen, device=DEV)
        s["tokens"] = top[up, kind % 3].to(torch.int32)
        s["tokens"] = torch.where(kind < 3, s["tokens"], torch.randint(0, v, (t,), generator=gen, device=DEV, dtype=torch.int32))
    s["u"], s["accept_u"] = uniform(t), uniform(t) if case["q"] else None
    s["path"] = torch.empty(t, dtype=torch.int32, device=DEV)
    s["count"], s["next"] = (torch.empty(b, dtype=torch.int32, device=DEV) for _ in range(2))
    s["parent_rows"] = parents
    s["ws"] = w12.verify_draft_workspace(t, b, v) if own else None
    return s


# ----------------------------------------------------------------------------------------------- run

def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_delta(s):
    import lossless_bit_weight_encode_amd as w12
    takes = s["case"]["form"] == "accept"
    out = w12.gated_delta(None if takes else s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["seq_ptr"], s["src"],
                          dst=s["dst"], l2norm=s["case"]["l2"], tree_mask=s["tree_mask"], lens=s["lens"], rows=s["rows"],
                          out=s["out"], outputs=not takes, ws=s["ws"])
    return {"out": out, "state": None if s["dst"] is None else s["state"]}


def _own_conv(s):
    import lossless_bit_weight_encode_amd as w12
    y = w12.short_conv(s["x"], s["weight"], s["state"], s["seq_ptr"], s["src"], dst=s["dst"], bias=s["bias"],
                       tree_mask=s["tree_mask"], lens=s["lens"], rows=s["rows"], y=s["y"],
                       outputs=s["case"]["form"] != "accept")
    return {"y": y, "state": None if s["dst"] is None else s["state"]}


def _own_verify(s):
    import lossless_bit_weight_encode_amd as w12
    w12.verify_draft(s["logits"], s["tokens"], s["u"], s["seq_ptr"], tree_mask=s["tree_mask"], q=s["q"],
                     accept_u=s["accept_u"], temperature=s["temperature"], path=s["path"], count=s["count"],
                     next_token=s["next"], ws=s["ws"])
    return {"path": s["path"], "count": s["count"], "next": s["next"]}


def _padded(s):
    """Row of every (sequence, place) and whether there is one."""
    t, b = s["seq_ptr"], s["case"]["b"]
    first, n = t[:-1].long(), (t[1:] - t[:-1]).long()
    if s["lens"] is not None:
        n = torch.minimum(n, s["lens"].long())
    at = torch.arange(min(MAX_TREE, s["case"]["n"]) if s["lens"] is not None else s["case"]["n"], device=DEV)
    there = at[None] < n[:, None]
    row = torch.where(there, first[:, None] + at[None], 0)
    if s["rows"] is not None:
        row = s["rows"].long()[row].clamp(min=0)
    return row.view(b, -1), there


def _chunk_terms(q, k, v, g, beta, anc, scale):
    """One chunk of every sequence and head: what does not depend on the state.  anc[i][j]: j is before i (or before i
    on its path); total decay of a row from the chunk's start, in 64 bits."""
    own_path = anc | torch.eye(anc.shape[-1], dtype=torch.bool, device=DEV)
    total = own_path.double() @ g.double()[..., None]                                     # [.., n, 1]
    decay = torch.exp((total - total.transpose(-1, -2)).float())
    zero = torch.zeros((), device=DEV)
    a = torch.where(anc, beta[..., None] * decay * (k @ k.transpose(-1, -2)), zero)
    n = a.shape[-1]
    inv = torch.eye(n, device=DEV).expand(a.shape).clone()
    for i in range(1, n):
        inv[..., i, :i] = -(a[..., i:i + 1, :i] @ inv[..., :i, :i])[..., 0, :]
    p = torch.where(own_path, scale * decay * (q @ k.transpose(-1, -2)), zero)
    total = total.float()
    return inv, p, torch.exp(total), torch.exp(total[..., -1:, :] - total)


def _plain_delta(s):
    c = s["case"]
    b, hk, hv, dk, dv = c["b"], c["hk"], c["hv"], c["dk"], c["dv"]
    row, there = _padded(s)
    n = row.shape[1]
    scale = dk ** -0.5
    step = n if s["tree_mask"] is not None else min(n, CHUNK)
    chunks = -(-n // step)
    row = torch.nn.functional.pad(row, (0, chunks * step - n))
    there = torch.nn.functional.pad(there, (0, chunks * step - n))

    def heads(x, h, d, group):
        x = x[row].float().view(b, chunks, step, h, d).permute(0, 3, 1, 2, 4)             # [b, h, chunks, step, d]
        x = torch.where(there.view(b, 1, chunks, step, 1), x, torch.zeros((), device=DEV))
        return x.repeat_interleave(group, 1)

    q, k, v = heads(s["q"], hk, dk, hv // hk), heads(s["k"], hk, dk, hv // hk), heads(s["v"], hv, dv, 1)
    if c["l2"]:
        q, k = (x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
    g, beta = heads(s["g"], hv, 1, 1)[..., 0], heads(s["beta"], hv, 1, 1)[..., 0]
    if s["tree_mask"] is not None:
        j = torch.arange(step, device=DEV)
        m = (s["tree_mask"][:, 0][row][..., None] >> j) & 1
        anc = (m.bool() & (j[None, :] < j[:, None]) & there[:, :, None]).view(b, 1, 1, step, step)
    else:
        anc = torch.ones(step, step, dtype=torch.bool, device=DEV).tril(-1)
    inv, p, grown, left = _chunk_terms(q, k, v, g, beta, anc, scale)
    state = s["state"][s["src"].long()].transpose(-1, -2)                                 # [b, hv, dk, dv]
    out = []
    for i in range(chunks):
        ki, bi, gi = k[:, :, i], beta[:, :, i, :, None], grown[:, :, i]
        u = inv[:, :, i] @ (bi * (v[:, :, i] - gi * (ki @ state)))
        if s["out"] is not None:
            out.append(scale * gi * (q[:, :, i] @ state) + p[:, :, i] @ u)
        if s["dst"] is not None:
            state = gi[..., -1:, :] * state + (ki * left[:, :, i]).transpose(-1, -2) @ u
    if s["out"] is not None:
        o = torch.cat(out, 2).permute(0, 2, 1, 3).reshape(b, chunks * step, hv * dv)
        s["out"][row[there]] = o[there].to(torch.bfloat16)
    if s["dst"] is not None:
        s["state"][s["dst"].long()] = state.transpose(-1, -2)
    return {"out": s["out"], "state": None if s["dst"] is None else s["state"]}


def _plain_conv(s):
    c = s["case"]
    b, w = c["b"], c["w"]
    row, there = _padded(s)
    n = row.shape[1]
    x = s["x"][row].float()                                                               # [b, n, c]
    past = s["state"][s["src"].long()].float()                                            # [b, w - 1, c], oldest first
    line = torch.cat((past, x), 1)
    if s["y"] is not None:
        place = torch.arange(n, device=DEV)[None].expand(b, n)
        if s["tree_mask"] is not None:
            j = torch.arange(n, device=DEV)
            m = (s["tree_mask"][:, 0][row][..., None] >> j) & 1
            before = torch.where(m.bool() & (j[None, :] < j[:, None]), j, -1).amax(2)     # the parent's place
        y = torch.zeros(b, n, c["c"], device=DEV) if s["bias"] is None else s["bias"].float().expand(b, n, -1).clone()
        wt = s["weight"].float()
        for tap in range(w):
            at = (w - 1 + place).clamp(min=0)
            y += wt[:, w - 1 - tap] * line.gather(1, at[..., None].expand(-1, -1, c["c"]))
            place = place - 1 if s["tree_mask"] is None else torch.where(
                place >= 0, before.gather(1, place.clamp(min=0)), place - 1)
        y = y * torch.sigmoid(y)
        s["y"][row[there]] = y[there].to(torch.bfloat16)
    if s["dst"] is not None:
        at = there.sum(1)[:, None] + torch.arange(w - 1, device=DEV)
        new = line.gather(1, at[..., None].expand(-1, -1, c["c"]))
        s["state"][s["dst"].long()] = new.to(s["state"].dtype)
    return {"y": s["y"], "state": None if s["dst"] is None else s["state"]}


def _plain_verify(s):
    c = s["case"]
    b, n = c["b"], c["n"]
    t, v = s["logits"].shape
    row, there = _padded(s)
    req = torch.searchsorted(s["seq_ptr"][1:].contiguous(), torch.arange(t, device=DEV).int(), right=True)
    temp = s["temperature"].double()[req][:, None]
    # probabilities of every row, and the token that its random number takes
    z = s["logits"].double()
    best = z.amax(1, keepdim=True)
    greedy = (z == best).int().argmax(1)
    p = torch.where(temp > 0, torch.exp((z - best) / torch.where(temp > 0, temp, 1.0)),
                    torch.zeros_like(z).scatter_(1, greedy[:, None], 1.0))
    p /= p.sum(1, keepdim=True)

    def sample(p, u):
        cum = p.cumsum(1)
        return (cum <= u.double()[:, None] * cum[:, -1:]).sum(1).clamp(max=v - 1)

    tok = s["tokens"].long()[row]                                                         # [b, n]
    place = torch.arange(n, device=DEV)
    if s["tree_mask"] is not None:
        m = (s["tree_mask"][:, 0][row][..., None] >> place) & 1
        before = torch.where(m.bool() & (place[None, :] < place[:, None]), place, -1).amax(2)
    else:
        before = (place - 1).expand(b, n)
    prev = row.gather(1, before.clamp(min=0))                                             # the parent's row
    if s["q"] is None:
        drawn = sample(p, s["u"])
        good = drawn[prev] == tok
    else:
        good = s["accept_u"].double()[row] * s["q"].double()[row, tok] < p[prev, tok]
    good &= there & (before >= 0)
    path = torch.full((b, n), -1, dtype=torch.int64, device=DEV)
    cur = torch.zeros(b, dtype=torch.int64, device=DEV)
    count = torch.zeros_like(cur)
    live = there[:, 0]
    last = cur
    for i in range(n):
        path[:, i] = torch.where(live, row.gather(1, cur[:, None])[:, 0], -1)
        count += live
        last = torch.where(live, cur, last)
        child = good & (before == cur[:, None])
        cur = child.int().argmax(1)
        live = live & child.any(1)
    end = row.gather(1, last[:, None])[:, 0]
    if s["q"] is None:
        nxt = drawn[end]
    else:
        # a chain that was cut off goes on with what the target has over the draft
        cut = count < there.sum(1)
        after = row.gather(1, (last + 1).clamp(max=n - 1)[:, None])[:, 0]
        rest = torch.where(cut[:, None], (p[end] - s["q"].double()[after]).clamp(min=0), p[end])
        rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, p[end])
        nxt = sample(rest, s["u"][end])
    s["path"].fill_(-1)
    out = s["seq_ptr"][:-1].long()[:, None] + place
    keep = there & (path >= 0)
    s["path"][out[keep]] = path[keep].int()
    s["count"].copy_(count)
    s["next"].copy_(nxt)
    return {"path": s["path"], "count": s["count"], "next": s["next"]}


_run_own = {"delta": _own_delta, "conv": _own_conv, "verify": _own_verify}
_run_plain = {"delta": _plain_delta, "conv": _plain_conv, "verify": _plain_verify}


# --------------------------------------------------------------------------------------------- exact

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"delta": _exact_delta, "conv": _exact_conv, "verify": _exact_verify}[case["op"]](s)


def _order(s):
    """The rows of every sequence in its order, and the place of each row's parent (-1: the state)."""
    ptr = s["seq_ptr"].tolist()
    rows, parents = [], []
    for b, n in enumerate(s["lengths"]):
        if s["case"]["form"] == "accept":
            mine = s["rows"].tolist()[ptr[b]:ptr[b] + s["taken"][b]]
        else:
            mine = list(range(ptr[b], ptr[b] + n))
        rows.append(mine)
        parents.append(s["parents"][b] if s["parents"] is not None else list(range(-1, len(mine) - 1)))
    return rows, parents


def _exact_delta(s):
    """The recurrence itself, token by token; sequences that still have a token go on together."""
    c = s["case"]
    hk, hv, dk, dv, b = c["hk"], c["hv"], c["dk"], c["dv"], c["b"]
    rows, parents = _order(s)
    tree = c["form"] == "tree"
    most = max(len(x) for x in rows)
    now = s["state"][s["src"].long()].double()                                            # [b, hv, dv, dk]
    kept = [now] if tree else None
    out = None if s["out"] is None else torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for i in range(most):
        act = [j for j in range(b) if len(rows[j]) > i]
        r = _ints([rows[j][i] for j in act], torch.int64)
        k = s["k"][r].double().view(-1, hk, dk)
        q = s["q"][r].double().view(-1, hk, dk)
        if c["l2"]:
            k = k / torch.sqrt(torch.linalg.vector_norm(k, dim=2, keepdim=True) ** 2 + 1e-6)
            q = q / torch.sqrt(torch.linalg.vector_norm(q, dim=2, keepdim=True) ** 2 + 1e-6)
        k, q = (x.repeat_interleave(hv // hk, 1) for x in (k, q))
        whole = len(act) == b
        idx = _ints(act, torch.int64)
        if tree:
            old = torch.stack([kept[parents[j][i] + 1][j] for j in act])
        else:
            old = now if whole else now[idx]
        st = old * torch.exp(s["g"][r].double())[..., None, None]
        d = s["beta"][r].double()[..., None] * (s["v"][r].double().view(-1, hv, dv) - torch.einsum("bhvk,bhk->bhv", st, k))
        st = st + d[..., None] * k[:, :, None]
        if out is not None:
            out[r] = (torch.einsum("bhvk,bhk->bhv", st, q) * dk ** -0.5).flatten(1)
        if tree:
            node = torch.zeros_like(now)
            node[idx] = st
            kept.append(node)
        elif whole:
            now = st
        else:
            now[idx] = st
    pool = None
    if s["dst"] is not None:
        pool = s["state"].double()
        pool[s["dst"].long()] = now
    return {"out": out, "state": pool}


def _exact_conv(s):
    c = s["case"]
    w = c["w"]
    rows, parents = _order(s)
    wt = s["weight"].double()
    bias = 0.0 if s["bias"] is None else s["bias"].double()
    y = None if s["y"] is None else torch.empty(s["y"].shape, dtype=torch.float64, device=DEV)
    pool = None if s["dst"] is None else s["state"].double()
    src, dst = s["places"]
    for b, mine in enumerate(rows):
        line = torch.cat((s["state"][src[b]].double(), s["x"][_ints(mine, torch.int64)].double()))
        if y is not None:
            total = torch.zeros(len(mine), c["c"], dtype=torch.float64, device=DEV) + bias
            at = list(range(len(mine)))
            for back in range(w):
                total += wt[:, w - 1 - back] * line[_ints([w - 1 + i for i in at], torch.int64)]
                at = [parents[b][i] if i >= 0 else i - 1 for i in at]
            y[_ints(mine, torch.int64)] = total / (1.0 + torch.exp(-total))
        if pool is not None:
            pool[dst[b]] = line[len(mine):]
    return {"y": y, "state": pool}


def _exact_verify(s):
    c = s["case"]
    v = c["v"]
    ptr = s["seq_ptr"].tolist()
    tokens, u = s["tokens"].tolist(), s["u"].tolist()
    path = torch.full((ptr[-1],), -1, dtype=torch.int32)
    count, nxt = [], []

    def law(row, temp):
        z = s["logits"][row].double()
        if temp == 0:
            p = torch.zeros(v, dtype=torch.float64, device=DEV)
            p[int((z == z.max()).nonzero()[0])] = 1.0
            return p
        return torch.softmax(z / temp, 0)

    def take(weights, x):
        edges = torch.cumsum(weights, 0)
        return min(int(torch.searchsorted(edges, x * edges[-1:], right=True)[0]), v - 1)

    for b, n in enumerate(s["lengths"]):
        temp = float(s["temperature"][b])
        node, found, rest = 0, [0], None
        while True:
            row = ptr[b] + node
            p = law(row, temp)
            children = [i for i in range(1, n) if s["parent_rows"][b][i] == node]
            token = None
            if s["q"] is None:
                token = take(p, u[row])
                children = [i for i in children if tokens[ptr[b] + i] == token]
            elif children:
                i = children[0]
                drafted = s["q"][ptr[b] + i].double()
                x = tokens[ptr[b] + i]
                if not float(s["accept_u"][ptr[b] + i]) * float(drafted[x]) < float(p[x]):
                    rest = torch.clamp(p - drafted, min=0)
                    token = take(rest if float(rest.sum()) > 0 else p, u[row])
                    children = []
            if not children:
                nxt.append(take(p, u[row]) if token is None else token)
                break
            node = children[0]
            found.append(node)
        count.append(len(found))
        path[ptr[b]:ptr[b] + len(found)] = torch.tensor([ptr[b] + i for i in found], dtype=torch.int32)
    return {"path": path.to(DEV), "count": _ints(count), "next": _ints(nxt)}
