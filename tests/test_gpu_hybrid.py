"""GPU tests of the gated delta rule, the short convolution and the verification of drafted tokens against plain
implementations in 64 bits on the CPU (hybrid_util, which says how far results may be off)."""
import random

import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from hybrid_util import B8, E24, conv_ref, delta_bounds, delta_steps, mask_of, tree, verify_ref
from test_gpu_operators import BF, F32, NAN, assert_close, out_buf, pitched, rnd

pytestmark = pytest.mark.gpu


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def uni(seed, *shape):
    return torch.rand(*shape, generator=torch.Generator().manual_seed(seed))


def starts(lengths, before=0):
    at = [before]
    for n in lengths:
        at.append(at[-1] + n)
    return at


# --------------------------------------------------------------------------------------------- delta

class Delta:
    """Inputs of a call on the CPU, in the kernel's types."""

    def __init__(self, t, slots, hk, hv, dk, dv, seed=0, l2=True):
        x = torch.nn.functional.silu(rnd(seed, t, 2 * hk * dk + hv * dv))
        if not l2:
            x[:, :2 * hk * dk] *= dk ** -0.5
        self.q, self.k, self.v = x.to(BF).split((hk * dk, hk * dk, hv * dv), 1)
        rate = torch.exp(torch.linspace(-7, 0.7, hv))
        self.g = -rate * torch.nn.functional.softplus(rnd(seed + 1, t, hv) + 0.5)
        self.beta = torch.sigmoid(2 * rnd(seed + 2, t, hv))
        self.state = rnd(seed + 3, slots, hv, dv, dk, scale=0.5)
        self.hk, self.hv, self.dk, self.dv, self.l2, self.scale, self.eps = hk, hv, dk, dv, l2, dk ** -0.5, 1e-6

    def head(self, h, rows, src):
        """One head's tokens and first state, in 64 bits."""
        i, dk, dv = h // (self.hv // self.hk), self.dk, self.dv
        r = torch.tensor(rows, dtype=torch.int64)
        s0 = self.state[src, h].double().t() if src is not None else torch.zeros(dk, dv, dtype=torch.float64)
        return (self.q[r, i * dk:(i + 1) * dk].double(), self.k[r, i * dk:(i + 1) * dk].double(),
                self.v[r, h * dv:(h + 1) * dv].double(), self.g[r, h].double(), self.beta[r, h].double(), s0,
                self.scale, self.l2, self.eps)

    def check(self, out, state, seqs, heads=None):
        """seqs: (rows in order, src or None, dst or None, parents or None) of every sequence."""
        new = self.state.clone() if state is not None else None
        for rows, src, dst, parents in seqs:
            for h in heads or range(self.hv):
                args = self.head(h, rows, src)
                o, s = delta_steps(*args, parents=parents)
                do, ds = delta_bounds(*args, parents=parents)
                if out is not None and rows:
                    assert_close(out[torch.tensor(rows), h * self.dv:(h + 1) * self.dv], o, do, f"out, head {h}")
                if state is not None and dst is not None:
                    tol = ds[:, None].expand(-1, self.dk) if rows else torch.zeros(self.dv, self.dk, dtype=torch.float64)
                    assert_close(state[dst, h], s.t().contiguous(), tol, f"state, head {h}")
                    new[dst, h] = state[dst, h].cpu()
        if state is not None:
            assert torch.equal(state.cpu(), new), "a state that no sequence names was changed"

    def on_gpu(self, gap=8):
        """The matrices with NaN between their rows, the state with NaN between its slots."""
        mats = [pitched(x.contiguous(), (x.shape[1] + 7) // 8 * 8 + gap)[0] for x in (self.q, self.k, self.v, self.g, self.beta)]
        slots = self.state.shape[0]
        each = self.state[0].numel()
        buf = torch.full((slots, each + 64), NAN)
        buf[:, :each] = self.state.view(slots, each)
        buf = buf.cuda()
        return mats, buf[:, :each].view(slots, *self.state.shape[1:])


SHAPES = [(1, 1, 64, 64), (2, 4, 128, 128), (1, 3, 64, 256), (4, 4, 128, 64), (1, 2, 128, 256)]


@pytest.mark.parametrize("hk,hv,dk,dv", SHAPES)
@pytest.mark.parametrize("lengths", [[1], [1, 1, 1, 1, 1], [2, 0, 5], [63], [64], [65], [130, 1, 0, 67], [300]])
@pytest.mark.parametrize("l2", [True, False])
def test_delta_sequences(hk, hv, dk, dv, lengths, l2):
    t, b = sum(lengths), len(lengths)
    ptr = starts(lengths, 3)
    d = Delta(t + 5, 2 * b + 2, hk, hv, dk, dv, seed=10, l2=l2)
    (q, k, v, g, beta), state = d.on_gpu()
    out, ok = out_buf(t + 5, hv * dv, hv * dv + 8, BF)
    order = torch.randperm(2 * b + 2, generator=torch.Generator().manual_seed(b)).tolist()
    src, dst = order[:b], order[b:2 * b]
    src[-1] = -1 if b > 1 else src[-1]
    got = w12.gated_delta(q, k, v, g, beta, state, ints(ptr), ints(src), dst=ints(dst), l2norm=l2, out=out)
    torch.cuda.synchronize()
    assert got is out and ok()
    seqs = [(list(range(ptr[i], ptr[i + 1])), src[i] if src[i] >= 0 else None, dst[i], None) for i in range(b)]
    d.check(out, state, seqs)
    rest = torch.ones(t + 5, dtype=torch.bool)
    rest[ptr[0]:ptr[-1]] = False
    assert (out.cpu()[rest].view(torch.int16) == 0x55).all(), "rows of no sequence"


@pytest.mark.parametrize("lengths", [[1, 1, 1], [7, 3], [200, 5]])
def test_delta_in_place_is_the_same(lengths):
    t, b = sum(lengths), len(lengths)
    d = Delta(t, 2 * b, 2, 4, 128, 128, seed=20)
    (q, k, v, g, beta), state = d.on_gpu()
    ptr = ints(starts(lengths))
    a = w12.gated_delta(q, k, v, g, beta, state, ptr, ints(list(range(b))), dst=ints(list(range(b, 2 * b))))
    apart = state[b:].clone()
    _, state = d.on_gpu()
    o = w12.gated_delta(q, k, v, g, beta, state, ptr, ints(list(range(b))), dst=ints(list(range(b))))
    assert torch.equal(a, o) and torch.equal(state[:b], apart)
    # and in two steps: the first of each sequence's tokens, then the others, from the states that they left
    _, state = d.on_gpu()
    firsts = [n // 2 for n in lengths]
    at = starts(lengths)
    rows1 = [at[i] + j for i in range(b) for j in range(firsts[i])]
    rows2 = [at[i] + j for i in range(b) for j in range(firsts[i], lengths[i])]
    same = ints(list(range(b)))
    pad = lambda r: ints(r + [-1] * (t - len(r)))
    out = torch.empty(t, 4 * 128, dtype=BF, device="cuda")
    w12.gated_delta(q, k, v, g, beta, state, ints(starts(firsts)), same, dst=same, rows=pad(rows1), out=out)
    w12.gated_delta(q, k, v, g, beta, state, ints(starts([n - f for n, f in zip(lengths, firsts)])), same, dst=same,
                    rows=pad(rows2), out=out)
    whole = d.on_gpu()[1]
    whole[:b] = state[:b]
    d.check(out, whole, [(list(range(at[i], at[i + 1])), i, i, None) for i in range(b)])


@pytest.mark.parametrize("n", [5, 70, 200])
def test_delta_rows_and_lens(n):
    """An accepted path: rows out of order, one that is none, a length that cuts; states alone and with outputs."""
    d = Delta(n + 9, 4, 2, 6, 128, 128, seed=30)
    (q, k, v, g, beta), state = d.on_gpu()
    r = random.Random(n)
    rows = r.sample(range(n + 9), n)
    bad = list(rows)
    bad[2], bad[3] = -1, n + 9
    lens = n - 1
    given = ints([0] * 4 + bad + [0] * 5)
    args = dict(dst=ints([2, 1]), lens=ints([lens, 0]), rows=given)
    w12.gated_delta(None, k, v, g, beta, state, ints([4, 4 + n, 4 + n + 5]), ints([0, 3]), outputs=False, **args)
    used = [x for i, x in enumerate(rows[:lens]) if i not in (2, 3)]
    seqs = [(used, 0, 2, None), ([], 3, 1, None)]
    d.check(None, state, seqs)
    again = d.on_gpu()[1]
    out, ok = out_buf(n + 9, 6 * 128, 6 * 128, BF)
    w12.gated_delta(q, k, v, g, beta, again, ints([4, 4 + n, 4 + n + 5]), ints([0, 3]), out=out, **args)
    assert torch.equal(again, state) and ok()
    d.check(out, again, seqs)
    untouched = [x for x in range(n + 9) if x not in used]
    assert (out.cpu()[untouched].view(torch.int16) == 0x55).all()


@pytest.mark.parametrize("hk,hv,dk,dv", SHAPES)
@pytest.mark.parametrize("nodes", [[1], [2], [16, 17, 1, 0, 31], [33], [48], [63], [64], [5] * 20])
def test_delta_trees(hk, hv, dk, dv, nodes):
    t, b = sum(nodes), len(nodes)
    r = random.Random(t)
    parents = [tree(r, n, roots=1 + i % 2) for i, n in enumerate(nodes)]
    d = Delta(t + 1, b + 1, hk, hv, dk, dv, seed=40)
    (q, k, v, g, beta), state = d.on_gpu()
    before = state.clone()
    mask = torch.cat([mask_of(p, 2) for p in parents if p] + [torch.zeros(1, 2, dtype=torch.int64)])
    ptr = starts(nodes)
    src = list(range(b, 0, -1))
    src[0] = src[-1]                    # two requests share a state
    out, ok = out_buf(t + 1, hv * dv, hv * dv, BF)
    w12.gated_delta(q, k, v, g, beta, state, ints(ptr), ints(src), tree_mask=mask.cuda(), out=out)
    assert ok() and torch.equal(state, before)
    d.check(out, None, [(list(range(ptr[i], ptr[i + 1])), src[i], None, parents[i]) for i in range(b)])
    assert (out.cpu()[t:].view(torch.int16) == 0x55).all()


def test_delta_tree_of_a_chain_and_a_range_too_long():
    d = Delta(100, 2, 2, 4, 128, 128, seed=50)
    (q, k, v, g, beta), state = d.on_gpu()
    chain = list(range(-1, 99))
    out, ok = out_buf(100, 512, 512, BF)
    w12.gated_delta(q, k, v, g, beta, state, ints([0, 100]), ints([1]), tree_mask=mask_of(chain, 2).cuda(), out=out)
    assert ok()
    d.check(out, None, [(list(range(64)), 1, None, None)])
    assert (out.cpu()[64:].view(torch.int16) == 0x55).all(), "nodes past the 64th"
    # the chain as a sequence whose state stays
    before = state.clone()
    o = w12.gated_delta(q, k, v, g, beta, state, ints([0, 100]), ints([1]))
    assert torch.equal(state, before)
    d.check(o, None, [(list(range(100)), 1, None, None)])


@pytest.mark.parametrize("n,form", [(9, "seq"), (150, "seq"), (40, "tree"), (12, "tree")])
def test_delta_strong_decays(n, form):
    """Log decays from 0 to -inf, strengths of 0, 1 and 2 and equal keys: states that are cleared, kept and turned over."""
    d = Delta(n, 2, 1, 4, 128, 64, seed=60)
    r = random.Random(1)
    for i in range(n):
        d.g[i] = torch.tensor([r.choice((0.0, -1e-6, -3.0, -30.0, -120.0, -1e6, float("-inf"))) for _ in range(4)])
        d.beta[i] = torch.tensor([r.choice((0.0, 1.0, 1.0, 2.0)) for _ in range(4)])
    d.k = d.k.clone()
    d.k[n // 2:] = d.k[n // 2 - 1]
    (q, k, v, g, beta), state = d.on_gpu()
    if form == "tree":
        parents = tree(r, n)
        out = w12.gated_delta(q, k, v, g, beta, state, ints([0, n]), ints([0]), tree_mask=mask_of(parents).cuda())
        seqs, state = [(list(range(n)), 0, None, parents)], None
    else:
        out = w12.gated_delta(q, k, v, g, beta, state, ints([0, n]), ints([0]), dst=ints([1]))
        seqs = [(list(range(n)), 0, 1, None)]
    # -1e4 clears as -inf does
    d.g = d.g.clamp(min=-1e4)
    d.check(out, state, seqs)


@pytest.mark.parametrize("what", ["k", "v", "q", "g", "beta"])
@pytest.mark.parametrize("value", [NAN, float("inf")])
def test_delta_bad_values_stay_on_their_path(what, value):
    """A NaN or infinity reaches its own row and what comes after it, and neither other branches, earlier tokens nor other
    heads and sequences."""
    lengths = [150, 30]
    d = Delta(180, 4, 2, 4, 128, 128, seed=70)
    (q, k, v, g, beta), state = d.on_gpu()
    args = dict(q=q, k=k, v=v, g=g, beta=beta)
    ptr, src = ints([0, 150, 180]), ints([0, 1])
    clean_state = state.clone()
    clean = w12.gated_delta(*args.values(), clean_state, ptr, src, dst=ints([2, 3]))
    at = 70
    args[what][at, 0] = value
    dirty = w12.gated_delta(*args.values(), state, ptr, src, dst=ints([2, 3]))
    assert torch.equal(dirty[:at], clean[:at]) and torch.equal(dirty[150:], clean[150:])
    assert torch.equal(state[3], clean_state[3])
    other = slice(2 * 128, None) if what in "qk" else slice(128, None)
    assert torch.equal(dirty[:, other], clean[:, other]), "heads that do not use the value"
    assert not dirty[at, :128].isfinite().all()
    args[what][at, 0] = 0.5
    # trees: an inner node is bad, its descendants may be
    nodes = 40
    parents = tree(random.Random(3), nodes)
    mask = mask_of(parents).cuda()
    below = [sum(int(m) >> i & 1 for m in mask[:, 0].tolist()) - 1 for i in range(nodes)]
    node = next(i for i in range(1, nodes) if 3 <= below[i] < nodes // 2)
    tp = ints([100, 100 + nodes])
    cut = {n: x[:100 + nodes] for n, x in args.items()}
    full = torch.zeros(100 + nodes, 1, dtype=torch.int64, device="cuda")
    full[100:] = mask
    clean = w12.gated_delta(*cut.values(), state[:2], tp, ints([1]), tree_mask=full)[100:]
    cut[what][100 + node, 0] = value
    dirty = w12.gated_delta(*cut.values(), state[:2], tp, ints([1]), tree_mask=full)[100:]
    hit = torch.tensor([bool(int(m) >> node & 1) for m in mask[:, 0].tolist()])
    assert hit.sum() > 1 and torch.equal(dirty[~hit], clean[~hit])
    assert not dirty[node, :128].isfinite().all()


def test_delta_offsets_past_32_bits():
    """Slots 2^31 elements apart."""
    d = Delta(70, 2, 1, 1, 64, 64, seed=80)
    (q, k, v, g, beta), _ = d.on_gpu()
    buf = torch.empty((1 << 31) + 64 * 64 + 64, device="cuda")
    state = torch.as_strided(buf, (2, 1, 64, 64), ((1 << 31) + 64, 64 * 64, 64, 1))
    state.copy_(d.state)
    out = w12.gated_delta(q, k, v, g, beta, state, ints([0, 1, 70]), ints([1, 0]), dst=ints([1, 0]))
    d.check(out, state, [([0], 1, 1, None), (list(range(1, 70)), 0, 0, None)])


def test_delta_decreasing_ranges_write_nothing_else():
    t = 300
    d = Delta(t, 40, 2, 4, 64, 64, seed=90)
    (q, k, v, g, beta), state = d.on_gpu()
    out, ok = out_buf(t, 256, 264, BF)
    ptr = [(0, t)[i % 2] for i in range(21)]
    need = w12.gated_delta_workspace_size(t, 20, 4, 64, 64)
    ws = torch.full((need + 256,), 7, dtype=torch.uint8, device="cuda")
    before = state.clone()
    w12.gated_delta(q, k, v, g, beta, state, ints(ptr), ints(list(range(20))), dst=ints(list(range(20, 40))), out=out, ws=ws[:need])
    assert ok() and (ws[need:] == 7).all() and torch.equal(state[:20], before[:20])
    w12.gated_delta(q, k, v, g, beta, state, ints([-5, 2 * t, -9]), ints([0, 1]), dst=ints([20, 21]), out=out, ws=ws[:need])
    assert ok() and (ws[need:] == 7).all()
    d.check(out, None, [(list(range(t)), 0, None, None)])


# ---------------------------------------------------------------------------------------------- conv

def conv_tol(y, mag, pre, w):
    """Sums of w + 1 products and the sigmoid: exp to 2^-22 (1 + |x|) of itself, a sum and a quotient."""
    return B8 * y.abs() + 1.2 * (w + 3) * E24 * mag + y.abs() * (pre.abs() + 4) * 2.0 ** -21


@pytest.mark.parametrize("src", [F32, BF])
@pytest.mark.parametrize("w", [2, 3, 4])
@pytest.mark.parametrize("c,lengths", [(1, [1]), (8, [1, 1, 2]), (100, [0, 3, 40]), (515, [16, 17, 1]), (1032, [33]), (64, [70, 2, 5])])
def test_conv_sequences(src, w, c, lengths):
    t, b = sum(lengths), len(lengths)
    ptr = starts(lengths, 2)
    ld = (c + 7) // 8 * 8 + 8
    x, past = rnd(1, t + 3, c).to(src), rnd(2, 2 * b + 1, w - 1, c).to(src)
    weight, bias = rnd(3, c, w, scale=0.6).to(BF), (rnd(4, c).to(BF) if c % 3 else None)
    xd, _ = pitched(x, ld)
    buf = torch.full(((2 * b + 1) * (w - 1), ld), NAN, dtype=F32).to(src)
    buf[:, :c] = past.reshape(-1, c)
    state = buf.cuda().view(2 * b + 1, w - 1, ld)[:, :, :c]
    y, ok = out_buf(t + 3, c, ld, BF)
    src_of = [i if i else -3 for i in range(b)] if b > 1 else [0]
    dst_of = [b + i for i in range(b)]
    silu = c != 8
    got = w12.short_conv(xd, weight.cuda(), state, ints(ptr), ints(src_of), dst=ints(dst_of),
                         bias=None if bias is None else bias.cuda(), silu=silu, y=y)
    assert got is y and ok()
    want = past.clone()
    for i in range(b):
        old = past[src_of[i]].double() if src_of[i] >= 0 else torch.zeros(w - 1, c, dtype=torch.float64)
        rows = slice(ptr[i], ptr[i + 1])
        args = (x[rows].double(), weight.double(), None if bias is None else bias.double(), old)
        ref, mag, new = conv_ref(*args, silu)
        pre = conv_ref(*args, False)[0]
        assert_close(y[rows], ref, conv_tol(ref, mag, pre, w) + 1e-38, "y")
        want[dst_of[i]] = new.to(src)
    assert torch.equal(state.cpu(), want)
    rest = torch.ones(t + 3, dtype=torch.bool)
    rest[ptr[0]:ptr[-1]] = False
    assert (y.cpu()[rest].view(torch.int16) == 0x55).all()
    # in place, in two calls, and without outputs: the same states
    inplace = torch.zeros(b, w - 1, ld, dtype=src, device="cuda")[:, :, :c]
    for i in range(b):
        inplace[i] = past[src_of[i]] if src_of[i] >= 0 else 0
    same = ints(list(range(b)))
    half = [n // 2 for n in lengths]
    rows1 = [ptr[i] + j for i in range(b) for j in range(half[i])]
    rows2 = [ptr[i] + j for i in range(b) for j in range(half[i], lengths[i])]
    pad = lambda r: ints(r + [-1] * (t + 3 - len(r)))
    y2 = out_buf(t + 3, c, ld, BF)[0]
    w12.short_conv(xd, weight.cuda(), inplace, ints(starts(half)), same, dst=same, rows=pad(rows1), y=y2, silu=silu,
                   bias=None if bias is None else bias.cuda())
    w12.short_conv(xd, weight.cuda(), inplace, ints(starts([n - h for n, h in zip(lengths, half)])), same, dst=same, rows=pad(rows2),
                   y=y2, silu=silu, bias=None if bias is None else bias.cuda())
    assert torch.equal(inplace.cpu(), want[b:2 * b]) and torch.equal(y2[ptr[0]:ptr[-1]], y[ptr[0]:ptr[-1]])


@pytest.mark.parametrize("src", [F32, BF])
@pytest.mark.parametrize("w", [2, 4])
@pytest.mark.parametrize("c,nodes", [(40, [1, 0, 9]), (520, [63]), (16, [64, 5]), (7, [70])])
def test_conv_trees(src, w, c, nodes):
    t, b = sum(nodes), len(nodes)
    r = random.Random(t)
    parents = [tree(r, n, roots=1 + i % 2, reach=5) for i, n in enumerate(nodes)]
    ld = (c + 7) // 8 * 8
    x, past = rnd(1, t, c).to(src), rnd(2, b, w - 1, c).to(src)
    x[3 % t] = NAN
    weight = rnd(3, c, w).to(BF)
    state = torch.zeros(b, w - 1, ld, dtype=src)
    state[:, :, :c] = past
    state = state.cuda()[:, :, :c]
    y, ok = out_buf(t, c, ld, BF)
    mask = torch.cat([mask_of(p, 2) for p in parents if p])
    ptr = starts(nodes)
    w12.short_conv(pitched(x, ld)[0], weight.cuda(), state, ints(ptr), ints(list(range(b))), tree_mask=mask.cuda(), y=y)
    assert ok() and torch.equal(state.cpu(), past)
    for i in range(b):
        n = min(nodes[i], 64)
        args = (x[ptr[i]:ptr[i] + n].double(), weight.double(), None, past[i].double())
        ref, mag, _ = conv_ref(*args, True, parents[i][:n])
        pre = conv_ref(*args, False, parents[i][:n])[0]
        tol = conv_tol(ref, mag, pre, w) + 1e-38
        assert_close(y[ptr[i]:ptr[i] + n], ref, tol.nan_to_num(0.0), "y")
    if max(nodes) > 64:
        assert (y.cpu()[64:].view(torch.int16) == 0x55).all()


# -------------------------------------------------------------------------------------------- verify

def verify_case(seed, nodes, v, form, temps, with_q=False, dtype=F32, match=0.7):
    r = random.Random(seed)
    t, b = sum(nodes), len(nodes)
    parents = [tree(r, n) if form == "tree" else list(range(-1, n - 1)) for n in nodes]
    ptr = starts(nodes)
    z = rnd(seed, t, v, scale=2.0)
    top = torch.randint(0, v, (t, 3), generator=torch.Generator().manual_seed(seed))
    for j in range(3):
        z[torch.arange(t), top[:, j]] = 12.0 - j
    z = z.to(dtype)
    up = [ptr[i] + max(p, 0) for i, ps in enumerate(parents) for p in ps]
    q = accept = None
    if with_q:
        q = torch.softmax(z.float()[up] + rnd(seed + 1, t, v, scale=0.5), 1)
        tokens = torch.multinomial(q, 1, generator=torch.Generator().manual_seed(seed))[:, 0].int() if t else torch.zeros(0).int()
        accept = uni(seed + 2, t)
    else:
        tokens = torch.tensor([int(top[up[i], r.randrange(3)]) if r.random() < match else r.randrange(v) for i in range(t)],
                              dtype=torch.int32)
    temp = {"one": torch.ones(b), "greedy": torch.zeros(b),
            "mixed": torch.tensor([r.choice((0.0, 0.3, 1.0, 1.7)) for _ in range(b)])}[temps]
    return dict(logits=z, tokens=tokens, u=uni(seed + 3, t), parents=parents, ptr=ptr, q=q, accept_u=accept, temp=temp)


def verify_check(c, words=1, ws=None, stream=None):
    t, v = c["logits"].shape
    b = len(c["parents"])
    ld = (v + 7) // 8 * 8 + 8
    mask = None
    if any(p != list(range(-1, len(p) - 1)) for p in c["parents"]):
        mask = torch.cat([mask_of(p, words) for p in c["parents"] if p]).cuda()
    path = torch.full((t,), 99, dtype=torch.int32, device="cuda")
    got = w12.verify_draft(pitched(c["logits"], ld)[0], c["tokens"].cuda(), c["u"].cuda(), ints(c["ptr"]), tree_mask=mask,
                           q=None if c["q"] is None else pitched(c["q"], ld)[0],
                           accept_u=None if c["accept_u"] is None else c["accept_u"].cuda(), temperature=c["temp"].cuda(),
                           path=path, ws=ws)
    assert got[0] is path
    path, count, nxt = (x.cpu().tolist() for x in got)
    want_path, want_count, want_next = [99] * t, [], []
    for i, p in enumerate(c["parents"]):
        a, e = c["ptr"][i], c["ptr"][i] + len(p)
        if not p:
            want_count.append(0)
            want_next.append(-1)
            continue
        part = lambda x: None if x is None else x[a:e]
        found, token = verify_ref(c["logits"][a:e], c["tokens"][a:e], c["u"][a:e], p, float(c["temp"][i]), part(c["q"]),
                                  part(c["accept_u"]))
        want_path[a:e] = [a + j for j in found] + [-1] * (len(p) - len(found))
        want_count.append(len(found))
        want_next.append(token)
    assert (count, nxt, path) == (want_count, want_next, want_path)
    return count


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("form,with_q", [("tree", False), ("chain", False), ("chain", True)])
@pytest.mark.parametrize("nodes,v,temps", [
    ([1], 1, "one"), ([1], 50257, "one"), ([17], 1000, "one"), ([63], 8191, "one"), ([64, 2, 0, 30], 8193, "mixed"),
    ([24] * 16, 5000, "mixed"), ([5, 5, 5], 131072, "greedy"), ([3, 1], 20001, "mixed"), ([200, 100], 300, "one"),
])
def test_verify(dtype, form, with_q, nodes, v, temps):
    for seed in range(3):
        c = verify_case(seed, nodes, v, form, temps, with_q, dtype)
        verify_check(c, words=-(-max(nodes) // 64))


def test_verify_walks_far():
    """Everything that is drafted is what the target says: the whole chain is accepted; and a tree that one path leads through."""
    c = verify_case(5, [40, 9], 3001, "chain", "greedy")
    for i, p in enumerate(c["parents"]):
        for j in range(1, len(p)):
            c["tokens"][c["ptr"][i] + j] = int(c["logits"][c["ptr"][i] + j - 1].argmax())
    assert verify_check(c) == [40, 9]
    c = verify_case(6, [60], 3001, "tree", "greedy")
    for j in range(1, 60):
        c["tokens"][j] = int(c["logits"][c["parents"][0][j]].argmax())       # siblings alike: the first of them counts
    firsts, at = 1, 0
    while at in c["parents"][0]:
        at = c["parents"][0].index(at)
        firsts += 1
    assert verify_check(c) == [firsts]


def test_verify_borders_ties_and_odd_numbers():
    v = 10000
    z = torch.full((12, v), -float("inf"))
    z[0] = 0.0                                       # uniform: u counts the tokens off
    z[1, 5], z[1, 9999] = 2.0, 2.0
    z[2] = NAN
    z[2, 77] = -1e30
    z[3, [8, 3]] = float("inf")
    # row 4 has nothing
    z[5, 9000:] = -3e38
    z[6] = torch.finfo(F32).min
    z[7] = 0.0
    z[8] = 0.0
    z[9, ::2] = 1.0
    z[10] = 88.0
    z[11] = -1e4
    u = torch.tensor([0.5, 0.5, 0.9, 0.3, 0.5, 0.99999994, 0.0, 1.0, NAN, 0.25, -3.0, float("inf")])
    got = w12.verify_draft(z.cuda(), torch.zeros(12, dtype=torch.int32, device="cuda"), u.cuda(), ints(list(range(13))))
    want = [verify_ref(z[i:i + 1], torch.zeros(1), u[i:i + 1], [-1], 1.0)[1] for i in range(12)]
    assert got[2].cpu().tolist() == want and want[4] == -1 and want[3] == 3 and want[0] == 5000 and want[1] == 9999
    greedy = w12.verify_draft(z.cuda(), torch.zeros(12, dtype=torch.int32, device="cuda"), u.cuda(), ints(list(range(13))),
                              temperature=torch.tensor([0.0, -1.0, NAN] * 4, device="cuda"))[2].cpu().tolist()
    assert greedy == [0, 5, 77, 3, -1, 9000, 0, 0, 0, 0, 0, 0]


def test_verify_q_edges():
    """Draft probabilities equal to the target's, tokens that cannot be drawn, out of range, no weight left over."""
    v, n = 4000, 6
    z = rnd(1, n, v)
    z[2] = -float("inf")
    p = torch.softmax(z.double(), 1)
    for change in range(5):
        q = torch.zeros(n, v)
        q[1:] = p[:-1].float()
        tokens = torch.tensor([0] + [int(z[i].argmax()) for i in range(n - 1)], dtype=torch.int32)
        accept, u = torch.full((n,), 0.25), uni(3, n)
        if change == 1:
            tokens[1] = v
        if change == 2:
            tokens[2] = -7
        if change == 3:
            accept[1], q[1] = 0.9, 1.0                # nothing is left over q: taken from p
        if change == 4:
            q[1, tokens[1]] = 0.0
            q[2] = NAN
        verify_check(dict(logits=z, tokens=tokens, u=u, parents=[list(range(-1, n - 1))], ptr=[0, n], q=q, accept_u=accept,
                          temp=torch.ones(1)))


def test_verify_many_nodes():
    """Past 4096 nodes the rest of a request does not count; their path says -1."""
    n, v = 4100, 40
    c = verify_case(8, [n], v, "chain", "greedy")
    for j in range(1, n):
        c["tokens"][j] = int(c["logits"][j - 1].argmax())
    got = w12.verify_draft(c["logits"].cuda(), c["tokens"].cuda(), c["u"].cuda(), ints([0, n]), temperature=c["temp"].cuda())
    assert got[1].item() == 4096 and got[2].item() == int(c["logits"][4095].argmax())
    assert got[0].cpu().tolist() == list(range(4096)) + [-1] * 4
