"""GPU tests of how the hybrid target's operators are called: captured and replayed, on another stream, several at once, with a
workspace for more rows, and together as a layer's step of speculative decoding."""
import random

import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from hybrid_util import mask_of, tree, verify_ref
from test_gpu_hybrid import Delta, ints, rnd, starts, verify_case

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def replays(call, outputs, change, n=4):
    """Captures call, and checks that replays give what the call itself gives, bit for bit, for inputs that change between them."""
    call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(n):
        change(i)
        call()
        torch.cuda.synchronize()
        want = [o.clone() for o in outputs]
        for o in outputs:
            o.zero_()
        (torch.ones(1000, device="cuda") * i).sum().item()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o.view(torch.uint8) if o.dtype == BF else o, w.view(torch.uint8) if w.dtype == BF else w)
                   for o, w in zip(outputs, want)), f"replay {i}"


@pytest.mark.parametrize("lengths", [[1, 1, 1], [100, 3, 70]])
def test_delta_replays_follow_their_inputs(lengths):
    """Values, ranges and slots change between replays; the launches are those of the capture."""
    t, b = sum(lengths), len(lengths)
    d = Delta(t, 8, 2, 4, 128, 128, seed=1)
    (q, k, v, g, beta), state = d.on_gpu()
    first = state.clone()
    ptr, src, dst = ints(starts(lengths)), ints([0, 1, 2]), ints([4, 5, 6])
    out = torch.zeros(t, 512, dtype=BF, device="cuda")
    ws = w12.gated_delta_workspace(t, b, state)

    def change(i):
        src.copy_(ints([i % 4, 3 - i % 4, 2]))
        dst.copy_(ints([7 - i % 3, 4, 0 if i == 3 else 3]))
        v.mul_(-0.5)
        if i % 2:
            ptr.copy_(ints([0, t // 3, t // 3, t]))

    # the call reads the states as well: each time from the same ones, and a copy of them is what is compared
    seen = torch.zeros_like(state)

    def call():
        state.copy_(first)
        w12.gated_delta(q, k, v, g, beta, state, ptr, src, dst=dst, out=out, ws=ws)
        seen.copy_(state)

    replays(call, [out, seen], change)


def test_tree_and_conv_replays():
    nodes = 40
    r = random.Random(5)
    d = Delta(nodes, 3, 2, 4, 128, 128, seed=2)
    (q, k, v, g, beta), state = d.on_gpu()
    mask = mask_of(tree(r, nodes)).cuda()
    ptr, src = ints([0, nodes]), ints([1])
    out = torch.zeros(nodes, 512, dtype=BF, device="cuda")
    x, past = rnd(3, nodes, 264).cuda(), rnd(4, 3, 3, 264).cuda()
    weight = rnd(5, 264, 4).to(BF).cuda()
    y = torch.zeros(nodes, 264, dtype=BF, device="cuda")

    def call():
        w12.short_conv(x, weight, past, ptr, src, tree_mask=mask, y=y)
        w12.gated_delta(q, k, v, g, beta, state, ptr, src, tree_mask=mask, out=out, ws=ws)

    ws = w12.gated_delta_workspace(nodes, 1, state)

    def change(i):
        mask.copy_(mask_of(tree(r, nodes)))
        src.fill_(i % 3)
        x.mul_(1.1)

    replays(call, [out, y], change)


@pytest.mark.parametrize("with_q", [False, True])
def test_verify_replays(with_q):
    c = verify_case(11, [20, 7, 12], 5003, "chain" if with_q else "tree", "mixed", with_q)
    t = 39
    pad = lambda z: torch.nn.functional.pad(z, (0, 5008 - 5003)).cuda()[:, :5003]
    logits, tokens, u = pad(c["logits"]), c["tokens"].cuda(), c["u"].cuda()
    q, accept = (pad(c["q"]), c["accept_u"].cuda()) if with_q else (None, None)
    mask = None if with_q else torch.cat([mask_of(p) for p in c["parents"]]).cuda()
    temp = c["temp"].cuda()
    path, count, nxt = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (t, 3, 3))
    ws = w12.verify_draft_workspace(t, 3, 5003)
    ptr = ints(c["ptr"])

    def call():
        w12.verify_draft(logits, tokens, u, ptr, tree_mask=mask, q=q, accept_u=accept, temperature=temp, path=path, count=count,
                         next_token=nxt, ws=ws)

    def change(i):
        u.copy_(torch.rand(t, generator=torch.Generator().manual_seed(i)))
        temp.copy_(torch.tensor([1.0, 0.0, 0.7 + i]))
        logits.mul_(0.9)

    replays(call, [path, count, nxt], change)


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, give what they give alone."""
    made = []
    for seed, lengths in ((1, [150, 20]), (2, [64, 64, 64])):
        d = Delta(sum(lengths), 8, 2, 4, 128, 128, seed=seed)
        mats, state = d.on_gpu()
        b = len(lengths)
        c = verify_case(seed, [30, 9], 20011, "tree", "mixed")
        made.append(dict(mats=mats, state=state, ptr=ints(starts(lengths)), src=ints(list(range(b))), dst=ints(list(range(4, 4 + b))),
                         logits=torch.nn.functional.pad(c["logits"], (0, 5)).cuda()[:, :20011], tokens=c["tokens"].cuda(), u=c["u"].cuda(),
                         vptr=ints(c["ptr"]), mask=torch.cat([mask_of(p) for p in c["parents"]]).cuda(),
                         stream=torch.cuda.Stream(), rows=sum(lengths), b=b))

    def run(m, stream=None):
        out = w12.gated_delta(*m["mats"], m["state"], m["ptr"], m["src"], dst=m["dst"], stream=stream)
        return (out, *w12.verify_draft(m["logits"], m["tokens"], m["u"], m["vptr"], tree_mask=m["mask"], stream=stream))

    alone = [run(m) for m in made]
    states = [m["state"].clone() for m in made]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [run(m, m["stream"]) for m in made]
        torch.cuda.synchronize()
        for a, g in zip(alone, got):
            assert torch.equal(a[0].view(torch.int16), g[0].view(torch.int16))
            assert torch.equal(a[2], g[2]) and torch.equal(a[3], g[3])
            for i, n in enumerate(a[2].tolist()):
                at = made[0]["vptr"].tolist()[i]
                assert torch.equal(a[1][at:at + n], g[1][at:at + n])
        assert all(torch.equal(m["state"], s) for m, s in zip(made, states))


def test_a_larger_workspace_full_of_anything():
    d = Delta(200, 4, 2, 4, 64, 128, seed=3)
    mats, state = d.on_gpu()
    args = (*mats, state, ints([0, 150, 200]), ints([0, 1]))
    want = w12.gated_delta(*args, dst=ints([2, 3]))
    want_state = state.clone()
    ws = torch.full((w12.gated_delta_workspace_size(5000, 900, 4, 64, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    got = w12.gated_delta(*args, dst=ints([2, 3]), ws=ws)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and torch.equal(state, want_state)
    z, tok, u = rnd(1, 9, 4096).cuda(), torch.zeros(9, dtype=torch.int32, device="cuda"), torch.rand(9, device="cuda")
    want = w12.verify_draft(z, tok, u, ints([0, 9]))
    ws = torch.full((w12.verify_draft_workspace_size(3000, 100, 70000),), 0xFF, dtype=torch.uint8, device="cuda")
    got = w12.verify_draft(z, tok, u, ints([0, 9]), ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_results_repeat_bit_for_bit():
    d = Delta(300, 4, 4, 8, 128, 128, seed=4)
    mats, state = d.on_gpu()
    args = (*mats, state, ints([0, 250, 300]), ints([0, 1]))
    first = w12.gated_delta(*args, dst=ints([2, 3]))
    kept = state.clone()
    for _ in range(5):
        assert torch.equal(w12.gated_delta(*args, dst=ints([2, 3])).view(torch.int16), first.view(torch.int16))
        assert torch.equal(state, kept)


def test_a_step_of_speculative_decoding():
    """A tree's rows through convolution and recurrence, the verification of its tokens, and the accepted path's way into the states:
    afterwards the layer stands where it would stand had the accepted tokens come one by one."""
    r = random.Random(9)
    nodes = [14, 9, 1]
    t, b, hk, hv, dk, dv, v = sum(nodes), 3, 2, 4, 128, 128, 4001
    ptr = starts(nodes)
    parents = [tree(r, n) for n in nodes]
    mask = torch.cat([mask_of(p) for p in parents]).cuda()
    c = 2 * hk * dk + hv * dv
    x = rnd(1, t, c)
    weight = rnd(2, c, 4, scale=0.5).to(BF)
    past, state = rnd(3, b, 3, c), rnd(4, b, hv, dv, dk, scale=0.3)
    g, beta = -0.2 * torch.rand(t, hv), torch.rand(t, hv)
    logits, tokens, u = rnd(5, t, v), torch.zeros(t, dtype=torch.int32), torch.rand(t)
    logits[:, 17] += 20.0
    for i, p in enumerate(parents):
        for j in range(1, nodes[i]):
            tokens[ptr[i] + j] = 17 if r.random() < 0.6 else 5
    xd, wd, gd, bd = x.cuda(), weight.cuda(), g.cuda(), beta.cuda()
    pastd, stated, seq, same = past.cuda(), state.cuda(), ints(ptr), ints([0, 1, 2])

    def split(y):
        return y.split((hk * dk, hk * dk, hv * dv), 1)

    y = w12.short_conv(xd, wd, pastd, seq, same, tree_mask=mask)
    out = w12.gated_delta(*split(y), gd, bd, stated, seq, same, tree_mask=mask)
    path, count, nxt = w12.verify_draft(torch.nn.functional.pad(logits, (0, 7)).cuda()[:, :v], tokens.cuda(), u.cuda(), seq, tree_mask=mask)
    move = dict(dst=same, lens=count, rows=path)
    w12.gated_delta(None, *split(y)[1:], gd, bd, stated, seq, same, outputs=False, **move)
    w12.short_conv(xd, wd, pastd, seq, same, outputs=False, **move)
    assert torch.isfinite(out.float()).all()
    taken = []
    for i in range(b):
        a, e = ptr[i], ptr[i + 1]
        found, token = verify_ref(logits[a:e], tokens[a:e], u[a:e], parents[i], 1.0)
        assert count[i].item() == len(found) and nxt[i].item() == token
        taken.append([a + j for j in found])
    assert max(len(x) for x in taken) > 1
    # one by one, from the same states
    past1, state1 = past.cuda(), state.cuda()
    for i, rows in enumerate(taken):
        for j in rows:
            one = ints([0, 1])
            y1 = w12.short_conv(xd[j:j + 1], wd, past1, one, ints([i]), dst=ints([i]))
            assert torch.equal(y1.view(torch.int16), y[j:j + 1].view(torch.int16)), "a node's convolution is its path's"
            w12.gated_delta(*split(y1), gd[j:j + 1], bd[j:j + 1], state1, one, ints([i]), dst=ints([i]))
    assert torch.equal(past1, pastd) and torch.equal(state1, stated)
    # and the tree's outputs are those of its paths, to what either may be off
    for i, rows in enumerate(taken):
        st = state[i].cuda().clone()[None]
        o = w12.gated_delta(*split(y), gd, bd, st, ints([0, len(rows)]), ints([0]), rows=ints(rows + [-1] * (t - len(rows))))
        assert (o[rows].float() - out[rows].float()).abs().max() <= 0.05 * out[rows].float().abs().max()


@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_conv_in_place_equals_out_of_place(width, dtype):
    """A state that is replaced where it stands is read by nobody after: sequences of all lengths about a tile's, at many channels."""
    lengths = [1, 2, 3, 4, 5, 6, 7, 8, 9, 17] * 12
    t, b, c = sum(lengths), len(lengths), 2056
    x = rnd(1, t, c).to(dtype).cuda()
    weight = rnd(2, c, width).to(BF).cuda()
    past = torch.zeros(2 * b, width - 1, c, dtype=dtype, device="cuda")
    past[:b] = rnd(3, b, width - 1, c).to(dtype).cuda()
    ptr, here, there = ints(starts(lengths)), ints(list(range(b))), ints(list(range(b, 2 * b)))
    want = w12.short_conv(x, weight, past, ptr, here, dst=there)
    for _ in range(3):
        state = past[:b].clone()
        got = w12.short_conv(x, weight, state, ptr, here, dst=here)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        assert torch.equal(state, past[b:])
