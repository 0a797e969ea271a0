"""GPU tests of the hybrid target's operators at the sizes that take other schedules: long prompts, many sequences, many rows of a large
vocabulary; and of the workspace that a call needs."""
import random

import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from hybrid_util import conv_ref, delta_steps, tree
from test_gpu_hybrid import Delta, conv_tol, ints, starts, verify_case, verify_check
from test_gpu_operators import BF, F32, assert_close, out_buf, rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 2, 128, 128), (1, 1, 64, 256)])
def test_delta_long_prompt(hk, hv, dk, dv):
    t = 2083
    d = Delta(t, 2, hk, hv, dk, dv, seed=40)
    (q, k, v, g, beta), state = d.on_gpu()
    out, ok = out_buf(t, hv * dv, hv * dv, BF)
    w12.gated_delta(q, k, v, g, beta, state, ints([0, t]), ints([1]), dst=ints([0]), out=out)
    assert ok()
    d.check(out, state, [(list(range(t)), 1, 0, None)])
    # the states alone are the same ones
    again = d.on_gpu()[1]
    w12.gated_delta(None, k, v, g, beta, again, ints([0, t]), ints([1]), dst=ints([0]), outputs=False)
    assert torch.equal(state, again)


@pytest.mark.parametrize("most", [2, 60, 150])
def test_delta_many_sequences(most):
    """300 sequences: more than a work-group has lanes, or threads, to look for its own; some without tokens."""
    r = random.Random(most)
    lengths = [r.randint(0, most) for _ in range(300)]
    t, ptr = sum(lengths), starts(lengths)
    d = Delta(t, 601, 1, 2, 64, 64, seed=50)
    (q, k, v, g, beta), state = d.on_gpu()
    slots = list(range(601))
    r.shuffle(slots)
    out, ok = out_buf(t, 128, 128, BF)
    w12.gated_delta(q, k, v, g, beta, state, ints(ptr), ints(slots[:300]), dst=ints(slots[300:600]), out=out)
    assert ok()
    sample = sorted(r.sample(range(300), 40))
    for i in range(300):
        if i not in sample:
            d.state[slots[300 + i]] = state[slots[300 + i]].cpu()
    d.check(out, state, [(list(range(ptr[i], ptr[i + 1])), slots[i], slots[300 + i], None) for i in sample])


def test_delta_many_trees():
    r = random.Random(3)
    nodes = [r.randint(0, 64) for _ in range(90)]
    parents = [tree(r, n) for n in nodes]
    from hybrid_util import mask_of
    t, ptr = sum(nodes), starts(nodes)
    d = Delta(t, 90, 1, 1, 128, 64, seed=60)
    (q, k, v, g, beta), state = d.on_gpu()
    out, ok = out_buf(t, 64, 64, BF)
    mask = torch.cat([mask_of(p) for p in parents if p]).cuda()
    w12.gated_delta(q, k, v, g, beta, state, ints(ptr), ints(list(range(90))), tree_mask=mask, out=out)
    assert ok()
    d.check(out, state, [(list(range(ptr[i], ptr[i + 1])), i, None, parents[i]) for i in range(90)])


@pytest.mark.parametrize("n", [5, 80])
def test_delta_rows_that_are_none_change_nothing(n):
    """Also where eps is 0, and a norm of zeros would be no number; n of 80: taken 64 at a time."""
    d = Delta(n, 3, 2, 2, 64, 64, seed=70)
    d.eps = 0.0
    (q, k, v, g, beta), state = d.on_gpu()
    rows = list(range(n - 2))
    out, ok = out_buf(n, 128, 128, BF)
    named = ints(rows[:2] + [-1, n, *rows[2:]])
    w12.gated_delta(q, k, v, g, beta, state, ints([0, n]), ints([0]), dst=ints([2]), rows=named, out=out, eps=0.0)
    assert ok()
    d.check(out, state, [(rows, 0, 2, None)])
    assert (out.cpu()[n - 2:].view(torch.int16) == 0x55).all()


def test_delta_workspace_where_it_is_needed():
    d = Delta(140, 6, 1, 2, 64, 64, seed=80)
    (q, k, v, g, beta), state = d.on_gpu()
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    few, enough = w12.DELTA_CHUNK_FROM, w12.DELTA_CHUNK_FROM_LENS

    def call(t, seqs, lens=None, ws=None, **more):
        out = torch.zeros(t, 128, dtype=BF, device="cuda")      # rows past lens are left as they are
        ptr = ints([0] + [t] * seqs)
        w12.gated_delta(*(x[:t] for x in (q, k, v, g, beta)), state, ptr, ints(list(range(seqs))), out=out, ws=ws, lens=lens, **more)
        return out

    for t, seqs, lens in ((few - 1, 1, None), (2 * few - 1, 2, None), (enough - 1, 1, ints([70])), (2 * enough - 1, 2, ints([70, 0]))):
        assert torch.equal(call(t, seqs, lens, none), call(t, seqs, lens))
    mask = torch.ones(1, 1, dtype=torch.int64, device="cuda")
    for t, seqs, more in ((few, 1, {}), (2 * few, 2, {}), (enough, 1, dict(lens=ints([70]))), (1, 1, dict(tree_mask=mask))):
        need = w12.gated_delta_workspace_size(t, seqs, 2, 64, 64)
        for short in (none, torch.empty(need - 1, dtype=torch.uint8, device="cuda")):
            with pytest.raises(RuntimeError, match="workspace"):
                call(t, seqs, ws=short, **more)
        call(t, seqs, ws=torch.empty(need, dtype=torch.uint8, device="cuda"), **more)


@pytest.mark.parametrize("src", [F32, BF])
@pytest.mark.parametrize("c", [4100, 8200])
def test_conv_long_tiles(src, c):
    """Rows and channels enough for the long tiles; sequences that end inside of them."""
    lengths, w = [2500, 0, 1, 15, 16, 17, 1547], 4
    t, b, ptr = sum(lengths), len(lengths), starts(lengths)
    ld = (c + 8) // 8 * 8
    x = torch.zeros(t, ld, dtype=src)
    x[:, :c] = rnd(1, t, c).to(src)
    past = torch.zeros(2 * b, w - 1, ld, dtype=src)
    past[:, :, :c] = rnd(2, 2 * b, w - 1, c).to(src)
    weight, bias = rnd(3, c, w, scale=0.6).to(BF), rnd(4, c).to(BF)
    state = past.cuda()[:, :, :c]
    y, ok = out_buf(t, c, ld, BF)
    w12.short_conv(x.cuda()[:, :c], weight.cuda(), state, ints(ptr), ints(list(range(b))), dst=ints(list(range(b, 2 * b))), bias=bias.cuda(), y=y)
    assert ok()
    want = past[:, :, :c].clone()
    for i in range(b):
        args = (x[ptr[i]:ptr[i + 1], :c].double(), weight.double(), bias.double(), past[i, :, :c].double())
        ref, mag, new = conv_ref(*args, True)
        pre = conv_ref(*args, False)[0]
        assert_close(y[ptr[i]:ptr[i + 1]], ref, conv_tol(ref, mag, pre, w) + 1e-38, "y")
        want[b + i] = new.to(src)
    assert torch.equal(state.cpu(), want)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("form,with_q", [("tree", False), ("chain", True)])
@pytest.mark.parametrize("nodes,v", [([40, 64, 0, 60, 36], 90001), ([3, 1, 0, 2] * 40, 1237), ([2], 1048579)])
def test_verify_schedules(dtype, form, with_q, nodes, v):
    """Long pieces of a row; more requests than a wave has lanes; a vocabulary with more pieces than a work-group threads."""
    count = verify_check(verify_case(90 + len(nodes), nodes, v, form, "mixed", with_q, dtype))
    assert len(nodes) < 3 or max(count) > 1
