"""GPU tests of the gated delta rule's calls whose sequences are of all lengths: which of them are taken token by token and which 64 at a
time goes by each one's own tokens."""
import random

import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from test_gpu_hybrid import Delta, ints, starts
from test_gpu_hybrid_calls import replays
from test_gpu_operators import BF, out_buf

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 256)])
@pytest.mark.parametrize("lengths", [[1] * 30 + [700] + [1] * 33, [64] + [1] * 20, [1, 0, 90, 0, 2, 11, 1] + [1] * 40,
                                     [100, 3, 12, 11, 70], [200, 1, 64] + [1, 0] * 30, [65] * 3 + [1] * 100])
def test_a_sequence_does_not_depend_on_its_neighbours(dk, dv, lengths):
    """Every sequence's outputs and state are, bit for bit, those of a call that it has to itself."""
    t, b, ptr = sum(lengths), len(lengths), starts(lengths, 2)
    d = Delta(t + 5, 2 * b, 2, 4, dk, dv, seed=200)
    mats, state = d.on_gpu()
    alone = state.clone()
    out, ok = out_buf(t + 5, 4 * dv, 4 * dv + 8, BF)
    w12.gated_delta(*mats, state, ints(ptr), ints(list(range(b))), dst=ints(list(range(b, 2 * b))), out=out)
    assert ok() and (out.cpu()[t + 2:].view(torch.int16) == 0x55).all()
    want = torch.zeros_like(out)
    for i in range(b):
        rows = slice(ptr[i], ptr[i + 1])
        if lengths[i]:
            want[rows] = w12.gated_delta(*(m[rows] for m in mats), alone, ints([0, lengths[i]]), ints([i]), dst=ints([b + i]))
        else:
            alone[b + i] = alone[i]
    assert same(out[2:t + 2], want[2:t + 2]) and torch.equal(state, alone)
    # without outputs, without new states
    _, again = d.on_gpu()
    w12.gated_delta(None, *mats[1:], again, ints(ptr), ints(list(range(b))), dst=ints(list(range(b, 2 * b))), outputs=False)
    assert torch.equal(again, state)
    stays = w12.gated_delta(*mats, again, ints(ptr), ints(list(range(b))))
    assert same(stays[2:t + 2], want[2:t + 2]) and torch.equal(again, state)


def test_sequences_of_all_lengths_are_right():
    lengths = [1, 300, 0, 1, 12, 1, 1, 64, 2] + [1] * 40
    t, b, ptr = sum(lengths), len(lengths), starts(lengths)
    d = Delta(t, 2 * b, 1, 2, 64, 64, seed=210)
    mats, state = d.on_gpu()
    out, ok = out_buf(t, 128, 128, BF)
    same_slots = ints(list(range(b)))
    w12.gated_delta(*mats, state, ints(ptr), same_slots, dst=same_slots, out=out)
    assert ok()
    d.check(out, state, [(list(range(ptr[i], ptr[i + 1])), i, i, None) for i in range(b)])


@pytest.mark.parametrize("lens", [[40, 3, 65, 1], [12, 11, 0, 64], [200, 1, 1, 1]])
def test_lengths_that_the_host_does_not_know(lens):
    """A padded batch: each sequence is what it is alone, whatever its neighbours' lengths; rows behind a length are left."""
    room = 200
    t, b, ptr = 4 * room, 4, [room * i for i in range(5)]
    d = Delta(t, 2 * b, 2, 4, 128, 64, seed=220)
    mats, state = d.on_gpu()
    alone = state.clone()
    out, ok = out_buf(t, 256, 256, BF)
    w12.gated_delta(*mats, state, ints(ptr), ints(list(range(b))), dst=ints(list(range(b, 2 * b))), lens=ints(lens), out=out)
    assert ok()
    for i, n in enumerate(lens):
        rows = slice(ptr[i], ptr[i] + n)
        if n:
            want = w12.gated_delta(*(m[rows] for m in mats), alone, ints([0, n]), ints([i]), dst=ints([b + i]))
            assert same(out[rows], want)
        else:
            alone[b + i] = alone[i]
        assert (out.cpu()[ptr[i] + n:ptr[i + 1]].view(torch.int16) == 0x55).all()
    assert torch.equal(state, alone)


def test_a_long_sequence_among_many_short_ones_token_by_token():
    """With lens and few rows a sequence, tokens go one by one however long a sequence is."""
    lengths, b = [200] + [3] * 9, 10
    t, ptr = sum(lengths), starts(lengths)
    d = Delta(t, 2 * b, 1, 2, 128, 64, seed=230)
    mats, state = d.on_gpu()
    out, ok = out_buf(t, 128, 128, BF)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    w12.gated_delta(*mats, state, ints(ptr), ints(list(range(b))), dst=ints(list(range(b, 2 * b))), lens=ints(lengths), out=out, ws=none)
    assert ok()
    seqs = [(list(range(ptr[i], ptr[i + 1])), i, b + i, None) for i in range(b)]
    d.check(out, state, seqs)
    # so they do in any call of fewer than 12 rows a sequence that has no workspace, or one that is too small
    need = w12.gated_delta_workspace_size(t + 60, b + 60, 2, 128, 64)
    for ws in (none, torch.empty(need // 2, dtype=torch.uint8, device="cuda")):
        _, again = d.on_gpu()
        lone, ok = out_buf(t, 128, 128, BF)
        src = ints(list(range(b)) + [-1] * 60)
        dst = ints(list(range(b, 2 * b)) + [-1] * 60)
        w12.gated_delta(*mats, again, ints(ptr + [t] * 60), src, dst=dst, out=lone, ws=ws)
        assert ok() and same(lone, out) and torch.equal(again, state)


def test_replays_with_lengths_that_change():
    """A captured call follows its ranges: a long sequence becomes short, and short ones long."""
    t, b = 300, 20
    r = random.Random(1)
    d = Delta(t, 2 * b, 2, 4, 128, 128, seed=240)
    mats, state = d.on_gpu()
    first = state.clone()
    ptr = ints(starts([200] + [1] * 18 + [82]))
    src, dst = ints(list(range(b))), ints(list(range(b, 2 * b)))
    out, seen = torch.zeros(t, 512, dtype=BF, device="cuda"), torch.zeros_like(state)
    ws = w12.gated_delta_workspace(t, b, state)

    def change(i):
        if i == 0:
            ptr.copy_(ints([0] * 20 + [t]))
        elif i == 1:
            ptr.copy_(ints([0] + [t] * 20))
        else:
            ptr.copy_(ints(sorted(r.randint(0, t) for _ in range(21))))

    def call():
        state.copy_(first)
        out.zero_()
        w12.gated_delta(*mats, state, ptr, src, dst=dst, out=out, ws=ws)
        seen.copy_(state)

    replays(call, [out, seen], change, n=6)


def test_many_long_sequences_among_short_ones():
    """More long sequences than the chip has work-groups for at a time, though the mean is short."""
    r = random.Random(2)
    lengths = [14] * 200 + [0] * 100
    r.shuffle(lengths)
    t, b, ptr = sum(lengths), 300, starts(lengths)
    d = Delta(t, 2 * b, 4, 4, 64, 128, seed=250)
    mats, state = d.on_gpu()
    alone = state.clone()
    out = w12.gated_delta(*mats, state, ints(ptr), ints(list(range(b))), dst=ints(list(range(b, 2 * b))))
    for i in r.sample(range(b), 40):
        rows = slice(ptr[i], ptr[i + 1])
        if lengths[i]:
            want = w12.gated_delta(*(m[rows] for m in mats), alone, ints([0, lengths[i]]), ints([i]), dst=ints([b + i]))
            assert same(out[rows], want)
        else:
            alone[b + i] = alone[i]
        assert torch.equal(state[b + i], alone[b + i])


@pytest.mark.parametrize("lengths", [[70, 1, 13, 0, 2] + [1] * 30, [14] * 120 + [1, 0] * 40])
def test_rows_of_long_and_short_sequences(lengths):
    """Rows that are named, in any order, some of them none; with and without new states."""
    r = random.Random(3)
    t, b, ptr = sum(lengths), len(lengths), starts(lengths)
    d = Delta(t, 2 * b, 4, 4, 64, 128, seed=260)
    mats, state = d.on_gpu()
    rows = list(range(t))
    r.shuffle(rows)
    for i in r.sample(range(t), 5):
        rows[i] = r.choice((-1, t, -7))
    src, dst, named = ints(list(range(b))), ints([b + i if i % 5 else -1 for i in range(b)]), ints(rows)
    out, ok = out_buf(t, 512, 512, BF)
    w12.gated_delta(*mats, state, ints(ptr), src, dst=dst, rows=named, out=out)
    assert ok()
    # the rows laid out in their order, zeros for none of them
    there = torch.tensor([0 <= x < t for x in rows])
    at = torch.tensor([x if 0 <= x < t else 0 for x in rows]).cuda()
    laid = [m[at] * there.cuda()[:, None] for m in mats]
    _, alone = d.on_gpu()
    want = w12.gated_delta(*laid, alone, ints(ptr), src, dst=dst)
    assert torch.equal(state, alone) and same(out[at[there.cuda()]], want[there.cuda()])
    left = sorted(set(range(t)) - {x for x in rows if 0 <= x < t})
    assert (out.cpu()[left].view(torch.int16) == 0x55).all()
    stays = w12.gated_delta(*mats, state, ints(ptr), src, rows=named)
    assert torch.equal(state, alone) and same(stays[at[there.cuda()]], want[there.cuda()])


def test_what_is_no_number_stays_in_its_sequence():
    """Among many long and short sequences, of which a work-group takes several one after another."""
    lengths = [14] * 120 + [3] * 60
    random.Random(4).shuffle(lengths)
    t, b, ptr = sum(lengths), len(lengths), starts(lengths)
    d = Delta(t, 2 * b, 4, 4, 64, 128, seed=270)
    mats, state = d.on_gpu()
    clean_state = state.clone()
    args = (ints(ptr), ints(list(range(b))))
    clean = w12.gated_delta(*mats, clean_state, *args, dst=ints(list(range(b, 2 * b))))
    hit = [5, 50, 51, 100, 170]
    for i in hit:
        mats[1][ptr[i] + 1, 0] = float("nan")
    dirty = w12.gated_delta(*mats, state, *args, dst=ints(list(range(b, 2 * b))))
    bad_rows = torch.zeros(t, dtype=torch.bool)
    for i in hit:
        bad_rows[ptr[i] + 1:ptr[i + 1]] = True
        assert state[b + i, 0].isnan().all() and torch.equal(state[b + i, 1:], clean_state[b + i, 1:])
    assert dirty[bad_rows][:, :128].isnan().all() and same(dirty[:, 128:], clean[:, 128:])
    assert same(dirty[~bad_rows], clean[~bad_rows])
    others = [b + i for i in range(b) if i not in hit]
    assert torch.equal(state[others], clean_state[others])
