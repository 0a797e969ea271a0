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
