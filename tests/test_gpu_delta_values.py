"""GPU tests of the gated delta rule with values at the edges of their type, token by token and 64 at a time."""
import random

import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from hybrid_util import mask_of, tree
from test_gpu_hybrid import Delta, ints, starts

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("lengths,at", [([11, 3], 4), ([11, 3], 10), ([1, 1], 0), ([150, 30], 70), ([150, 30], 149), ([64, 5], 3)])
@pytest.mark.parametrize("what", ["k", "v", "q", "g", "beta"])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_what_is_no_number_reaches_what_follows(lengths, at, what, value):
    """All of it: every later token of the heads that use it and their new state; of v its own column; of q its own token alone."""
    if what == "g" and value == -INF:
        pytest.skip("a log decay of -inf is a number: it clears the state")
    t = sum(lengths)
    d = Delta(t, 4, 2, 4, 128, 128, seed=300)
    mats, state = d.on_gpu()
    clean_state = state.clone()
    ptr, src, dst = ints(starts(lengths)), ints([0, 1]), ints([2, 3])
    clean = w12.gated_delta(*mats, clean_state, ptr, src, dst=dst)
    mats[["q", "k", "v", "g", "beta"].index(what)][at, 0] = value
    dirty = w12.gated_delta(*mats, state, ptr, src, dst=dst)
    heads = 2 if what in "qk" else 1                      # value heads that use it
    wide = 1 if what == "v" else heads * 128              # and their columns
    n = lengths[0]
    assert same(dirty[:at], clean[:at]) and same(dirty[n:], clean[n:]) and torch.equal(state[3], clean_state[3])
    assert same(dirty[:, wide:], clean[:, wide:])
    assert not dirty[at, :wide].isfinite().any()
    if what == "q":
        assert same(dirty[at + 1:], clean[at + 1:]) and torch.equal(state, clean_state)
    else:
        assert not dirty[at:n, :wide].isfinite().any()
        new, old = state[2].flatten(0, 1), clean_state[2].flatten(0, 1)      # [heads x columns, dk]
        assert not new[:wide].isfinite().any() and torch.equal(new[wide:], old[wide:])


@pytest.mark.parametrize("what", ["k", "v", "q", "g", "beta"])
@pytest.mark.parametrize("value", [NAN, INF])
def test_in_a_tree_it_reaches_all_descendants(what, value):
    nodes = 50
    parents = tree(random.Random(4), nodes)
    mask = mask_of(parents).cuda()
    d = Delta(nodes, 1, 2, 4, 64, 64, seed=310)
    mats, state = d.on_gpu()
    call = dict(tree_mask=mask)
    clean = w12.gated_delta(*mats, state, ints([0, nodes]), ints([0]), **call)
    paths = [int(m) for m in mask[:, 0].tolist()]
    node = max(range(1, 20), key=lambda i: sum(p >> i & 1 for p in paths))
    mats[["q", "k", "v", "g", "beta"].index(what)][node, 0] = value
    dirty = w12.gated_delta(*mats, state, ints([0, nodes]), ints([0]), **call)
    wide = 1 if what == "v" else (2 if what == "q" or what == "k" else 1) * 64
    hit = torch.tensor([bool(p >> node & 1) if what != "q" else i == node for i, p in enumerate(paths)])
    assert what == "q" or hit.sum() > 2
    assert same(dirty[~hit], clean[~hit]) and same(dirty[:, wide:], clean[:, wide:])
    assert not dirty[hit][:, :wide].isfinite().any()


@pytest.mark.parametrize("lengths", [[5, 3], [90, 12]])
@pytest.mark.parametrize("size", [1e25, 2e19])
@pytest.mark.parametrize("what", ["q", "k"])
def test_a_norm_past_its_type_is_no_number(lengths, size, what):
    """Values whose squares add up to more than FP32 holds: what follows is NaN, not a key or a query of zeros."""
    t, at = sum(lengths), 2
    d = Delta(t, 4, 1, 2, 64, 64, seed=320)
    mats, state = d.on_gpu()
    ptr, src, dst = ints(starts(lengths)), ints([0, 1]), ints([2, 3])
    clean_state = state.clone()
    clean = w12.gated_delta(*mats, clean_state, ptr, src, dst=dst)
    mats["qk".index(what)][at, 5] = size
    out = w12.gated_delta(*mats, state, ptr, src, dst=dst)
    n = lengths[0]
    assert same(out[:at], clean[:at]) and same(out[n:], clean[n:])
    assert out[at].isnan().all()
    if what == "q":
        assert same(out[at + 1:n], clean[at + 1:n]) and torch.equal(state, clean_state)
    else:
        assert out[at:n].isnan().all() and state[2].isnan().all() and torch.equal(state[3], clean_state[3])


@pytest.mark.parametrize("lengths", [[5], [90]])
@pytest.mark.parametrize("what", ["q", "k"])
@pytest.mark.parametrize("size", [0.0, 1e-23])
def test_a_norm_of_nothing_is_no_number_without_eps(lengths, what, size):
    """Sums of squares of 0, or too small for their type, with eps 0; with the usual eps they are numbers."""
    n, at = lengths[0], 2
    d = Delta(n, 2, 1, 1, 64, 64, seed=330)
    mats, state = d.on_gpu()
    mats["qk".index(what)][at] = size
    args = (ints([0, n]), ints([0]))
    assert w12.gated_delta(*mats, state.clone(), *args, dst=ints([1])).isfinite().all()
    out = w12.gated_delta(*mats, state, *args, dst=ints([1]), eps=0.0)
    assert out[:at].isfinite().all() and out[at].isnan().all()
    if what == "q":
        assert out[at + 1:].isfinite().all() and state.isfinite().all()
    else:
        assert out[at:].isnan().all() and state[1].isnan().all()
