"""GPU tests of the gated delta rule with values at the edges of their type, token by token and 64 at a time."""
import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from test_gpu_hybrid import Delta, ints, starts

pytestmark = pytest.mark.gpu

def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


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
