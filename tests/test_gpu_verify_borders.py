"""GPU tests of verify_draft where the running sum passes its target at a border between two pieces of a row."""
import numpy as np
import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from test_gpu_hybrid import ints

pytestmark = pytest.mark.gpu

VOCAB, PIECE = 131072, 2048


def rows_with_a_period(period, n, seed):
    """Rows whose runs of 2048 logits have weights that repeat with a period: sums over threads and waves are then rounded apart, and
    targets u times the total with few bits in u fall on borders between runs."""
    r = np.random.default_rng(seed)
    z = np.full((n, VOCAB), -np.inf, dtype=np.float32)
    for i in range(n):
        each = r.uniform(-2.0, 2.0, (period, 3)).astype(np.float32)
        for p in range(VOCAB // PIECE):
            at = p * PIECE + np.sort(r.choice(PIECE, 3, replace=False))
            z[i, at] = each[p % period]
    return z


def allowed(weights, u):
    """The tokens that the border's own error allows: the running sum passes u of the total, to 2^-40 of the total."""
    edges = np.cumsum(weights.astype(np.longdouble))
    total = edges[-1]
    target, off = np.longdouble(u) * total, total * np.longdouble(2.0) ** -40
    before = edges - weights
    return set(np.nonzero((weights > 0) & (before - off <= target) & (target < edges + off))[0].tolist())


@pytest.mark.parametrize("n", [60, 240])           # short pieces, and long ones
@pytest.mark.parametrize("period", [2, 4, 8])
def test_a_border_is_missed_by_a_neighbour_at_most(period, n):
    z = rows_with_a_period(period, n, period)
    u = ((np.arange(n) % 15 + 1) / 16).astype(np.float32)
    one = ints(list(range(n + 1)))
    got = w12.verify_draft(torch.tensor(z).cuda(), torch.zeros(n, dtype=torch.int32, device="cuda"), torch.tensor(u).cuda(), one)[2]
    far = []
    for i, token in enumerate(got.tolist()):
        may = allowed(np.exp(z[i].astype(np.longdouble) - z[i].max()), float(u[i]))
        assert 1 <= len(may) <= 2
        far += [] if token in may else [(i, float(u[i]), token, may)]
    assert not far, far[:5]


@pytest.mark.parametrize("period", [2, 4, 8])
def test_a_border_of_what_is_left_over_is_missed_by_a_neighbour_at_most(period):
    """Chains of two nodes whose second is rejected: its token has no probability, and what is left over is the row itself."""
    n = 45
    z = np.repeat(rows_with_a_period(period, n, 10 + period), 2, axis=0)
    tokens = np.zeros(2 * n, dtype=np.int32)
    q = torch.zeros(2 * n, VOCAB, device="cuda")
    for i in range(n):
        tokens[2 * i + 1] = np.nonzero(np.isneginf(z[2 * i]))[0][-1]
        q[2 * i + 1, int(tokens[2 * i + 1])] = 1.0
    u = np.zeros(2 * n, dtype=np.float32)
    u[::2] = ((np.arange(n) % 15 + 1) / 16).astype(np.float32)
    accept = torch.full((2 * n,), 0.5, device="cuda")
    got = w12.verify_draft(torch.tensor(z).cuda(), torch.tensor(tokens).cuda(), torch.tensor(u).cuda(), ints(list(range(0, 2 * n + 1, 2))),
                           q=q, accept_u=accept)
    assert got[1].tolist() == [1] * n
    far = []
    for i, token in enumerate(got[2].tolist()):
        may = allowed(np.exp(z[2 * i].astype(np.longdouble) - z[2 * i].max()), float(u[2 * i]))
        far += [] if token in may else [(i, float(u[2 * i]), token, may)]
    assert not far, far[:5]
