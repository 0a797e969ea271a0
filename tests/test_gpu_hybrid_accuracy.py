"""GPU tests of how near the gated delta rule's outputs are to 64 bits where tokens are taken 64 at a time: their rounding to BF16,
and nothing else of that size."""
import random

import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from hybrid_util import B8, BIG, S16, ancestors, delta_bounds, delta_steps, mask_of, tree
from test_gpu_hybrid import Delta, ints, starts
from test_gpu_operators import BF, assert_close

pytestmark = pytest.mark.gpu


def magnitudes(q, k, v, g, beta, s0, scale, l2, eps, parents=None):
    """scale e^G |Q| |S| and |P| |U| of every output, as in delta_bounds: the sums of magnitudes behind its two products."""
    if l2:
        q, k = (x / torch.sqrt((x * x).sum(1, keepdim=True) + eps) for x in (q, k))
    n, s = k.shape[0], s0
    qs, pu = (torch.zeros(n, v.shape[1], dtype=torch.float64) for _ in range(2))
    step = n if parents is not None else BIG
    for c in range(0, n, step):
        qc, kc, vc, gc, bc = (x[c:c + step] for x in (q, k, v, g, beta))
        m = kc.shape[0]
        before = torch.ones(m, m, dtype=torch.bool).tril(-1)
        if parents is not None:
            before = torch.zeros(m, m, dtype=torch.bool)
            for i, up in enumerate(ancestors(parents)):
                before[i, sorted(up)] = True
        eye = torch.eye(m, dtype=torch.float64)
        own = before | eye.bool()
        total = own.double() @ gc
        decay = torch.where(own, torch.exp(torch.where(own, total[:, None] - total[None], 0.0)), 0.0)
        a = torch.where(before, bc[:, None] * (kc @ kc.t()) * decay, 0.0)
        grown = torch.exp(total)[:, None]
        u = torch.linalg.solve_triangular(a + eye, bc[:, None] * (vc - grown * (kc @ s)), upper=False)
        qs[c:c + m] = scale * grown * (qc.abs() @ s.abs())
        pu[c:c + m] = (scale * decay * (qc @ kc.t())).abs() @ u.abs()
        s = torch.exp(total[-1]) * s + (torch.exp(total[-1] - total)[:, None] * kc).t() @ u
    return qs, pu


def check(d, out, rows, src, parents=None):
    for h in range(d.hv):
        args = d.head(h, rows, src)
        o, _ = delta_steps(*args, parents=parents)
        qs, pu = magnitudes(*args, parents=parents)
        # delta_bounds allows S and U (and P's rest) as one BF16 value each, off by 2^-8.  Two values are off by 2^-16; and of P U the
        # product of the two rests, of 2^-8 each, may be left out.
        tol = delta_bounds(*args, parents=parents)[0] - 1.01 * (1.02 * B8 * qs + 2.04 * B8 * pu) + 1.01 * S16 * (qs + 3.1 * pu)
        assert_close(out[torch.tensor(rows), h * d.dv:(h + 1) * d.dv], o, tol, f"out, head {h}")


@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 2, 128, 128), (1, 1, 64, 256), (1, 2, 128, 64)])
@pytest.mark.parametrize("lengths", [[12], [64], [65], [300, 17, 128]])
def test_delta_outputs_are_rounded_once(hk, hv, dk, dv, lengths):
    t, b, ptr = sum(lengths), len(lengths), starts(lengths)
    d = Delta(t, 2 * b, hk, hv, dk, dv, seed=100)
    (q, k, v, g, beta), state = d.on_gpu()
    out = w12.gated_delta(q, k, v, g, beta, state, ints(ptr), ints(list(range(b))), dst=ints(list(range(b, 2 * b))))
    for i in range(b):
        check(d, out, list(range(ptr[i], ptr[i + 1])), i)
    # the state stays: the outputs are the same
    _, state = d.on_gpu()
    stays = w12.gated_delta(q, k, v, g, beta, state, ints(ptr), ints(list(range(b))))
    assert torch.equal(out.view(torch.int16), stays.view(torch.int16))


@pytest.mark.parametrize("hk,hv,dk,dv", [(1, 2, 128, 128), (1, 1, 64, 64)])
@pytest.mark.parametrize("nodes", [[1], [24, 63, 5], [64]])
def test_delta_tree_outputs_are_rounded_once(hk, hv, dk, dv, nodes):
    t, b, ptr = sum(nodes), len(nodes), starts(nodes)
    parents = [tree(random.Random(n), n) for n in nodes]
    d = Delta(t, b, hk, hv, dk, dv, seed=110)
    (q, k, v, g, beta), state = d.on_gpu()
    mask = torch.cat([mask_of(p) for p in parents]).cuda()
    out = w12.gated_delta(q, k, v, g, beta, state, ints(ptr), ints(list(range(b))), tree_mask=mask)
    for i in range(b):
        check(d, out, list(range(ptr[i], ptr[i + 1])), i, parents[i])


def test_delta_outputs_with_states_of_any_size():
    """Columns of the state from 2^-40 to 2^40: what is left over after its first BF16 value counts at every size."""
    d = Delta(130, 2, 1, 1, 128, 64, seed=120)
    size = 2.0 ** torch.linspace(-40, 40, 64).round()
    d.state *= size[None, None, :, None]
    d.v = (d.v.float() * size[None]).to(BF)
    (q, k, v, g, beta), state = d.on_gpu()
    out = w12.gated_delta(q, k, v, g, beta, state, ints([0, 130]), ints([1]), dst=ints([0]))
    check(d, out, list(range(130)), 1)
