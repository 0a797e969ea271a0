"""The example's layer step: what its operators give when they run together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_layer.py")
    spec = importlib.util.spec_from_file_location("verify_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rows(m, n, seed):
    return torch.randn(n, m.HIDDEN, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))


def test_chain_as_a_tree_is_the_chain(example):
    """The same nodes with and without a mask: one computation, the same bits."""
    layer = example.Layer()
    layer.step(_rows(example, 200, 1), 0)
    x = _rows(example, 7, 2)
    depth, mask = example.tree_of([-1, 0, 1, 2, 3, 4, 5])
    a, (yq, sa) = layer.step(x, 200, depth, mask)
    b, (zq, sb) = layer.step(x, 200)
    assert torch.isfinite(a).all()
    assert torch.equal(a, b) and torch.equal(yq.view(torch.uint8), zq.view(torch.uint8)) and torch.equal(sa, sb)


def test_siblings_do_not_see_each_other(example):
    """Another value in one branch leaves the rows of the other branches as they were, bit for bit."""
    layer = example.Layer()
    layer.step(_rows(example, 100, 3), 0)
    x = _rows(example, 5, 4)
    depth, mask = example.tree_of([-1, 0, 0, 1, 2])      # 0 -> 1 -> 3, 0 -> 2 -> 4
    a, _ = layer.step(x, 100, depth, mask)
    x[2] = -x[2] + 1
    b, _ = layer.step(x, 100, depth, mask)
    same = [0, 1, 3]
    assert torch.equal(a[same], b[same])
    assert not torch.equal(a[2], b[2]) and not torch.equal(a[4], b[4])


def test_drafter_mlp(example):
    """The 8-bit product of the quantised rows against its formula in 64 bits: FP32 sums of n products are off by at
    most n 2^-24 of the sum of magnitudes, and each scale and its product by 2^-24 (3 in all)."""
    layer = example.Layer()
    _, (yq, ys) = layer.step(_rows(example, 9, 5), 0)
    w, ws = layer.up8
    got = example.w12.gemm_e4m3(yq, ys, w, ws).double()
    a = yq.double() * ys.double().repeat_interleave(128, 1)
    b = w.double() * ws.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    bound = (example.HIDDEN + 3) * 2.0 ** -24 * (a.abs() @ b.abs().t())
    assert ((got - a @ b.t()).abs() <= bound).all()
    assert torch.isfinite(layer.drafter_mlp(yq, ys)).all()
