"""The recurrent layer's example: it runs, accepts what it drafted, and its states stand where the accepted tokens lead."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_example_runs():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_layer.py")
    spec = importlib.util.spec_from_file_location("recurrent_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    count, off = m.main()
    # from a node to its first child: 0, 1, 3, 6 and 0, 1, 2, 4
    assert count.tolist() == [4, 4]
    # a BF16 value that falls to its neighbour is off by 2^-7 of itself; a token's step has three of them (k twice, v or q) in a product
    assert max(off) <= 2.0 ** -5
