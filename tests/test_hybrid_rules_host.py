"""Host-side checks of the rule by which gated_delta() has use for a workspace: the binding allocates one where the library asks for it."""
import os
import re

import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from lossless_bit_weight_encode_amd import _lib as L

I32, BF = torch.int32, torch.bfloat16


def test_the_binding_has_the_header_s_numbers():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "w12.h")).read()
    for name in ("DELTA_CHUNK_FROM", "DELTA_CHUNK_FROM_LENS", "DELTA_CHUNK_LONG"):
        assert int(re.search(rf"#define W12_{name} (\d+)", text).group(1)) == getattr(w12, name)


FEW, LENS, LONG = w12.DELTA_CHUNK_FROM, w12.DELTA_CHUNK_FROM_LENS, w12.DELTA_CHUNK_LONG


@pytest.mark.parametrize("t,count,form,used", [
    (1, 1, "", False), (FEW - 1, 1, "", False), (FEW, 1, "", True), (2 * FEW - 1, 2, "", False), (2 * FEW, 2, "", True),
    (30, 30, "", False), (29 + LONG - 1, 30, "", False), (29 + LONG, 30, "", True), (1000, 30, "", True),
    (LENS - 1, 1, "lens", False), (LENS, 1, "lens", True), (29 + LONG, 30, "lens", False), (1000, 30, "lens", False),
    (30 * LENS, 30, "lens", True), (1, 1, "tree", True), (30, 30, "tree", True),
])
def test_a_workspace_where_it_is_of_use(monkeypatch, t, count, form, used):
    from lossless_bit_weight_encode_amd import _hybrid, _ops
    given = []

    class Library:
        w12_gated_delta_workspace_size = L.lib().w12_gated_delta_workspace_size

        @staticmethod
        def w12_gated_delta(a, s, ws, ws_bytes, stream):
            given.append((ws, ws_bytes))
            return 0

    monkeypatch.setattr(_hybrid, "lib", lambda: Library)
    monkeypatch.setattr(_hybrid, "_device", lambda *a: 0)
    monkeypatch.setattr(_ops, "_current_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    ints = lambda n: torch.zeros(n, dtype=I32)
    more = {"": {}, "lens": dict(lens=ints(count)), "tree": dict(tree_mask=torch.zeros(t, 1, dtype=torch.int64))}[form]
    q, k, v = (torch.zeros(t, 64, dtype=BF) for _ in range(3))
    w12.gated_delta(q, k, v, torch.zeros(t, 1), torch.zeros(t, 1), torch.zeros(1, 1, 64, 64), ints(count + 1), ints(count), **more)
    (ws, ws_bytes), = given
    assert (ws is not None) == used
    assert ws_bytes == (w12.gated_delta_workspace_size(t, count, 1, 64, 64) if used else 0)
