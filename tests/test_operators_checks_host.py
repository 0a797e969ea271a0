"""Host-side checks of the operators' binding and schedules: what has to happen before anything is launched, and
what a launch is sized for.  No GPU is touched."""
import contextlib

import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from lossless_bit_weight_encode_amd import _lib as L
from test_operators_host import cache


class _Recorder:
    """A stand-in for the library: notes the calls that would launch something, and asks the real one for sizes."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return getattr(L.lib(), name)
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def recorder(monkeypatch):
    """The binding with neither library nor GPU behind it: what it would have launched is in the recorder."""
    from lossless_bit_weight_encode_amd import _ops
    rec = _Recorder()
    monkeypatch.setattr(_ops, "lib", lambda: rec)
    monkeypatch.setattr(_ops, "_current_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    return rec


def _cpu_cache():
    """A cache handle as KVCache would refuse to make it, for the checks of the calls themselves."""
    c = w12.KVCache.__new__(w12.KVCache)
    c.k = c.v = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    c.k_scale = c.v_scale = None
    c.pages, c.page_size, c.heads, c.dim, c.desc = 2, 16, 1, 64, cache(pages=2, heads=1)
    return c


@pytest.mark.parametrize("call", [
    lambda bf, f8: w12.gemm_e4m3(torch.zeros(1, 17408).to(f8), torch.ones(1, 136), torch.zeros(5120, 17408).to(f8),
                                 torch.ones(40, 136)),
    lambda bf, f8: w12.gemm_e4m3_workspace(1, 5120, 17408, "cpu"),
    lambda bf, f8: w12.gemm_e4m3_workspace(1, 5120, 17408, torch.device("cuda", 1)),
    lambda bf, f8: w12.add_rmsnorm(torch.zeros(2, 64, dtype=bf), torch.ones(64, dtype=bf)),
    lambda bf, f8: w12.rope_append(torch.zeros(1, 192), _cpu_cache(), torch.zeros(1, 1, dtype=torch.int32),
                                   torch.zeros(1, dtype=torch.int64), torch.zeros(32, dtype=torch.float64), 1),
    lambda bf, f8: w12.tree_attention(torch.zeros(1, 64, dtype=bf), _cpu_cache(), torch.zeros(1, 1, dtype=torch.int32),
                                      torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)),
], ids=["gemm_e4m3", "workspace_cpu", "workspace_other_gpu", "norm", "rope", "attention"])
def test_nothing_is_launched_before_the_tensors_are_checked(recorder, monkeypatch, call):
    """Outputs and workspaces that a call would allocate itself: a launch on them would reach host memory, or a GPU
    that is not the current one."""
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(a) or empty(*a, **{**k, "device": "cpu"}))
    with pytest.raises(ValueError, match="GPU"):
        call(torch.bfloat16, torch.float8_e4m3fn)
    assert recorder.calls == [] and made == []
