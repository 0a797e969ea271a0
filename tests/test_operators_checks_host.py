"""Host-side checks of the operators' binding and schedules: what has to happen before anything is launched, and
what a launch is sized for.  No GPU is touched."""
import contextlib
import os
import subprocess

import pytest
import torch

import lossless_bit_weight_encode_amd as w12
from lossless_bit_weight_encode_amd import _lib as L
from test_operators_host import cache, gemm


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


PLAN_MAIN = r"""
#include <cstdio>
#include <random>
#include <vector>
#include "w12_attention_plan.h"
using namespace w12;
// Plans a call and prints how it was cut; false where an item has no tile, the workspace no place for it, or the sums differ.
static bool plan(const std::vector<int>& nodes, const std::vector<int>& lens, int heads, int group, int target, bool show) {
  int64_t T = 0;
  for (int n : nodes) T += n;
  const int requests = (int)nodes.size();
  auto blocks = [&](int b) { return blocks_of(nodes[b] * group, lens[b]); };
  auto sum = [&](auto value) { int64_t s = 0; for (int b = 0; b < requests; ++b) s += value(b); return s; };
  const Plan p = plan_of(requests, heads, (int)(T * group), target, blocks, sum);
  const int64_t most = most_items(T * group, requests, heads, target);
  const int64_t items = p.chunk > 0 ? sum([&](int b) { return items_of(blocks(b), heads, p.chunk); }) : -1;
  const bool ok = p.chunk >= kMinChunk && items == p.items && p.items <= most;
  if (show || !ok)
    std::printf("%s requests %d heads %d group %d T %lld len %d: chunk %d items %lld of %lld\n", ok ? "ok" : "BAD", requests, heads,
                group, (long long)T, lens[0], p.chunk, (long long)p.items, (long long)most);
  return ok;
}
int main() {
  bool ok = true;
  // the largest lengths of every request, and of one beside short ones
  for (int heads : {8, 128, 1024})
    for (int target : {512, 1024}) {
      ok &= plan(std::vector<int>(1024, 1), std::vector<int>(1024, (1 << 30) - 1), heads, 1, target, true);
      ok &= plan(std::vector<int>(1024, 1024), std::vector<int>(1024, (1 << 30) - 1), heads, 1, target, true);
      std::vector<int> one(1000, 3);
      one[7] = (1 << 30) - 1;
      ok &= plan(std::vector<int>(1000, 2), one, heads, 4, target, true);
      ok &= plan({64}, {(1 << 30) - 1}, heads, 5, target, true);
    }
  std::mt19937 g(5);
  auto pick = [&](int lo, int hi) {      // spread over the logarithm
    const double l = std::uniform_real_distribution<>(0, 1)(g);
    return (int)(lo * std::pow((double)hi / lo, l));
  };
  for (int i = 0; i < 20000 && ok; ++i) {
    const int requests = i % 3 == 0 ? 1 : pick(1, 1024), heads = pick(1, 64), group = pick(1, 64);
    std::vector<int> nodes(requests), lens(requests);
    const int top = pick(1, 1 << 24), n = pick(1, requests == 1 ? 8192 : 300);
    for (int b = 0; b < requests; ++b) {
      nodes[b] = i % 2 ? n : std::uniform_int_distribution<>(0, n)(g);
      lens[b] = nodes[b] + (i % 5 ? std::uniform_int_distribution<>(0, top)(g) : b ? 0 : top);
    }
    ok &= plan(nodes, lens, heads, group, i % 7 ? 1024 : 512, false);
  }
  return ok ? 0 : 1;
}
"""


def test_attention_plan_fits_its_workspace(tmp_path):
    """The plan of a call, compiled for the host: every chunk has tiles, and the items fit what the workspace is sized
    for, over the lengths that the header allows (1024 requests of 2^30 - 1 tokens among them) and random batches."""
    src = tmp_path / "plan.cpp"
    src.write_text("#include <cmath>\n" + PLAN_MAIN)
    csrc = os.path.join(os.path.dirname(w12.__file__), "csrc")
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-O2", "-std=c++17", "-D__host__=", "-D__device__=", "-I", csrc, str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_only_the_counters_of_a_workspace_are_cleared(recorder, monkeypatch):
    """The partial sums (22 MB for one row of 5120 x 17408) are written before they are read."""
    sizes = []
    recorder.w12_gemm_workspace_init = lambda p, n, s: sizes.append(n) or 0
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **{**k, "device": "cpu"}))
    ws = w12.gemm_e4m3_workspace(1, 5120, 17408)
    assert ws.numel() == w12.gemm_e4m3_workspace_size(1, 5120, 17408) > 1 << 20
    assert sizes == [w12.gemm_plan(16, 5120, 17408)["counter_bytes"]]


SHAPES = [(32768, 4096), (5120, 17408), (34816, 5120), (5120, 5120), (65536, 2048), (256, 65536), (130, 127), (8192, 28672)]


@pytest.mark.parametrize("n,k", SHAPES)
def test_a_workspace_for_many_rows_serves_fewer(n, k):
    """The size never falls as rows are added, and a call of any number of rows accepts a workspace that was sized for
    more (the call's own check comes before any launch: a misaligned workspace is its next complaint)."""
    rows = sorted({1, 2, 4, 5, 8, 32, 63, 64, 65, 100, 128, 129, 256, 257, 384, 512, 513, 1000, 1024, 2048, 2500, 4095, 4096})
    sizes = [w12.gemm_e4m3_workspace_size(m, n, k) for m in rows]
    assert sizes == sorted(sizes)
    for m in rows:
        assert gemm(M=m, N=n, K=k, ldx=k + 15 & ~15, ldw=k + 15 & ~15, ldxs=1024, ldws=1024, ldy=n, ws=0x100008,
                    ws_bytes=sizes[-1]) == -5


def test_gemm_e4m3_refuses_a_workspace_that_is_too_small():
    need = w12.gemm_e4m3_workspace_size(3, 256, 4096)
    assert need > 16384
    call = dict(M=3, N=256, K=4096, ldx=4096, ldw=4096, ldxs=32, ldws=32, ldy=256)
    assert gemm(**call, ws_bytes=16384) == -3 and gemm(**call, ws=None) == -1
