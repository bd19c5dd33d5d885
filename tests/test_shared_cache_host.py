"""runtime.BatchCache on the host: what it allocates where, and what it refuses; the cluster that eviction
launches (no GPU)."""
import contextlib
import os
import shutil
import subprocess
import types

import numpy as np
import pytest

from sparse_paged_kv_gb300 import binding as B
from sparse_paged_kv_gb300 import build_lib, runtime


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.load_library(build_lib.build())


def cache(batch=2, max_pages=4, prefix=2, **kw):
    """A cache in host memory, `prefix` pages shared by all of its sequences."""
    table = np.arange(batch * max_pages).reshape(batch, max_pages)
    table[:, :prefix] = table[0, :prefix]
    cfg = B.LocksConfig(batch=batch, n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=64, rank=8, max_pages=max_pages,
                        num_blocks=batch * max_pages)
    return runtime.BatchCache(cfg, table, [0, batch], [prefix], device="cpu", **kw)


class Recorder:
    """torch for one cache: notes the stream on which each allocation is made."""

    def __init__(self, torch):
        self.torch, self.current, self.made = torch, None, []
        self.cuda = types.SimpleNamespace(stream=self._stream, ExternalStream=lambda x: ("external", x),
                                          default_stream=lambda: "default")

    @contextlib.contextmanager
    def _stream(self, stream):
        before, self.current = self.current, stream
        yield
        self.current = before

    def _note(self, make, *a, **kw):
        self.made.append(self.current)
        return make(*a, **kw)

    def empty(self, *a, **kw):
        return self._note(self.torch.empty, *a, **kw)

    def empty_like(self, *a, **kw):
        return self._note(self.torch.empty_like, *a, **kw)

    def __getattr__(self, name):
        return getattr(self.torch, name)


@pytest.mark.parametrize("stream,on", [(None, None), ("side", "side"), (7, ("external", 7)), (0, "default")])
def test_results_are_allocated_on_the_stream_of_the_call(monkeypatch, stream, on):
    import torch
    calls = []
    for name in ("locks_prefix_decode", "locks_weigh", "locks_evict"):
        monkeypatch.setattr(B, name, lambda *a, _n=name, **kw: calls.append((_n, kw["stream"])))
    c = cache(budget_tokens=64, recent_tokens=8, max_rows=4)
    c.torch = rec = Recorder(torch)
    c.observe(torch.zeros(2, 4, 8, 128, dtype=torch.bfloat16), stream=stream)
    assert rec.made == [on, on]
    assert calls == [(n, stream) for n in ("locks_prefix_decode", "locks_weigh", "locks_evict")]
    c.attend(torch.zeros(2, 8, 128, dtype=torch.bfloat16), stream=stream)
    assert rec.made == [on, on]                       # (one row: the cache's own buffers)


def test_a_budget_leaves_room_for_a_token():
    for kw in (dict(budget_tokens=128), dict(budget_tokens=200), dict(budget_tokens=64, fixed=[128, 192])):
        with pytest.raises(ValueError, match="budget_tokens"):
            cache(**kw)                               # 256 slots a sequence, 128 of them its prefix
    for kw in (dict(budget_tokens=127), dict(budget_tokens=63, fixed=[128, 192]), dict(fixed=[128, 256]),
               dict(budget_tokens=127, fixed=[128, 256]), dict(budget_tokens=127, fixed=[1 << 30, 128])):
        cache(**kw)                                   # (a sequence that is fixed whole is never cut)


def test_a_bool_for_each_sequence_is_expected():
    import torch
    with pytest.raises(ValueError, match="sequences"):
        cache(budget_tokens=64).observe(torch.zeros(2, 8, 128, dtype=torch.bfloat16), sequences=[True])


def test_positions_before_anything_is_observed():
    c = cache(budget_tokens=64)
    table = c.block_table.numpy()
    for b in range(2):
        assert (c.positions.numpy()[table[b]] == np.arange(256).reshape(4, 1, 64)).all()
    assert c.positions.shape == (8, 2, 64) and c.positions.is_contiguous()
    cfg = B.LocksConfig(batch=1, n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=64, rank=8, max_pages=3, num_blocks=4)
    c = runtime.BatchCache(cfg, [[3, -1, 9]], budget_tokens=64, device="cpu")         # pages without a block yet
    assert (c.positions.numpy()[3] == np.arange(64)).all() and (c.positions.numpy()[:3] == 0).all()


RULE = r"""
#include <cstdio>
#include <cstdlib>
#include "locks_batch.h"
// units, slots and what fits, for 1 to 16 blocks -> the blocks of a cluster
int main(int, char** a) {
  int fit[17] = {0};
  for (int c = 1; c <= 16; ++c) fit[c] = std::atoi(a[2 + c]);
  std::printf("%d", locks::evict_blocks(std::atoi(a[1]), std::atoll(a[2]), fit));
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("needs a C++ compiler")
    at = tmp_path_factory.mktemp("rule")
    (at / "rule.cpp").write_text(RULE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build_lib.nvcc()))), "include")
    subprocess.run([cxx, "-std=c++17", "-I" + build_lib.CSRC, "-I" + cuda, "-o", str(at / "rule"), str(at / "rule.cpp")],
                   check=True)

    def run(units, slots, fit):
        return int(subprocess.run([str(at / "rule"), str(units), str(slots), *map(str, fit)], check=True,
                                  capture_output=True, text=True).stdout)
    return run


def test_eviction_launches_clusters_that_the_device_takes(rule):
    whole = [152 // c for c in range(1, 17)]
    small = [n if c <= 8 else 0 for c, n in enumerate(whole, 1)]      # clusters above 8 blocks are refused
    for slots in (100, 2047, 2048, 5000, 40000, 1 << 20):
        for units in (1, 2, 7, 8, 9, 10, 15, 19, 20, 38, 76, 77, 152, 153, 400):
            for fit in (whole, small):
                c = rule(units, slots, fit)
                assert c == 1 or (fit[c - 1] > 0 and slots // c >= 1024), (units, slots, c)
                assert units * c > 152 or c == 1 or fit[c - 1] >= units
    assert rule(10, 1 << 16, whole) == 16 and rule(10, 1 << 16, small) == 8
    assert rule(8, 1 << 17, [152 // c if c < 13 else 6 for c in range(1, 17)]) == 12
    assert rule(200, 1 << 17, whole) == 1 and rule(3, 2047, whole) == 1


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The queries and the pools of a call lie on the current device."""
    import torch
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    c = B.LocksConfig(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=64, rank=8, max_pages=4, num_blocks=8)

    class Tensor:
        is_cuda = True

        def __init__(self, device, dtype, *shape):
            self.device, self.dtype, self.shape = device, dtype, torch.Size(shape)
            self.nbytes = 1 << 30

        def __getattr__(self, name):
            return {"dim": lambda: len(self.shape), "get_device": lambda: self.device, "is_contiguous": lambda: True,
                    "data_ptr": lambda: 0x10000}[name]

    def call(fn, q=0, k=0):
        qs, pool = Tensor(q, torch.bfloat16, 2, 8, 128), Tensor(k, torch.bfloat16, 8, 2, 64, 128)
        ints, table = Tensor(0, torch.int32, 2), Tensor(0, torch.int32, 2, 4)
        rec, ws = Tensor(0, torch.float32, 8, 2, 64), Tensor(0, torch.uint8, 1 << 30)
        if fn is B.locks_prefix_decode:
            fn(c, qs, pool, pool, table, ints, None, None, qs, ws)
        elif fn is B.locks_weigh:
            fn(c, qs, Tensor(0, torch.float32, 2, 8), pool, table, ints, None, rec)
        else:
            fn(c, 64, 0, pool, pool, table, ints, rec, Tensor(0, torch.int32, 8, 2, 64), ints, ws)

    for fn, where in ((B.locks_prefix_decode, "q"), (B.locks_prefix_decode, "k"), (B.locks_weigh, "q"),
                      (B.locks_weigh, "k"), (B.locks_evict, "k")):
        with pytest.raises(ValueError, match="current device"):
            call(fn, **{where: 1})
