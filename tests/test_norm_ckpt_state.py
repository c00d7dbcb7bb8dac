"""Host-side checks of the norm and checkpoint calls' bookkeeping (CPU)."""

import contextlib
import os
import subprocess

import pytest
import torch

import __graft_entry__


@pytest.fixture(scope="module")
def clp():
    __graft_entry__.build()
    import chunked_log_prob_gb300 as m

    return m


def test_lose_copy_refuses_what_is_no_index(clp):
    for bad in (-2, 1 << 30, 1 << 40):
        with pytest.raises(clp.GrpoError) as e:
            clp.grpo_selftest_lose_copy(bad)
        assert e.value.code == -1
    clp.grpo_selftest_lose_copy(5)
    clp.grpo_selftest_lose_copy(-1)  # takes it back


class FakeCuda:
    """One thread's current device, and streams numbered 1000 + device."""

    def __init__(self, clp, monkeypatch, current):
        self.current, self.calls = current, []
        monkeypatch.setattr(clp._binding, "_current_device", lambda: self.current)
        monkeypatch.setattr(clp._binding, "_raw_stream", lambda index: 1000 + index)
        monkeypatch.setattr(torch.cuda, "device", self.guard)

    @contextlib.contextmanager
    def guard(self, device):
        before, self.current = self.current, torch.device(device).index
        try:
            yield
        finally:
            self.current = before

    def fn(self, *args):
        self.calls.append((self.current, args))
        return -5


@pytest.mark.parametrize("current", [0, 1, 3])
def test_calls_run_on_the_tensors_device(clp, monkeypatch, current):
    fake = FakeCuda(clp, monkeypatch, current)
    assert clp._binding.call_on(torch.device("cuda", 1), fake.fn, 7, None) == -5
    assert fake.calls == [(1, (7, None, 1001))]
    assert fake.current == current  # the caller's device is back


def test_calls_leave_the_device_as_it_was_after_an_error(clp, monkeypatch):
    fake = FakeCuda(clp, monkeypatch, 0)

    def broken(*args):
        raise RuntimeError

    with pytest.raises(RuntimeError):
        clp._binding.call_on(torch.device("cuda", 2), broken)
    assert fake.current == 0


def test_calls_refuse_the_cpu(clp):
    with pytest.raises(ValueError):
        clp._binding.call_on(torch.device("cpu"), None)


def _every_call(clp):
    bf = torch.bfloat16
    h, w = torch.zeros(8, 256, dtype=bf), torch.zeros(512, 256, dtype=bf)
    ids, row = torch.zeros(8, dtype=torch.int32), torch.zeros(8)
    ws = torch.zeros(1 << 12, dtype=torch.uint8)
    c = clp.alloc_ckpt(8, 256)
    return {
        "grpo_logp_fwd": lambda: clp.grpo_logp_fwd(h, w, ids),
        "grpo_loss_fwd_bwd": lambda: clp.grpo_loss_fwd_bwd(h, w, ids, None, row, row, row, 1),
        "grpo_logp_fwd_noalloc": lambda: clp.grpo_logp_fwd_noalloc(h, w, ids, row),
        "grpo_read_device_status": lambda: clp.grpo_read_device_status(ws),
        "grpo_norm_fwd": lambda: clp.grpo_norm_fwd(h),
        "grpo_norm_bwd": lambda: clp.grpo_norm_bwd(h, h, None, None, row),
        "grpo_ckpt_pack": lambda: clp.grpo_ckpt_pack(h),
        "grpo_ckpt_unpack": lambda: clp.grpo_ckpt_unpack(c),
        "grpo_ckpt_wgrad": lambda: clp.grpo_ckpt_wgrad(h, c),
    }


def test_every_launching_call_goes_to_the_tensors_device(clp, monkeypatch):
    # The library launches where it finds itself: no call may reach it otherwise.
    seen = []

    def record(device, fn, *args):
        seen.append((device.type, fn.__name__))
        return 0

    monkeypatch.setattr(clp._binding, "call_on", record)
    monkeypatch.setattr(clp._norm_ckpt, "call_on", record)
    for name, call in _every_call(clp).items():
        call()
        assert seen.pop() == ("cpu", name)
        assert not seen


CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "chunked_log_prob_gb300", "csrc")


def run_cpp(tmp_path, source):
    """Compiles and runs a program of the host headers; fails on a nonzero exit."""
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", CSRC,
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_what_is_kept_of_a_kernel_holds_for_its_device_only(tmp_path):
    run_cpp(tmp_path, r"""
#include <cstdio>
#include <thread>
#include "kernel_fit.h"
using grpo::KernelFit;
#define NEED(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
  static KernelFit f;
  int n = -1;
  NEED(!f.opted_in(0) && !f.find(0, 512, 65536, &n));
  f.set_opted_in(0);
  f.keep(0, 512, 65536, 3);
  NEED(f.opted_in(0) && f.find(0, 512, 65536, &n) && n == 3);
  // Another device: neither the opt-in nor the answer.
  NEED(!f.opted_in(1) && !f.find(1, 512, 65536, &n));
  f.keep(1, 512, 65536, 2);
  NEED(f.find(0, 512, 65536, &n) && n == 3);
  NEED(f.find(1, 512, 65536, &n) && n == 2);
  NEED(!f.opted_in(1));
  // Another shape of the launch.
  NEED(!f.find(0, 256, 65536, &n) && !f.find(0, 512, 65552, &n));
  f.keep(0, 1024, 232448, 0);
  NEED(f.find(0, 1024, 232448, &n) && n == 0 && !f.find(0, 512, 65536, &n));
  // Devices out of range keep nothing; a count too large for its byte neither.
  f.keep(-1, 512, 65536, 3);
  f.keep(grpo::kMaxDevices, 512, 65536, 3);
  f.set_opted_in(grpo::kMaxDevices);
  f.keep(2, 512, 65536, 256);
  NEED(!f.find(-1, 512, 65536, &n) && !f.find(grpo::kMaxDevices, 512, 65536, &n));
  NEED(!f.opted_in(grpo::kMaxDevices) && !f.find(2, 512, 65536, &n));
  // Threads that keep different shapes: what is found belongs to its shape.
  int wrong[4] = {};
  std::thread t[4];
  for (int k = 0; k < 4; ++k)
    t[k] = std::thread([&, k] {
      for (int i = 0; i < 200000; ++i) {
        const int threads = 32 * (1 + (i + k) % 5);
        int got = 0;
        f.keep(3, threads, 1024, threads / 32);
        if (f.find(3, 32 * (1 + i % 5), 1024, &got) && got != 1 + i % 5) ++wrong[k];
      }
    });
  for (auto& x : t) x.join();
  NEED(wrong[0] + wrong[1] + wrong[2] + wrong[3] == 0);
  return 0;
}
""")


def test_wgrad_work_is_dealt_once_on_any_number_of_pairs(tmp_path):
    # Every stage of every tile is some pair's, once; the pieces of a cut tile lie
    # in their own partial tiles of the workspace, where the join looks for them.
    out = run_cpp(tmp_path, r"""
#include <cstdio>
#include <random>
#include <set>
#include <vector>
#include "wgrad_plan.h"
using namespace grpo;
static int check(long long n, int out, int in, int pairs, int& cuts) {
  const WgradPlan p = make_plan(n, out, in, pairs);
  const int tiles = p.n_m * p.n_n, grid = launch_pairs(p, pairs);
  if (p.whole + p.cut != tiles || grid < 1 || grid > pairs) return 1;
  cuts += p.cut > 0;
  std::vector<std::vector<int>> seen(tiles, std::vector<int>(p.kt, 0));
  std::vector<std::set<int>> slots(tiles);
  std::set<int> used;
  for (int q = 0; q < grid; ++q) {
    WgradWork w;
    WgradItem it;
    while (w.next(p, q, grid, it)) {
      if (it.tile < 0 || it.tile >= tiles || it.kb < 0 || it.kb >= it.ke || it.ke > p.kt) return 2;
      for (int k = it.kb; k < it.ke; ++k) seen[it.tile][k]++;
      if (it.slot < 0) {
        if (it.kb != 0 || it.ke != p.kt) return 3;
      } else {
        if (it.tile < p.whole || !used.insert(it.slot).second) return 4;
        if (static_cast<size_t>(it.slot) >= partial_tiles(n, out, in)) return 5;
        slots[it.tile].insert(it.slot);
      }
    }
  }
  std::set<long long> places;
  for (int t = 0; t < tiles; ++t) {
    for (int c : seen[t])
      if (c != 1) return 6;
    int m, nn;
    tile_place(p, t, m, nn);
    if (m < 0 || m >= p.n_m || nn < 0 || nn >= p.n_n) return 7;
    if (!places.insert(static_cast<long long>(m) * p.n_n + nn).second) return 8;
  }
  for (int t = 0; t < p.cut; ++t) {
    std::set<int> joined;
    for (int q = first_piece(p, t); q <= last_piece(p, t); ++q) joined.insert(piece_slot(p, t, q));
    if (joined != slots[p.whole + t] || joined.size() < 2) return 9;
  }
  return 0;
}
int main() {
  std::mt19937 r(1);
  auto log_int = [&](int bits) { return 1 + static_cast<int>(r() >> (32 - 1 - r() % bits)); };
  int cuts = 0, cases = 0;
  for (int pairs : {1, 2, 3, 16, 37, 64, 66, 70, 74, 75, 76})
    for (int k = 0; k < 300; ++k, ++cases) {
      const long long n = log_int(17);
      const int out = log_int(13), in = log_int(13);
      const int e = check(n, out, in, pairs, cuts);
      if (e) {
        std::printf("%d: n %lld out %d in %d pairs %d\n", e, n, out, in, pairs);
        return 1;
      }
    }
  std::printf("%d %d\n", cases, cuts);
  return cuts > cases / 20 ? 0 : 2;
}
""")
    assert out.split()[0] == "3300"
