"""The rings of the integer products with the weights on the tensor core's lanes (no GPU): no warp reads a slot
before its copy has landed, and every schedule ends. The order of the waits is the kernel's own, from its header."""

import ctypes
import os
import subprocess

import pytest

from moe_decode_layer_gb300 import _lib, build
from tests import fake_cuda

# The kernel's warps over barriers that are waited for by parity. One event (a copy, a warp's step, an instruction)
# is held back until nothing else can go on; then all go on to the end. `only_full`: without the wait for the tensor core.
MODEL = r"""
#include <vector>
#include "rings.h"
using moe::rows::Ring;
using namespace moe::dense;

struct Barrier {
  int count = 1, pending = 1, done = 0;
  bool passes(unsigned parity) const { return (unsigned)(done & 1) != parity; }
  void arrive() { if (--pending == 0) done++, pending = count; }
};
enum Event { WEIGHTS, ROWS, WARP_READS, WARP_WRITES, ISSUE, COMPLETE };

extern "C" int run(int slots, int stages, int n, int held, int held_at, int held_warp, int only_full, int* finished) {
  std::vector<Barrier> full(slots), empty(slots), rows(slots), ready(stages), used(stages);
  for (Barrier& b : ready) b.count = b.pending = 4;
  std::vector<int> slot_has(slots, -1), rows_have(slots, -1), wide(4 * stages, -1);
  int wrong = 0;
  bool hold = true;
  auto may = [&](int e, int i, int w = 0) { return !(hold && e == held && i == held_at && (w == held_warp || e == WEIGHTS || e == ROWS || e >= ISSUE)); };
  struct Copy { int step, slot; };
  std::vector<Copy> weights, xs;
  int copied = 0, first = slots < n ? slots : n;
  Ring p_it;
  for (int i = 0; i < first; i++) weights.push_back({i, i});
  struct Warp { int i, group, q; bool read; Ring it, at; };
  std::vector<Warp> warps;
  for (int w = 0; w < 8; w++) warps.push_back({0, w >> 2, w & 3, false, Ring(), Ring()});
  int issued = 0, completed = 0;
  Ring m_it, m_at, c_it, c_at;
  auto go = [&]() {
    bool any = false;
    if (copied < n && (copied < first || empty[p_it.slot].passes(p_it.parity ^ 1))) {
      if (copied >= first) weights.push_back({copied, (int)p_it.slot});
      xs.push_back({copied++, (int)p_it.slot});
      p_it.next(slots);
      any = true;
    }
    for (size_t k = 0; k < weights.size();) {
      if (!may(WEIGHTS, weights[k].step)) { k++; continue; }
      slot_has[weights[k].slot] = weights[k].step;
      full[weights[k].slot].arrive();
      weights.erase(weights.begin() + k);
      any = true;
    }
    for (size_t k = 0; k < xs.size();) {
      if (!may(ROWS, xs[k].step)) { k++; continue; }
      rows_have[xs[k].slot] = xs[k].step;
      rows[xs[k].slot].arrive();
      xs.erase(xs.begin() + k);
      any = true;
    }
    for (size_t w = 0; w < warps.size(); w++) {
      Warp& a = warps[w];
      while (a.i < n && (a.i & 1) != a.group) a.i++, a.it.next(slots), a.at.next(stages);
      if (a.i >= n) continue;
      if (!a.read) {
        auto wait = [&](LaneWait what, unsigned s, unsigned parity) {
          return what == LANE_FULL ? full[s].passes(parity) : only_full || empty[s].passes(parity);
        };
        if (!may(WARP_READS, a.i, (int)w) || !landed(a.it, slots, stages, wait)) continue;
        wrong += slot_has[a.it.slot] != a.i;
        a.read = any = true;
      } else if (may(WARP_WRITES, a.i, (int)w) && used[a.at.slot].passes(a.at.parity ^ 1)) {
        if (completed < a.i - stages + 1) wrong++;  // over what the tensor core still reads
        wide[4 * a.at.slot + a.q] = a.i;
        ready[a.at.slot].arrive();
        a.i++, a.it.next(slots), a.at.next(stages), a.read = false;
        any = true;
      }
    }
    if (issued < n && may(ISSUE, issued) && ready[m_at.slot].passes(m_at.parity) && rows[m_it.slot].passes(m_it.parity)) {
      for (int q = 0; q < 4; q++) wrong += wide[4 * m_at.slot + q] != issued;
      wrong += rows_have[m_it.slot] != issued;
      issued++, m_it.next(slots), m_at.next(stages);
      any = true;
    }
    if (completed < issued && may(COMPLETE, completed)) {
      completed++;
      empty[c_it.slot].arrive();
      used[c_at.slot].arrive();
      c_it.next(slots), c_at.next(stages);
      any = true;
    }
    return any;
  };
  while (go()) {
  }
  hold = false;
  while (go()) {
  }
  *finished = completed == n;
  return wrong;
}

// Every event held back in turn; how many runs read or wrote too early, and how many did not end.
extern "C" void all(int slots, int stages, int n, int only_full, int* early, int* stuck) {
  *early = *stuck = 0;
  for (int e = WEIGHTS; e <= COMPLETE; e++)
    for (int i = 0; i < n; i++)
      for (int w = 0; w < (e == WARP_READS || e == WARP_WRITES ? 8 : 1); w++) {
        int ended;
        *early += run(slots, stages, n, e, i, w, only_full, &ended) != 0;
        *stuck += !ended;
      }
}
"""

BEHIND = r"""
#include "rings.h"
extern "C" int behind(int stages, int group) { return moe::dense::behind_at(stages, group); }
"""

# a launch of lanes_kernel leaves its parameters' first words
KEPT = "cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {\n" \
       "  if (g_names[f].find(\"lanes_kernel\") != std::string::npos) memcpy(g_lanes, args[0], sizeof(g_lanes));"


def _compiled(folder, text):
    src, out = os.path.join(folder, "model.cpp"), os.path.join(folder, "librings.so")
    with open(src, "w") as f:
        f.write(text)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-O2", "-w", "-I", cuda, "-I", build.CSRC, src, "-o", out], check=True)
    return ctypes.CDLL(out)


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    lib = _compiled(str(tmp_path_factory.mktemp("rings")), MODEL)

    def run(slots, stages, n, only_full=False):
        early, stuck = ctypes.c_int(), ctypes.c_int()
        lib.all(slots, stages, n, int(only_full), ctypes.byref(early), ctypes.byref(stuck))
        return early.value, stuck.value
    return run


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    stub = fake_cuda.STUB
    try:
        head = "cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {"
        fake_cuda.STUB = stub.replace(head, KEPT).replace("int g_capturing = 0;", "int g_capturing = 0, g_lanes[11];") \
            .replace("int fake_bad_maps()", "int fake_lanes(int i) { return g_lanes[i]; }\nint fake_bad_maps()")
        assert fake_cuda.STUB.count("g_lanes") == 4
        return fake_cuda.make(str(tmp_path_factory.mktemp("fake")))
    finally:
        fake_cuda.STUB = stub


@pytest.mark.parametrize("slots", range(2, 13))
def test_no_slot_is_read_before_its_copy_has_landed(model, slots):
    for stages in range(2, 7):
        for n in (1, 2, slots, slots + 1, 3 * slots + 2, 3 * slots + 3):
            assert model(slots, stages, n) == (0, 0), (stages, n)


def test_the_model_sees_a_wait_that_passes_early(model):
    """Waits for the copies alone pass too early where the number of slots is odd and the stages do not hold the group back."""
    for slots in range(2, 13):
        for stages in (5, 6):
            early, _ = model(slots, stages, 3 * slots + 3, only_full=True)
            assert (early > 0) == (slots % 2 == 1 and slots < stages + 2), (slots, stages)


def test_launches_are_within_the_model(lib):
    """Slots and stages of every number of rows, widths with and without a split of K."""
    x, out, w, s, ws = (ctypes.c_void_p(i << 44) for i in range(1, 6))
    seen = set()
    for inner in (16, 2064, 16384):
        for outer in (8, 1032, 3000, 9728, 16000):
            for swiglu in (0, 1):
                cfg = _lib.Int8Config(inner, outer, swiglu, _lib.MOE_I8, 0)
                for rows in range(9, 193):
                    lib.fake_reset(-1, -1, 0)
                    assert lib.moe_decode_project_int8(cfg, w, s, x, s, inner, None, out, rows, ws, 1 << 40, None) == _lib.MOE_OK
                    if "lanes_kernel" not in lib.fake_name(lib.fake_launches() - 1).decode():
                        continue
                    got = [lib.fake_lanes(i) for i in range(11)]
                    assert got[:4] == [rows, inner, outer, swiglu]
                    split, slots, stages = got[5], got[6], got[9]
                    assert split in (1, 2, 4, 8) and 2 <= slots <= 12 and 2 <= stages <= 6
                    seen.add((slots, stages))
    assert {(3, 5), (5, 6), (7, 6)} <= seen  # the ones where the copies' barriers alone would not do


def test_each_group_waits_once_for_the_launch_before(tmp_path):
    """At a step of its own (the groups take steps in turn), or after its last one; odd numbers of stages too."""
    behind = _compiled(str(tmp_path), BEHIND).behind
    for stages in range(2, 7):
        for group in (0, 1):
            at = behind(stages, group)
            assert at >= stages
            for n in range(1, 40):
                assert sum(i == at for i in range(n) if i % 2 == group) + (n <= at) == 1, (stages, group, n)
