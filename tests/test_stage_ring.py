"""The staging ring of the 4-bit tile kernel, as its kernel computes it (csrc/pa_stage_ring.h), in a model of
its barriers that walks every order in which copies land and warps run: no reader may take a slot before its
own copy is there or find another one in it, and nothing may wait for ever.  Host code only."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_gqa_attn_gb300", "csrc")

MODEL = r"""
#include <cstdio>
#include <set>
#include <vector>

#include "pa_stage_ring.h"

// The same ring with one landed-barrier per slot: what the model has to find wrong.
struct PerSlot : pa::StageRing {
  static constexpr int kFullBars = kSlots;
  static int full_bar(int u) { return u % kSlots; }
  static unsigned full_parity(int u) { return (unsigned)(u / kSlots) & 1u; }
};

constexpr int kSteps = 9, kUses = 2 * kSteps;

// A barrier that one arrival (and its copy's bytes) completes is its number of completed phases; a wait for
// parity P passes when the phase that completed last has that parity (a new barrier: parity 1 passes).
template <class Ring>
struct State {
  int filled = 0;                  // uses copied so far
  unsigned landed = 0;             // bit per use
  int step[2] = {0, 0};            // next step of the K and of the V reader
  bool reading[2] = {false, false};
  int full[8] = {}, empty[8] = {};
  int slot[8] = {-1, -1, -1, -1, -1, -1, -1, -1};  // use that was copied into the slot last
  std::vector<int> key() const {
    std::vector<int> k = {filled, (int)landed, step[0], step[1], reading[0], reading[1]};
    for (int i = 0; i < 8; ++i) { k.push_back(full[i]); k.push_back(empty[i]); k.push_back(slot[i]); }
    return k;
  }
};

inline bool passes(int completed, unsigned parity) { return ((unsigned)(completed - 1) & 1u) == parity; }

template <class Ring>
const char* walk(long* states) {
  std::set<std::vector<int>> seen;
  std::vector<State<Ring>> todo = {State<Ring>()};
  seen.insert(todo[0].key());
  while (!todo.empty()) {
    const State<Ring> s = todo.back();
    todo.pop_back();
    std::vector<State<Ring>> next;
    // the producer starts the next copy
    if (s.filled < kUses) {
      const int u = s.filled;
      if (u < Ring::kSlots || passes(s.empty[Ring::empty_bar(u)], Ring::empty_parity(u))) {
        if (s.slot[Ring::slot(u)] >= 0 && !((s.landed >> s.slot[Ring::slot(u)]) & 1u)) return "copied over a copy in flight";
        State<Ring> n = s;
        n.slot[Ring::slot(u)] = u;
        ++n.filled;
        next.push_back(n);
      }
    }
    // any copy in flight lands
    for (int u = 0; u < s.filled; ++u)
      if (!((s.landed >> u) & 1u)) {
        State<Ring> n = s;
        n.landed |= 1u << u;
        ++n.full[Ring::full_bar(u)];
        next.push_back(n);
      }
    // a reader passes its wait, or gives its slot back
    for (int r = 0; r < 2; ++r) {
      if (s.step[r] == kSteps) continue;
      const int u = Ring::use(s.step[r], r == 1);
      State<Ring> n = s;
      if (!s.reading[r]) {
        if (!passes(s.full[Ring::full_bar(u)], Ring::full_parity(u))) continue;
        if (u >= s.filled || !((s.landed >> u) & 1u)) return "read before its copy landed";
        n.reading[r] = true;
      } else {
        n.reading[r] = false;
        ++n.step[r];
        ++n.empty[Ring::empty_bar(u)];
      }
      if (s.slot[Ring::slot(u)] != u) return "read another copy";
      next.push_back(n);
    }
    if (next.empty() && !(s.filled == kUses && s.step[0] == kSteps && s.step[1] == kSteps)) return "waits for ever";
    for (const auto& n : next)
      if (seen.insert(n.key()).second) todo.push_back(n);
  }
  *states = (long)seen.size();
  return nullptr;
}

int main() {
  long states = 0, none = 0;
  const char* ring = walk<pa::StageRing>(&states);
  const char* control = walk<PerSlot>(&none);
  std::printf("%s|%s|%ld\n", ring ? ring : "sound", control ? control : "sound", states);
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_reader_gets_its_own_copy_in_every_order(tmp_path):
    src, exe = tmp_path / "ring.cc", tmp_path / "ring"
    src.write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, str(src), "-o", str(exe)], check=True, timeout=120)
    ring, control, states = subprocess.run([str(exe)], check=True, capture_output=True, text=True,
                                           timeout=120).stdout.strip().split("|")
    assert ring == "sound", ring
    assert control == "read before its copy landed", control  # the model sees the fault of a barrier per slot
    assert int(states) > 100
    # and the kernel takes its slots, barriers and parities from that header alone
    kernel = open(os.path.join(CSRC, "pa_prefill.cuh"), encoding="utf-8").read()
    waits = [line for line in kernel.splitlines() if "bar_raw_" in line and ("wait" in line or "arrive" in line)]
    assert len(waits) == 4 and all("StageRing::" in line for line in waits), waits
