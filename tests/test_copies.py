"""The bookkeeping of copies on their way (csrc/copies.cuh), compiled for the host and run
with waits that run out: whatever a stage's copy was sent for and no wait has seen arrive,
drain() waits for, at the phase that the copy completes.  The barriers are counters, with the
rule of mbarrier.try_wait.parity."""

import subprocess

from invariant_decode_attention_gb300 import build as B

PROGRAM = r"""
#include <cstdio>
#include <random>

#include "copies.cuh"

constexpr int kStages = 3;

struct Ring {
  int sent[kStages] = {}, done[kStages] = {};  // copies of each stage: issued, arrived
  // the phase of this parity has completed (done phases have)
  bool passed(int stage, uint32_t parity) const { return (done[stage] & 1) != (int)parity; }
};

#define CHECK(x) if (!(x)) { std::printf("round %d: %s\n", round, #x); return 1; }

int main() {
  std::mt19937 rng(1);
  int lost_rounds = 0;
  for (int round = 0; round < 20000; ++round) {
    Ring ring;
    da::Copies c;
    const int tiles = 1 + rng() % 20, late = rng() % 24;  // the wait that runs out, if there are so many
    int next = 0;
    bool boxed[64];
    auto send = [&]() {
      if (next >= tiles || c.lost) return;
      const int stage = next % kStages;
      boxed[next] = rng() % 4 != 0;  // the others go another way
      if (boxed[next]) ++ring.sent[stage], c.sent(stage);
      ++next;
    };
    for (int i = 0; i < kStages - 1; ++i) send();
    for (int t = 0; t < tiles; ++t) {
      const int stage = t % kStages;
      const bool was_lost = c.lost;
      bool asked = false;
      c.wait(stage, [&](int s, uint32_t parity) {
        asked = true;
        if (s != stage || ring.passed(s, parity)) return true;  // (a wait that passes too early: seen below)
        if (t == late) return false;
        ++ring.done[s];
        return ring.passed(s, parity);
      });
      CHECK(asked == (!was_lost && t < next && boxed[t]));
      CHECK(c.lost == (was_lost || (asked && t == late)));
      if (!c.lost) CHECK(ring.done[stage] == ring.sent[stage]);
      send();
    }
    if (c.lost) {
      ++lost_rounds;
      // some that were on their way have arrived by themselves
      for (int s = 0; s < kStages; ++s)
        if (ring.done[s] < ring.sent[s] && rng() % 2) ++ring.done[s];
      int waited[kStages] = {};
      const da::Copies before = c;
      c.drain(kStages, [&](int s, uint32_t parity) {
        ++waited[s];
        if (!ring.passed(s, parity)) ++ring.done[s];
        return true;
      });
      CHECK(waited[late % kStages] == 1);  // the very copy whose wait ran out
      for (int s = 0; s < kStages; ++s) CHECK(ring.done[s] == ring.sent[s] && waited[s] == (int)(before.out >> s & 1));
    } else {
      CHECK(c.out == 0);
    }
  }
  std::printf("lost %d\n", lost_rounds);
  return lost_rounds > 1000 ? 0 : 1;
}
"""


def test_a_copy_whose_wait_ran_out_is_waited_for(tmp_path):
    source = tmp_path / "copies.cc"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", B.CSRC, str(source), "-o", str(tmp_path / "copies")],
                   check=True)
    r = subprocess.run([str(tmp_path / "copies")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
