"""Index arithmetic of the cache kernels (csrc/ring.h) compiled for the host: what a CTA waits for before it leaves, against
barriers that complete with time, and walks over positions up to the longest context."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_verification_02_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "ring.h"

// A ring as the tensor memory accelerator or the tensor core completes it: phase f of a stage (counted from 0) completes at its own
// time, phases of a stage in order.  A parity test holds when the phase before the current one has that parity.
struct Ring {
  int stages, begun, slow, late;  // `late`: the stage whose last phase is `slow` tests late
  int now = 0;
  int phases(int s) const { return begun / stages + (s < begun % stages ? 1 : 0); }
  int completed(int s) const { return s == late && now < slow && phases(s) > 0 ? phases(s) - 1 : phases(s); }
  bool test(int s, int parity) {
    ++now;
    return (completed(s) & 1) != parity;
  }
  bool pending() const {
    for (int s = 0; s < stages; ++s)
      if (completed(s) < phases(s)) return true;
    return false;
  }
};

int main() {
  for (int stages = 1; stages <= 6; ++stages)
    for (int begun = 0; begun <= 4 * stages + 1; ++begun)
      for (int late = 0; late < stages; ++late)
        for (int k = 0; k < 5; ++k) {
          const int slow = k < 3 ? k : k == 3 ? 50 : 1000;
          Ring ring{stages, begun, slow, late};
          const bool ok = sv::ring_landed(stages, begun, 4096, [&](int s, int parity) { return ring.test(s, parity); });
          if (!ok || ring.pending()) return std::printf("left early: %d stages, %d begun, %d late by %d\n", stages, begun, late, slow), 1;
          // one that never completes is given up after its tests, and said so
          Ring stuck{stages, begun, 1 << 30, late};
          const bool said = sv::ring_landed(stages, begun, 64, [&](int s, int parity) { return stuck.test(s, parity); });
          if (said == stuck.pending() || stuck.now > 64 + stages) return std::printf("stuck: %d %d %d\n", stages, begun, late), 1;
        }
  return 0;
}
"""


SPANS = r"""
#include <cstdio>
#include "ring.h"

// Spans of 256 pages over the last positions that a table can hold: they meet, cover what is left, and end.
int main() {
  for (int page = 16; page <= 256; page *= 2) {
    const int step = 256 * page, most = (2147483647 - 256) / page * page;
    for (int k = 0; k < 6; ++k)
      for (int spans = 1; spans <= 3; ++spans) {
        const int less[6] = {0, 1, page, step - 1, step, step + 1}, to = most - less[k];
        int at = (most - spans * step) / page * page, rounds = 0;
        while (at < to) {
          const int next = sv::next_span(at, to, step);
          if (next <= at || next > to || next - at > step || ++rounds > 4) return std::printf("page %d: %d to %d\n", page, at, next), 1;
          at = next;
        }
        if (at < to) return 1;
      }
  }
  return 0;
}
"""


def run(tmp_path, program):
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(program)
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-Wall", "-Werror", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_a_cta_waits_for_what_it_began(tmp_path):
    run(tmp_path, PROGRAM)


def test_walks_end_at_the_longest_context(tmp_path):
    run(tmp_path, SPANS)


@pytest.mark.parametrize("name,rings", [("cache_attend_tile.cuh", ["k_full", "v_full", "k_empty", "s_full", "pv_done"]),
                                        ("cache_weights.cu", ["k_full", "k_empty", "s_full"])])
def test_every_ring_of_copies_and_products_is_waited_for(name, rings):
    """Each ring that a copy or a product completes is landed, and no wait takes either parity for an answer."""
    text = open(os.path.join(CSRC, name)).read()
    for ring in rings:
        assert f"ring_land(sm.{ring}," in text, ring
    assert "bar_try(" not in text


def test_a_weights_status_is_only_raised():
    """The CTAs that share a request set its status in any order: each by a maximum, of which the code of a wait that ran out is the largest."""
    text = open(os.path.join(CSRC, "cache_weights.cu")).read()
    kernel = text[text.index("cache_weights_tile_kernel(const"):text.index("cudaError_t launch_weight_tiles")]
    assert kernel.count("P.status[") == kernel.count("atomicMax(&P.status[") == 3
