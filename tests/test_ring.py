"""What a CTA waits for before it leaves (csrc/ring.h), compiled for the host against barriers that complete with time."""
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


def test_a_cta_waits_for_what_it_began(tmp_path):
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("name,rings", [("cache_attend_tile.cuh", ["k_full", "v_full", "k_empty", "s_full", "pv_done"]),
                                        ("cache_weights.cu", ["k_full", "k_empty", "s_full"])])
def test_every_ring_of_copies_and_products_is_waited_for(name, rings):
    """Each ring that a copy or a product completes is landed, and no wait takes either parity for an answer."""
    text = open(os.path.join(CSRC, name)).read()
    for ring in rings:
        assert f"ring_land(sm.{ring}," in text, ring
    assert "bar_try(" not in text
