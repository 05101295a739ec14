"""CPU checks of host-compilable parts of the full-attention kernels: when a wait is given up."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WAIT = r"""
#include <stdio.h>
#include "gdn_wait.cuh"
// A wait that begins at 1000 and asks every `step`; something moves every `every` until `last`.
// Prints when it is given up, or -1 if not before `end`.
static long given_up(uint64_t limit, uint64_t step, uint64_t every, uint64_t last, uint64_t end) {
  uint64_t moved = 1000;
  for (uint64_t now = 1000; now < end; now += step) {
    while (moved + every <= now && moved + every <= last) moved += every;
    if (gdn::stands_still(now, moved, limit)) return (long)now;
  }
  return -1;
}
int main(void) {
  const uint64_t limit = 2000;
  printf("%ld\n", given_up(limit, 7, 1000, 900000, 900000));  // long, but it moves
  printf("%ld\n", given_up(limit, 7, 1, 0, 900000));          // never moves
  printf("%ld\n", given_up(limit, 7, 100, 50000, 900000));    // stops at 50000
  printf("%d\n", gdn::stands_still(5000, 5040, limit));       // moved after the time was read
  return 0;
}
"""


def test_a_wait_is_given_up_when_nothing_moves_not_when_it_is_long(tmp_path):
    src, exe = tmp_path / "wait.cpp", tmp_path / "wait"
    src.write_text(WAIT)
    csrc = os.path.join(ROOT, "chunked_state_scan_gated_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    out = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert out[0] == -1 and out[3] == 0
    assert 1000 + 2000 < out[1] <= 1000 + 2000 + 7
    assert 50000 + 2000 < out[2] <= 50000 + 2000 + 7


def test_no_wait_of_the_attention_kernels_is_bounded_by_its_own_length():
    """Waits may last as long as an item: each asks whether anything has moved."""
    with open(os.path.join(ROOT, "chunked_state_scan_gated_gb300", "csrc", "gdn_attn_tc.cuh")) as f:
        text = f.read()
    assert text.count("mbarrier.try_wait.parity") == 2  # arrived(), of one CTA or of a pair
    assert text.count("arrived<") == 2 and text.count("kWaitLimitNs &&") == 2
    assert text.count("stands_still(clock64(), alive.moved,") == 2
