"""Rings of barriers, compiled for the host: the places walked back from where a warp's copies end are those of its last
copies, which is what a launch that gives up waits for."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_logit_gb300", "csrc")
PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include "asv_ring.h"
// ring, first place, step, uses: the places used, then those walked back
int main(int, char** v) {
  const int n = atoi(v[1]), first = atoi(v[2]), by = atoi(v[3]), uses = atoi(v[4]);
  asv::Ring r;
  if (first) r.next(n);
  for (int i = 0; i < uses; ++i, r.next(n, by)) printf("%d %u\\n", r.slot, r.phase);
  for (int i = 0; i < (n + 1) / by && i < uses; ++i) {
    r.back(n, by);
    printf("%d %u\\n", r.slot, r.phase);
  }
}
"""


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    (d / "p.cpp").write_text(PROGRAM)
    subprocess.run([os.environ.get("CXX", "g++"), f"-I{CSRC}", str(d / "p.cpp"), "-o", str(d / "p")], check=True)

    def run(n, first, by, uses):
        text = subprocess.run([str(d / "p"), *map(str, (n, first, by, uses))], check=True, capture_output=True, text=True).stdout
        got = [tuple(map(int, line.split())) for line in text.splitlines()]
        return got[:uses], got[uses:]
    return run


@pytest.mark.parametrize("n,by", [(1, 1)] + [(n, by) for n in (2, 4, 5, 8, 10, 16) for by in (1, 2)])
def test_back_undoes_next(places, n, by):
    for first in (0, 1):
        for uses in range(0, 4 * n + 1):
            used, back = places(n, first if n > 1 else 0, by, uses)
            # the i-th use: its place in an endless row, and which time round
            assert used == [((first * (n > 1) + by * i) % n, (first * (n > 1) + by * i) // n % 2) for i in range(uses)]
            assert back == used[::-1][:(n + 1) // by]
