"""CPU check of how the producers of the windowed attention wait for their copies before a
block exits, also when another warp has given up: the library's own function, on barriers
that count their phases as the hardware's do."""

import re

import pytest

from block_sparse_local_nb_b200.build import CSRC
from tests.host_util import run_host_program

PROGRAM = r"""
#include <stdio.h>
#include "serving.cuh"

template <int N>
int check() {
  int bad = 0;
  for (int issued = 0; issued <= 5 * N + 1; ++issued)
    for (int landed = 0; landed <= issued; ++landed) {  // the first `landed` copies are there
      const int i = issued % N;
      const uint32_t ph = static_cast<uint32_t>(issued / N) & 1u;
      int phases[N] = {}, flying[N] = {}, waited[N] = {};
      bool possible = true;  // a stage is refilled only when its copy before has landed
      for (int j = 0; j < issued; ++j) {
        if (j < landed) ++phases[j % N];
        else if (flying[j % N]++) possible = false;
      }
      if (!possible) continue;
      nb::sm100::drain_ring<N>(i, ph, [&](int s, uint32_t parity) {
        // a wait for the parity of the phase that runs blocks until it is complete
        const bool blocks = (static_cast<uint32_t>(phases[s]) & 1u) == parity;
        if (s < 0 || s >= N || blocks != (flying[s] == 1)) ++bad;
        waited[s] = 1;
      });
      for (int s = 0; s < N; ++s) bad += !waited[s];
    }
  return bad;
}
int main() { printf("%d %d %d %d\n", check<1>(), check<2>(), check<3>(), check<6>()); }
"""


def test_every_copy_in_flight_is_waited_for_and_no_other(tmp_path):
    assert run_host_program(tmp_path, PROGRAM).split() == ["0", "0", "0", "0"]


@pytest.mark.parametrize("file,role", [
    ("attn_sink_fwd.cu", "producer"), ("attn_sink_fwd.cu", "v_producer"),
    ("attn_sink_bwd.cu", "producer"), ("attn_sink_bwd.cu", "y_producer")])
def test_a_producer_ends_nowhere_without_it(file, role):
    with open(f"{CSRC}/{file}") as f:
        text = f.read()
    body = text[re.search(r"__device__ int %s\(" % role, text).start():]
    body = body[:body.index("\n}\n")]
    # the role's returns stand in run(); behind it there is one way out, through the drain
    at = body.index("const int err = run();")
    assert len(re.findall(r"\breturn\b", body[at:])) == 1 and "drain_ring" in body[at:]
    assert body.index("auto run = [&]() -> int {") < body.index("return kErr")
