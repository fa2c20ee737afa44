"""CPU check of how a decode warp that gives up on a page waits for the copies that it
still has in flight: the library's own function, on barriers that count their passes as
the hardware's do."""

import pytest

from tests.host_util import run_host_program

PROGRAM = r"""
#include <stdio.h>
#include "kv4.cuh"

// Stages 0..N-1: passes complete (the page has landed), and whether a copy is in flight.
template <int N>
int check() {
  int bad = 0;
  for (int count = 1; count <= 5 * N + 1; ++count)
    for (int i = 0; i < count; ++i) {  // the wait for page i gives up
      int passes[N] = {}, page[N];
      for (int s = 0; s < N; ++s) page[s] = -1;
      for (int j = 0; j < N && j < count; ++j) page[j] = j;
      for (int j = 0; j < i; ++j) {  // pages before i landed, were used, and refilled
        ++passes[j % N];
        page[j % N] = j + N < count ? j + N : -1;
      }
      bool waited[N] = {};
      nb::kv4::drain_pages<N>(i, count, [&](int s, uint32_t parity) {
        // a wait returns at once when the phase of that parity is complete
        const bool at_once = (static_cast<uint32_t>(passes[s]) & 1u) != parity;
        if (s < 0 || s >= N || page[s] < 0 || at_once || waited[s]) ++bad;
        waited[s] = true;
      });
      for (int s = 0; s < N; ++s)
        if (page[s] >= 0 && !waited[s]) ++bad;  // a copy that nobody waits for
    }
  return bad;
}
int main() { printf("%d %d %d\n", check<1>(), check<3>(), check<4>()); }
"""


def test_every_copy_in_flight_is_waited_for(tmp_path):
    assert run_host_program(tmp_path, PROGRAM).split() == ["0", "0", "0"]


@pytest.mark.parametrize("mistake", ["0u", "static_cast<uint32_t>(i) & 1u"])
def test_the_check_sees_a_wrong_parity(tmp_path, mistake):
    """The same check on a copy of the function that waits for another parity."""
    wrong = PROGRAM.replace('#include "kv4.cuh"', '#include "kv4.cuh"\n' + r"""
template <int N, class Wait>
void wrong(int i, int count, Wait&& wait) {
  for (int end = count - i < N ? count : i + N; i < end; ++i) wait(i % N, PARITY);
}
""".replace("PARITY", mistake)).replace("nb::kv4::drain_pages<N>(", "wrong<N>(")
    assert any(x != "0" for x in run_host_program(tmp_path, wrong).split()[1:])
