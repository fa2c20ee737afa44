"""CPU checks of what nb_kernel_error reports: every wait has a code of its own, no code
of a wait can be taken for a token that the cache skipped, and neither hides the other."""

import glob
import os
import re

from block_sparse_local_nb_b200.build import CSRC, ROOT
from tests.host_util import run_host_program


def public_codes():
    with open(os.path.join(ROOT, "include", "nb.h")) as f:
        return {n: int(v, 16) for n, v in re.findall(r"#define (NB_KERR_\w+) +(0x[0-9a-f]+)", f.read())}


def wait_sites():
    """(file, name, value) of every site code of the kernels."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for body in re.findall(r"enum : int \{([^}]*)\}", text):
            value = None
            for entry in body.split(","):
                name, _, given = (x.strip() for x in entry.partition("="))
                if given.startswith("NB_KERR"):  # a public code: not a wait
                    continue
                value = int(given, 16) if given else value + 1
                yield os.path.basename(path), name, value


def test_every_wait_has_a_code_of_its_own():
    seen = {}
    for file, name, value in wait_sites():
        assert 0 < value < public_codes()["NB_KERR_WAIT"]
        assert value not in seen, (file, name, seen[value])
        seen[value] = (file, name)
    assert len(seen) > 60


def test_waits_and_skipped_tokens_cannot_be_confused(tmp_path):
    codes = public_codes()
    assert all(not v & codes["NB_KERR_WAIT"] for n, v in codes.items() if n != "NB_KERR_WAIT")
    out = run_host_program(tmp_path, r"""
#include <stdio.h>
#include "serving.cuh"
int main() {
  const int words[4][2] = {{0, 0}, {0, NB_KERR_KV4_WRITE}, {0x51, 0}, {0x51, NB_KERR_KV4_DECODE}};
  for (auto& w : words) {
    const nb::KernelReport r = nb::kernel_report(w);
    printf("%d %d\n", r.code, r.word);
  }
}
""")
    got = [tuple(map(int, line.split())) for line in out.splitlines()]
    wait = codes["NB_KERR_WAIT"] | 0x51
    # a reset of the word that was reported leaves the other for the next call
    assert got == [(0, 1), (codes["NB_KERR_KV4_WRITE"], 1), (wait, 0), (wait, 0)]


def test_the_binding_has_the_public_codes():
    import block_sparse_local_nb_b200 as nb

    assert public_codes() and all(getattr(nb, n) == v for n, v in public_codes().items())
