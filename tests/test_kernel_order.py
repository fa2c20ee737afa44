"""Kernels are launched so that they may begin while the kernel before them on the
stream still runs; what that one (and those before it) wrote is promised to be visible
only behind griddepcontrol.wait.  So a kernel waits without a condition, and before
everything else that touches global memory.  Read from the sources; no GPU."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_sparse_local_nb_b200", "csrc")
# launched in plain stream order: it starts when everything before it is complete
PLAIN = {"attn_fwd_f32_kernel"}


def kernels():
    """(file, name, body without comments) of every kernel."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\(", text):
            start = text.index("{", m.end())
            depth, at = 1, start + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            yield os.path.basename(path), m.group(1), text[start + 1:at - 1]


KERNELS = list(kernels())


def test_kernels_are_found():
    names = {name for _, name, _ in KERNELS}
    assert {"attn_sink_bwd_kernel", "sink_rows_kernel", "kv4_decode_kernel",
            "attn_fwd_tc_kernel"} <= names


@pytest.mark.parametrize("file,name,body", KERNELS, ids=[k[1] for k in KERNELS])
def test_a_kernel_waits_for_what_came_before_it(file, name, body):
    if name in PLAIN:
        assert "pdl_" not in body
        return
    # a statement of the body itself: two spaces in, nothing before it on its line
    wait = re.search(r"^  pdl_wait\(\);", body, re.M)
    assert wait, f"{file}: {name} does not wait in every thread"
    before = body[:wait.start()]
    # before it: shared memory, barriers, tensor memory and descriptors in the parameters
    for word in ("length_of", "lengths", "build_table", "sched_build", "__ldcg", "atomic",
                 "bulk_load", "tma_load", "producer", "p.q", "p.taken"):
        assert word not in before, f"{file}: {name} has {word} before it waits"
