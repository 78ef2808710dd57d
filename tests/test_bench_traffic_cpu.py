"""The sources that the DRAM traffic record is held to: those of the kernel it was taken of, and no other kernel's."""
import os
import re

import bench

CSRC = os.path.join(bench.ROOT, "paged_kv_decode_19_gb300", "csrc")


def _reached(name, seen):
    """The file and what it includes, of this library."""
    if name in seen or not os.path.exists(os.path.join(CSRC, name)):
        return seen
    seen.add(name)
    for inc in re.findall(r'#include "([^"]+)"', open(os.path.join(CSRC, name)).read()):
        _reached(inc, seen)
    return seen


def test_the_record_follows_the_sources_of_its_kernel_alone():
    need = set()
    for name in os.listdir(CSRC):
        if name.startswith("decode_mma") and name.endswith(".cu"):
            _reached(name, need)
    have = set(bench._traffic_sources())
    assert need <= have
    # beside them the host's plan, and what it includes without changing the launch
    assert have - need <= {"api.cu"}
