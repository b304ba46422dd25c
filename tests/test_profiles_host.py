"""The committed captures of DRAM traffic belong to the committed kernels: bench.py leaves the traffic out where a kernel's source
has changed since its capture (so a change of a kernel, or of what all kernels include, asks for new captures)."""
import glob
import os
import re

import pytest

import bench

CAPTURES = [os.path.basename(p)[:-3] for p in sorted(glob.glob(os.path.join(bench.ROOT, "profiles", "*.md")))
            if re.search(r"^source_digest:", open(p).read(), re.M)]


def test_there_are_captures():
    assert len(CAPTURES) >= 8


@pytest.mark.parametrize("name", CAPTURES)
def test_capture_belongs_to_the_source(name):
    kernel, workload = name.split(".", 1)
    traffic = bench.recorded_traffic(kernel, workload)
    assert traffic is not None and traffic > 0
