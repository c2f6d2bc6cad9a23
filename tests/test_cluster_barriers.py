"""Cluster barriers in their .aligned form are undefined where a warp's threads
do not reach them together.  Nothing shows that from outside, so the sources
are held to one pair of helpers, which bring the warp together first."""
import glob
import os
import re

import pytest

from int4_weight_only_gptq_b200.build import CSRC

SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_aligned_cluster_barriers_follow_a_warp_barrier(path):
    lines = [ln.strip() for ln in open(path) if ln.strip()]
    for i, line in enumerate(lines):
        if re.search(r"barrier\.cluster\.\S*\.aligned", line):
            assert lines[i - 1] == "__syncwarp();", f"{os.path.basename(path)}: {line}"
