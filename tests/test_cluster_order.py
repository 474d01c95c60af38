"""Kernels that write another CTA's shared memory wait for the cluster first (read from the sources: nothing but luck
tells on a GPU)."""
import glob
import os
import re

import token_level_sparse_gb300 as T

CSRC = os.path.join(os.path.dirname(os.path.abspath(T.__file__)), "csrc")


def test_shared_memory_of_other_ctas_is_touched_behind_a_cluster_barrier():
    """A CTA's shared memory is defined for its cluster once it is known to run: the first access of a kernel to
    another's stands behind a barrier of the cluster that every thread waits at."""
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for body in text.split("__global__")[1:]:
            first = re.search(r"map_shared_rank|\bmapa\b", body)
            if not first:
                continue
            seen += 1
            before = body[:first.start()]
            assert re.search(r"cluster\.sync\(\)|cluster\.barrier_wait\(|barrier\.cluster\.wait", before), os.path.basename(path)
            assert before.count("cluster.barrier_arrive(") == before.count("cluster.barrier_wait("), os.path.basename(path)
    assert seen >= 1
