"""Distributed shared memory may be used only once every CTA of the cluster is known to run: in each
kernel a barrier of the cluster has been waited for before the first access to, or arrival in, another
CTA's shared memory (read from the sources; no GPU needed)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ternary_quantized_moe_b200", "csrc")
REMOTE = re.compile(r"st\.shared::cluster|\bst_async_f4\(|\bld_dsmem_\w+\(|\bmbar_arrive_remote\w*\(|\btma_load_2d_pair\(|"
                    r"\bumma_commit_pair\(")
JOINED = re.compile(r"\bcluster_sync\(\)|barrier\.cluster\.wait")


def kernels():
    """(file, name, body) of every __global__ function."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), open(path).read())
        for m in re.finditer(r"__global__[^;{]*?\b(\w+)\s*\((?:[^(){}]|\([^()]*\))*\)\s*\{", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            yield os.path.basename(path), m.group(1), text[m.end():i]


REMOTE_KERNELS = [(f, n, b) for f, n, b in kernels() if REMOTE.search(b)]


def test_kernels_are_found():
    names = {n for _, n, _ in REMOTE_KERNELS}
    assert {"xproj_kernel", "fp8_rows_kernel", "fp8_stream_kernel", "fp8_pair_kernel"} <= names


@pytest.mark.parametrize("file,name,body", REMOTE_KERNELS, ids=[n for _, n, _ in REMOTE_KERNELS])
def test_cluster_barrier_before_remote_shared_memory(file, name, body):
    joined = JOINED.search(body)
    assert joined and joined.start() < REMOTE.search(body).start()
