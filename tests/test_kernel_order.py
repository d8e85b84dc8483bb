"""CPU tier: the order of steps in the kernels' sources that keeps launches
from waiting for each other."""
import glob
import os
import re

import pytest

from rmsnorm_fwd_bwd_02_gb300 import build

FILES = sorted(f for d in build.SOURCE_DIRS for ext in ("*.cu", "*.cuh") for f in glob.glob(os.path.join(d, ext)))


def kernels(text):
    """(name, body) of the kernels defined in a source file, without comments."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\((?:[^()]|\([^()]*\))*\))*\)\s*)?(\w+)\s*\(",
                         text):
        at = text.find("{", m.end())
        depth, i = 1, at + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[at:i]


def test_every_kernel_is_seen():
    found = [name for f in FILES for name, _ in kernels(open(f).read())]
    assert len(found) == sum(len(re.findall(r"^__global__|\n__global__", open(f).read())) for f in FILES)
    assert "kv4_prompt" in found and "rms_fp8_gemm" in found


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(f) for f in FILES])
def test_tensor_memory_is_held_before_dependents_start(path):
    """A dependent launch may allocate tensor memory before it waits for this
    grid. Were it let in first, a CTA here that still has to allocate would
    wait for columns that are freed only after this grid: so the allocation,
    then a barrier of the CTA, then the signal."""
    for name, body in kernels(open(path).read()):
        alloc, signal = re.search(r"\btmem_alloc\w*\(", body), re.search(r"\bgriddep_launch_dependents\(", body)
        if alloc is None or signal is None:
            continue
        assert alloc.start() < signal.start(), name
        assert re.search(r"__syncthreads\(|cluster_wait\w*\(|cluster_sync\w*\(", body[alloc.end():signal.start()]), name
