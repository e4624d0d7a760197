"""TMEM columns without a cycle of waits, shown on the host.

tcgen05.alloc waits until its columns are free, without a limit.  A launch that
programmatic serialisation starts early keeps the columns it gets until the launch before
it has ended, so that one must own all of its columns by then: a kernel lets its dependents
start only behind the barrier after its allocation (one call of a block is enough to
let them)."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_ffn_06_b200", "csrc")


def _kernels_with_tmem():
    """(file, name, body) of every kernel that allocates TMEM."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for part in text.split("__global__")[1:]:
            body = part[:part.find("\n}\n")]
            if "tmem_alloc" in body:
                name = re.search(r"(\w+_kernel)\(", body).group(1)
                found.append((os.path.basename(path), name, body))
    return found


def test_the_kernels_with_tmem_are_found():
    assert [(f, n) for f, n, _ in _kernels_with_tmem()] == [
        ("decode_tc.cu", "decode_tc_kernel"), ("gemm_tc.cu", "grouped_gemm_kernel"),
        ("linear_i8.cu", "linear_i8_kernel")]


@pytest.mark.parametrize("kernel", _kernels_with_tmem(), ids=lambda k: k[1])
def test_dependents_start_behind_the_allocation(kernel):
    body = kernel[2]
    alloc = max(m.start() for m in re.finditer(r"tmem_alloc", body))
    owned = body.index("tmem_base = ctl->tmem_base")
    barrier = body.rindex("__syncthreads()", 0, owned)  # the barrier that publishes the columns
    triggers = [m.start() for m in re.finditer(r"pdl_trigger\(\)", body)]
    assert alloc < barrier and triggers and min(triggers) > owned
