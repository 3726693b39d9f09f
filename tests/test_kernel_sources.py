"""Rules of the kernel sources that no run can show to be broken."""
import os
import re

import pytest

from compressed_sparse_kv_04_b200 import build as csa_build

# Non-coherent loads (ld.global.nc: __ldg, or loads through a const __restrict__
# pointer) are defined only for data that nothing writes while the kernel is
# resident.  A kernel launched with programmatic serialization is resident while
# the kernel before it still writes, so it may use them only for data that is
# complete before it can start:
READ_ONLY = {
    # The queries' codes, scales and head weights: the caller's, complete before the
    # call's first kernel lets this one start.
    "indexer.cu": {"__ldg": 3},
    # Launched in the ordinary way (shard_candidates_kernel).
    "topk.cu": {"__restrict__": 3},
    # Loaded with __ldcg (proj_reduce_kernel).
    "proj.cu": {"__restrict__": 1},
}


def _code(path):
    s = open(path).read()
    s = re.sub(r"/\*.*?\*/", "", s, flags=re.S)
    return re.sub(r"//[^\n]*", "", s)


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(csa_build.CSRC)
                                        if f.endswith((".cu", ".cuh"))))
def test_data_of_a_running_predecessor_is_read_coherently(name):
    code = _code(os.path.join(csa_build.CSRC, name))
    found = {"__ldg": len(re.findall(r"\b__ldg\s*\(", code)),
             "__restrict__": len(re.findall(r"\bconst\s+\w+\s*\*\s*__restrict__", code))}
    allowed = READ_ONLY.get(name, {})
    for what, n in found.items():
        assert n <= allowed.get(what, 0), f"{name}: {n} uses of {what}"
    assert "ld.global.nc" not in code
