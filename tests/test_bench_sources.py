"""bench.py reports recorded DRAM traffic only for the sources it was captured from (CPU)."""
import os
import re

import bench
from tests import kernel_source as S


def test_every_device_source_of_the_gemms_counts():
    seen, todo = set(), ["q8_gemm.cu"]
    while todo:
        f = todo.pop()
        seen.add(f)
        with open(os.path.join(S.CSRC, f)) as fh:
            todo += [g for g in re.findall(r'#include "(\w+\.cuh)"', fh.read()) if g not in seen]
    assert seen == set(bench.GEMM_SOURCES)
