"""The check of the attention's split records, compiled for the host (no GPU)."""
import os
import shutil
import subprocess

import pytest

from sparse_attention_paged_gb300 import _native

pytestmark = pytest.mark.skipif(shutil.which(_native.NVCC) is None, reason="nvcc not available")

MAIN = r"""
#include <stdio.h>
#include "dsa_indexer.h"
#include "latent_common.cuh"
int main() {
  int row, last, first, rows, ctas;
  while (scanf("%d %d %d %d %d", &row, &last, &first, &rows, &ctas) == 5)
    printf("%d\n", (int)dsa::split_record_ok(row, last, first, rows, ctas));
}
"""


def test_records_outside_the_call(tmp_path):
    src, exe = tmp_path / "records.cu", tmp_path / "records"
    src.write_text(MAIN)
    subprocess.run([_native.NVCC, *_native.ARCH_FLAGS, *_native.NVCC_FLAGS, str(src), "-o", str(exe)], check=True,
                   capture_output=True)
    most = 2 ** 31 - 1
    good = [(0, 0, 0, 1, 1), (4, 151, 0, 5, 152), (0, 3, 3, 9, 76)]
    bad = [(-2, 1, 0, 5, 152), (5, 1, 0, 5, 152), (most, 1, 0, 5, 152), (0, 152, 0, 5, 152), (0, most, 0, 5, 152),
           (0, 0, 1, 5, 152), (0, 1, -1, 5, 152), (0, -1, -most, 5, 152), (2143289344, 2143289344, 2143289344, 5, 152)]
    text = "\n".join(" ".join(map(str, r)) for r in good + bad)
    got = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split()
    assert got == ["1"] * len(good) + ["0"] * len(bad)
    with open(os.path.join(_native.CSRC, "latent_attention_sm103.cu")) as f:
        join = f.read().split("latent_join_kernel(const LatentAttnParams p,")[1]
    # before the record's first use as an address
    assert join.index("split_record_ok(row, rec.y, rec.z, p.rows, p.ctas)") < join.index("p.ws + ((long long)rec.z")
