"""How the selection shares a row's pages out among blocks, compiled for the host (no GPU)."""
import shutil
import subprocess

import pytest

from sparse_attention_paged_gb300 import _native

pytestmark = pytest.mark.skipif(shutil.which(_native.NVCC) is None, reason="nvcc not available")

MAIN = r"""
#include <stdio.h>
#include "paged_common.cuh"
// rows without pages and with a length past the table among them: a division by zero is no constant
static_assert(dsa::select_run(0, 1) == 1 && dsa::select_run(0, 8) == 1, "run");
static_assert(dsa::select_active(0, dsa::select_run(0, 8)) == 1, "blocks");
int main() {
  int n, blocks;
  while (scanf("%d %d", &n, &blocks) == 2) {
    const int run = dsa::select_run(n, blocks);
    printf("%d %d\n", run, dsa::select_active(n, run));
  }
}
"""


def test_runs_of_a_row(tmp_path):
    src, exe = tmp_path / "runs.cu", tmp_path / "runs"
    src.write_text(MAIN)
    subprocess.run([_native.NVCC, *_native.ARCH_FLAGS, *_native.NVCC_FLAGS, str(src), "-o", str(exe)], check=True,
                   capture_output=True)
    cases = [(n, b) for b in (1, 2, 4, 8) for n in (0, 1, 2, 255, 256, 257, 511, 512, 513, 1000, 2047, 2048, 2049, 4097, 32768)]
    text = "\n".join(f"{n} {b}" for n, b in cases)
    out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split()
    most = {}
    for i, (n, blocks) in enumerate(cases):
        run, active = int(out[2 * i]), int(out[2 * i + 1])
        assert run >= 1 and 1 <= active <= blocks
        # the runs have every page, the last one at least one of them, and no row more than the widest
        assert active * run >= n and (active == 1 or (active - 1) * run < n)
        assert active == 1 or run >= 256
        assert run >= most.get(blocks, 0)
        most[blocks] = run
