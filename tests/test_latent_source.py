"""Rules of the latent attention's kernel that no run shows, read from its source."""
import os
import re

from sparse_attention_paged_gb300 import _native


def test_one_register_count_per_warpgroup():
    """All warps of a warpgroup run the same setmaxnreg instruction: each count stands once, at the
    head of a branch that whole warpgroups take (the counts' own sums are static assertions)."""
    with open(os.path.join(_native.CSRC, "latent_attention_sm103.cu")) as f:
        lines = [line.strip() for line in f if not line.strip().startswith("//")]
    at = [i for i, line in enumerate(lines) if re.fullmatch(r"(more|fewer)_registers<\w+>\(\);", line)]
    counts = [re.search(r"<(\w+)>", lines[i]).group(1) for i in at]
    assert sorted(counts) == ["kRegsLoad", "kRegsMisc", "kRegsSoftmax"]
    for i, count in zip(at, counts):
        branch = {"kRegsLoad": "if (warp >= kLoadWarp0) {", "kRegsMisc": "} else if (warp >= kMmaWarp) {",
                  "kRegsSoftmax": "} else {"}[count]
        assert lines[i - 1] == branch
