"""What the 8-bit kernels' sources keep to where a run cannot show it (no GPU)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_modular_int8_gb300", "csrc")


def test_status_is_cleared_before_the_next_kernel_starts():
    """A product beside the one before it keeps the status that this one clears.  So in the block that clears it the
    next kernel is let go by the clearing thread alone, behind a fence: no thread of that block passes another
    allow_dependents() first."""
    found = 0
    for path in glob.glob(os.path.join(CSRC, "f8_*.cu*")):
        with open(path) as f:
            lines = [re.sub(r"//.*", "", s).strip() for s in f]
        code = [s for s in lines if s]
        if not any("keep_status" in s for s in code):  # no product of which another could keep the status
            continue
        for i, s in enumerate(code):
            if not s.endswith("status = 0;"):
                continue
            found += 1
            assert re.match(r"if \(blockIdx\.x == 0 && !\w+\.keep_status\) \{$", code[i - 2]), path
            assert code[i - 1] == "if (threadIdx.x == 0) {", path
            assert code[i + 2:i + 8] == ["__threadfence();", "allow_dependents();", "}", "} else {", "allow_dependents();",
                                         "}"], path
            start = max(j for j in range(i) if "__device__" in code[j] or "__global__" in code[j])
            assert not any("allow_dependents" in c for c in code[start:i]), path
    assert found == 2
    assert all("clear_status" not in open(p).read() for p in glob.glob(os.path.join(CSRC, "f8_*.cu*")))
