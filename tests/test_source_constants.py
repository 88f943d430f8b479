"""Launch rules of the sources that depend on the device, read from them on the CPU."""
from __future__ import annotations

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4_gemm_error_b200", "csrc")


def test_no_launch_rule_has_the_number_of_sms_in_it():
    """B200's 148 SMs appear as the value of a variable that the device's own count replaces, nowhere else."""
    bad = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*")) + glob.glob(os.path.join(CSRC, "*.h"))):
        for i, line in enumerate(open(path), 1):
            code = re.sub(r"//.*", "", line)
            if re.search(r"\b148\b", code) and not re.fullmatch(r"\s*int \w+ = 148;\s*", code):
                bad.append((os.path.basename(path), i, line.strip()))
    assert not bad, bad
