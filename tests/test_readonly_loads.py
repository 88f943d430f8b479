"""The read-only load path (ld.global.nc, __ldg) serves the layer's own weights alone.

Every forward kernel is launched with programmatic serialization and so runs beside the earlier
kernels of the stream that write its operands (activations, scales, bias, multiplier, residual);
the path is for memory that nothing writes meanwhile.  Read from the sources, on the CPU.
"""
from __future__ import annotations

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4_gemm_error_b200", "csrc")
# what packing writes: scales, zero points, codes and the Error Compensator's B and G
WEIGHTS = {"p.s", "p.z", "s", "z", "p.Bt", "Bt", "g0", "g1", "at"}
# launched without programmatic serialization: nothing runs beside them
PLAIN_LAUNCH = {"pack.cu", "gate_noalloc.cu"}
CALL = re.compile(r"\b(?:__ldg|ld_nc|ld_stream)\((?:reinterpret_cast<[^>]*>\()?\s*\(?\s*([A-Za-z_][\w.]*)")


def calls(text):
    return [m.group(1) for m in CALL.finditer(re.sub(r"//[^\n]*", "", text)) if m.group(1) not in ("const",)]


FILES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu*")))


@pytest.mark.parametrize("name", FILES)
def test_only_weights_are_read_as_constants(name):
    text = open(os.path.join(CSRC, name)).read()
    if name in PLAIN_LAUNCH:
        assert "programmaticStreamSerializationAllowed" not in text
        return
    text = re.sub(r"(?ms)^__device__ __forceinline__ uint4 ld_nc\(const void \*p\)\n\{.*?^\}", "", text)
    bad = [c for c in calls(text) if c not in WEIGHTS]
    assert not bad, (name, bad)


def test_the_search_finds_an_operand():
    """Planted mistakes, in the forms that the sources use."""
    for line in ("o.bias = bf16_lo(__ldg(e.bias + n));", "xs = __ldg(p.xs + t);", "a = ld_nc(src);",
                 "const uint2 q = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(x) + i));",
                 "p.epi.bias ? __ldg(reinterpret_cast<const uint32_t *>(p.epi.bias + n)) : 0u;"):
        assert any(c not in WEIGHTS for c in calls(line)), line
