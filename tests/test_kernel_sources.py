"""What the kernels' sources must not hold, read on the CPU."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "segmented_gather_gemm_amd", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h")))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_inline_assembly_only_waits(path):
    """The compiler leaves the wait states that a matrix instruction's result needs only ahead of
    instructions that it knows: one in inline assembly may read the registers too early."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for body in re.findall(r"\basm\b\s*(?:volatile)?\s*\(\s*\"([^\"]*)\"", text):
        for line in re.split(r"\\n|;", body):
            assert not line.strip() or line.split()[0] == "s_waitcnt", (path, body)
    assert len(re.findall(r"\basm\b", text)) == \
        len(re.findall(r"\basm\b\s*(?:volatile)?\s*\(\s*\"", text)), path
