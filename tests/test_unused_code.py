"""The HIP sources hold no function or variable that nothing reaches: the
compiler's own warnings, for the host and for gfx950.  Runs on the CPU."""
import os
import re
import subprocess

import pytest

from token_routing_expert_amd import build as tre_build


@pytest.mark.timeout(300)
@pytest.mark.parametrize("source", tre_build.SOURCES)
def test_nothing_unused(source):
    r = subprocess.run([tre_build.hipcc(), *tre_build.FLAGS, "-fsyntax-only", os.path.join(tre_build.CSRC, source)],
                       capture_output=True, text=True, timeout=280)
    assert r.returncode == 0, r.stderr[-2000:]
    found = re.findall(r"^.*\[-Wunused-(?!command-line-argument).*\]$", r.stderr, re.M)
    assert not found, "\n".join(found)
