"""Kernels that are launched behind another one while that one still runs (launch_behind): they have to wait for
it, and may not promise that what it writes is read-only."""
import glob
import os
import re

import shared_prompt_exact_gb300 as pkg

CSRC = os.path.join(os.path.dirname(pkg.__file__), "csrc")


def _kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for name in re.findall(r"launch_behind\(\s*(\w+)", text):
            found = re.search(r"__global__[^;{]*?\b" + name + r"\s*\(([^{]*)\)\s*\{(.*?)\n\}", text, re.S)
            assert found, (path, name)
            yield name, found.group(1), found.group(2)


def test_kernels_launched_behind_another():
    kernels = list(_kernels())
    assert len(kernels) >= 2
    for name, parameters, body in kernels:
        assert "cudaGridDependencySynchronize()" in body, name
        # const __restrict__ lets the compiler move a read of the predecessor's output before the wait
        assert not re.search(r"const[^,]*\*\s*__restrict__", parameters), name
        assert "__ldg" not in body and ".nc" not in body, name
