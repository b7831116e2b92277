"""What the library keeps between calls, from its sources (no GPU): state that belongs to a device is
not kept for the process."""
import glob
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "ternary_weight_linear_02_gb300", "csrc")


def test_no_result_of_a_cuda_call_is_kept_in_a_static():
    """A static initialised by a CUDA call holds the answer for the device that was current first (a
    kernel's shared-memory limit, say), and a failure for good."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.c*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\bstatic\b[^;{}()]*=\s*cuda\w+\s*\(", text):
            found.append(f"{os.path.basename(path)}: {' '.join(m.group(0).split())}")
    assert not found, found


def test_limits_are_remembered_per_device_and_only_on_success():
    """The attention kernels' limits: a bit per device, set after the call that succeeded."""
    text = open(os.path.join(CSRC, "attn_sched.cuh")).read()
    body = text[text.index("attn_allow_smem"):]
    body = body[:body.index("\n}")]
    assert body.index("cudaGetDevice") < body.index("cudaFuncSetAttribute") < body.index("fetch_or")
    assert re.search(r"if \(e == cudaSuccess\) done\.fetch_or\(bit", body)
