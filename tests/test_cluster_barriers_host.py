"""Cluster barriers in the sources of the calls that take pages (no GPU): they hang on launch arguments alone."""
import os
import re

from conftest import ROOT


def test_taking_pages_meets_every_barrier():
    """A barrier under a condition that a block computes from memory could leave the cluster's other blocks waiting: each
    stands directly under `if (C > 1)`, in the kernel's own body."""
    text = open(os.path.join(ROOT, "ternary_weight_linear_02_gb300", "csrc", "kern_pages.cu")).read()
    text = re.sub(r"//[^\n]*", "", text)
    body = text[text.index("pages_take_kernel(PagesTakeArgs a) {"):]
    depth, found = 0, 0
    stack = []
    for m in re.finditer(r"\{|\}|cl_arrive_release\(\)|cl_wait_acquire\(\)|cluster_wait\(\)", body):
        if m.group() == "{":
            stack.append(" ".join(body[:m.start()].split())[-24:])
        elif m.group() == "}":
            stack.pop()
            if not stack:
                break
        else:
            found += 1
            assert len(stack) == 2 and stack[1].endswith("if (C > 1)"), stack
    assert found == 5
