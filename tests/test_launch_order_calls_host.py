"""Order of tensor-memory allocation and dependent launch where a device function allocates for a kernel (no GPU).

tests/test_launch_order_host.py looks at kernels that allocate in their own body.  Here: those that call a function which does.
Each of their triggers comes after the call and a barrier, or belongs to the instantiations that make no such call."""
import glob
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "ternary_weight_linear_02_gb300", "csrc")
ALLOC, TRIGGER, SYNC = r"\btmem_alloc\(", r"\bpdl_launch_dependents\(\)\s*;", r"\b__syncthreads\(\)\s*;"


def functions():
    """(file, qualifier, name, body) of the functions of the sources that run on the device."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__(global|device)__", text):
            brace, semi = text.find("{", m.start()), text.find(";", m.start())
            if brace < 0 or 0 <= semi < brace:
                continue  # a declaration
            depth = 0
            for end in range(brace, len(text)):
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                if depth == 0:
                    break
            names = re.findall(r"(\w+)\s*\(", text[m.start():brace])
            names = [n for n in names if n not in ("__launch_bounds__", "__align__")]
            if names:
                yield os.path.basename(path), m.group(1), names[0], text[brace:end]


ALL = list(functions())


def allocating():
    """Names of device functions that allocate, by themselves or by a call."""
    names = {n for _, q, n, body in ALL if q == "device" and re.search(ALLOC, body)}
    while True:
        more = {n for _, q, n, body in ALL if q == "device" and any(re.search(rf"\b{f}\s*(<[^;{{}}]*?>)?\(", body) for f in names)} - names - {"tmem_alloc"}
        if not more:
            return names - {"tmem_alloc"}
        names |= more


def conditions(body, at):
    """The text before each brace that is open at a place of a body."""
    open_, last = [], 0
    for m in re.finditer(r"[{}]", body[:at]):
        if m.group() == "{":
            open_.append(" ".join(body[last:m.start()].split())[-60:])
        else:
            open_.pop()
        last = m.end()
    return open_


def check(body, calls):
    for t in re.finditer(TRIGGER, body):
        if max(calls) < t.start() and re.search(SYNC, body[max(calls):t.start()]):
            continue
        guard = re.search(r"if (?:constexpr )?\(!(\w+)\)\s*$", body[:t.start()])
        assert guard, "dependents may start before the tensor memory is allocated"
        for at in calls:
            assert any(c.endswith(f"if constexpr ({guard.group(1)})") for c in conditions(body, at)), "the call is made by instantiations that trigger early"


def test_kernels_that_allocate_by_a_call():
    names, seen = allocating(), set()
    assert "shrink_big" in names
    for file, kind, name, body in ALL:
        calls = [m.start() for f in names for m in re.finditer(rf"\b{f}\s*(<[^;{{}}]*?>)?\(", body)] if kind == "global" else []
        if calls:
            seen.add((file, name))
            check(body, calls)
    assert ("kern_lora.cuh", "lora_kernel") in seen


def test_the_check_sees_a_trigger_that_comes_too_early():
    (body,) = [b for f, q, n, b in ALL if (f, q, n) == ("kern_lora.cuh", "global", "lora_kernel")]
    calls = [m.start() for m in re.finditer(r"\bshrink_big\s*<T>\(", body)]
    assert len(calls) == 1
    check(body, calls)
    wrong = body.replace("if (!BIG) pdl_launch_dependents();", "pdl_launch_dependents();")
    assert wrong != body
    try:
        check(wrong, [m.start() for m in re.finditer(r"\bshrink_big\s*<T>\(", wrong)])
    except AssertionError:
        return
    raise AssertionError("an early trigger went unnoticed")
