"""Launches that may start early (programmatic dependents) and the order of memory: only a
kernel's own griddepcontrol.wait makes what the launches before it wrote visible to it, so
each kernel of the matrix operators waits, unconditionally, before it reads or writes
anything of global memory (checked in the source, no GPU needed)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rms_backward_gb300", "csrc")
WAIT = "ptx::grid_dependency_wait()"
# what touches global memory: copies, the epilogues' and inputs' reads, stores, plain accesses by index (the prefetch
# of weights in the token kernel reads no value and needs no order)
ACCESS = re.compile(r"tma_load|\.raw\(|epi\.(read|write|ahead)|\.store\(|over_pieces|partial\[|all\.c\[|a\.x\b|a\.out\b")


def _body(text, start):
    """The kernel's body: from its first brace at the end of the signature to the brace that closes it."""
    at = text.index(") {", start) + 2
    depth, i = 0, at
    while True:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
        if depth == 0:
            return text[at:i]


def _kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "mhcm_*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for k in re.finditer(r"__global__", text):
            body = _body(text, k.start())
            name = re.search(r"(\w+_kernel)\(", text[k.start():]).group(1)
            yield pytest.param(body, id=f"{os.path.basename(path)}-{name}")


@pytest.mark.parametrize("body", list(_kernels()))
def test_waits_before_it_touches_memory(body):
    before, waits = "", []
    depth = 0
    for line in body.split("\n"):
        if WAIT in line:
            waits.append((line.strip(), depth, before))
        before += line + "\n"
        depth += line.count("{") - line.count("}")
    assert len(waits) == 1, "one wait"
    line, depth, before = waits[0]
    assert line == WAIT + ";" and depth == 1, f"unconditional: {line}"
    assert not re.search(r"\bif \([^\n]*\)\s*$", before.rstrip()), "not the body of an if"
    assert not (found := ACCESS.search(before)), f"before the wait: {found.group(0)}"


def test_every_kernel_is_seen():
    assert len(list(_kernels())) == 6
