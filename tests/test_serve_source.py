"""What the kernels that overlap the end of the kernel before them may do first, read
from their source: a GPU test would need that kernel to fail."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mask_aware_sparse_gb300", "csrc")


def _kernels():
    """(name, body) of every __global__ function of the files that launch dependent kernels."""
    out = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        if "grid_dependency_wait" not in text:
            continue
        for m in re.finditer(r"__global__[^{;]*?(\w+_kernel)\s*\([^{;]*\)\s*\{", text):
            depth, end = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            out.append((m.group(1), text[m.end():end]))
    return out


def test_kernels_are_found():
    names = {n for n, _ in _kernels()}
    assert {"qk_kernel", "qk_weights_kernel", "write_kernel", "read_kernel", "few_kernel", "chunk_kernel", "plan_kernel",
            "join_kernel"} <= names


@pytest.mark.parametrize("name, body", _kernels(), ids=[n for n, _ in _kernels()])
def test_no_memory_of_earlier_kernels_before_the_wait(name, body):
    wait = re.search(r"grid_dependency_wait\(\)|look_up<", body)  # (look_up starts with it)
    assert wait, name
    before = body[:wait.start()]
    # the error word, tensors and plans all come through the parameter p
    for use in re.findall(r"[=(,;{!]\s*\*\s*p\.\w+|p\.[\w.]+\s*\[|\(p\.err|timeout_pending", before):
        pytest.fail(f"{name} touches {use.strip()} before it waits")


def test_the_chunk_kernel_ends_with_nothing_in_flight():
    # a wait that ran out elsewhere in the CTA must not let it end under its own copies or products:
    # the last acts of the warp that starts each kind are waits for all of them, whatever `ok` says
    body = dict(_kernels())["chunk_kernel"]
    copies = body[body.index("uint32_t asked"):body.index("else if (warp == 9)")]
    for started in ("++asked_q;", "++asked;"):
        assert copies.count(started) == 1
    end = copies[copies.rindex("if (lane == 0) {"):]
    assert all(x in end for x in ("asked_q > 0", "C::QFULL", "C::RFULL", "C::VFULL", "C::KFULL", "r < asked"))
    assert "ok" not in re.findall(r"\b\w+\b", end)
    products = body[body.index("else if (warp == 9)"):]
    assert re.search(r"mma_commit\(&bars\[C::MEND\]\);\s*mbar_wait\(&bars\[C::MEND\]", products)
