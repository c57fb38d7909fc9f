"""Kernels that start beside the end of the one before them (programmatic dependent launch) may not promise the compiler that
what that one writes is constant while they run: a `const __restrict__` pointer allows loads by the read-only path and
ahead of the wait, which orders no such load."""
import os
import re

import pytest

import paged_kv_attention_29_gb300 as pkv

CSRC = os.path.join(os.path.dirname(os.path.abspath(pkv.__file__)), "csrc")


def kernels():
    """(name, parameters, body) of every __global__ function."""
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__", text):
            start = text.index("{", m.end())
            depth, end = 1, start + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            head = text[m.end():start]
            kernel = re.search(r"(\w+)\s*\((?!.*\b\w+\s*\(\s*const)", re.sub(r"__launch_bounds__\([^)]*\)|__grid_constant__", "", head), re.S).group(1)
            yield f"{name}:{kernel}", head, text[start:end]


WAITING = [(n, h) for n, h, body in kernels() if "griddepcontrol.wait" in body]


def test_the_kernels_are_found():
    names = {n for n, _ in WAITING}
    assert {"tree_decode.cu:tree_decode_kernel", "tree_decode.cu:tree_join_kernel", "tree_decode_rows.cu:tree_rows_join_kernel",
            "decode.cu:decode_combine_kernel"} <= names, names


@pytest.mark.parametrize("name,head", WAITING, ids=[n for n, _ in WAITING])
def test_no_promise_of_constant_memory(name, head):
    assert not re.search(r"\bconst\s+\w+\s*\*\s*(const\s+)?__restrict__", head)
