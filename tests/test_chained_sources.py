"""Kernels that start while the grid ahead still writes their inputs promise the compiler nothing about them."""
import os
import re

import pytest

from gqa_softmax_attention_attn_b200.build import CSRC, SOURCES


def chained_kernels():
    """(file, name, parameter list, the file) of every kernel that waits for the grid ahead."""
    for f in SOURCES:
        with open(os.path.join(CSRC, f)) as fh:
            text = fh.read()
        for m in re.finditer(r"\b__global__\b", text):
            head = re.match(r"__global__ void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\(([^{]*?)\)\s*\{",
                            text[m.start():])
            if head is None:
                continue
            end = text.find("\n}\n", m.start())
            if "grid_dep_wait()" in text[m.start():end]:
                yield f, head.group(1), head.group(2), text


def test_every_chained_kernel_is_seen():
    names = {k[1] for k in chained_kernels()}
    assert {"tree_tc_kernel", "tree_join_kernel", "tree_simt_kernel", "tree_combine_kernel", "page_map_kernel",
            "qk_norm_fwd_kernel", "qk_norm_bwd_kernel", "qk_norm_finish_kernel", "decode_combine_kernel",
            "bwd_tc_kernel", "bwd_finish_kernel", "fwd_tc_kernel"} <= names


@pytest.mark.parametrize("kernel", list(chained_kernels()), ids=lambda k: k[1])
def test_no_promise_of_unwritten_inputs(kernel):
    f, name, params, text = kernel
    assert "__restrict__" not in params, f"{f}: {name}"
    structs = re.findall(r"const (\w+) &?\w+(?:,|$)", params)
    while structs:
        body = re.search(r"struct %s \{(.*?)\n\};" % structs.pop(), text, re.S)
        if body:  # (shared headers hold no such pointers)
            assert "__restrict__" not in body.group(1), f"{f}: {name}"
            structs += re.findall(r"^    (\w+) \w+;", body.group(1), re.M)


def test_shared_headers():
    for f in ("kernels.h", "tree_path.cuh"):
        with open(os.path.join(CSRC, f)) as fh:
            code = re.sub(r"//.*", "", fh.read())
        assert "__restrict__" not in code
