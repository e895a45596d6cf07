"""The order in which kernels take tensor memory, read from the sources (no GPU needed): an allocation waits until
other kernels on the SM give columns back, so a block must not hold any while it waits for another kernel's end, and
the next kernel may start only when every block holds its own."""
import glob
import os
import re

import pytest

import residual_stream_norm_gb300 as rsn

CSRC = os.path.join(os.path.dirname(os.path.abspath(rsn.__file__)), "csrc")


def kernels():
    """(file, kernel's text without comments) of every kernel that allocates tensor memory."""
    for path in sorted(glob.glob(os.path.join(CSRC, "**", "*.cu"), recursive=True)):
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path, encoding="utf-8").read(), flags=re.S)
        for body in text.split("__global__")[1:]:
            if re.search(r"\btmem_alloc\w*\(", body):
                yield os.path.basename(path), body


def test_the_kernels_are_found():
    assert [name for name, _ in kernels()] == ["attn_prefix_tc.cu", "kv4_attn.cu"]


@pytest.mark.parametrize("name", ["attn_prefix_tc.cu", "kv4_attn.cu"])
def test_allocation_stands_behind_the_wait_and_before_the_trigger(name):
    body = dict(kernels())[name]
    steps = ["pdl_wait(", "tmem_alloc", "__syncthreads(", "pdl_launch_dependents("]
    at = [body.index(s) for s in steps]  # the first of each
    assert at == sorted(at), dict(zip(steps, at))
