"""What cannot be provoked on a GPU without faulting it, read in the kernels' source."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "paged_kv_cache_272_gb300", "csrc")


def kernels(name):
    """(kernel, body without comments) of every __global__ function of a source file."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s+)?(\w+)\(",
                         text):
        at = text.index("{", text.index(")", m.end()))
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield m.group(1), text[at:end]


@pytest.mark.parametrize("name", ["tree_attention.cu", "tree_masks.cu", "qk_rope.cu", "prefill.cu"])
def test_no_kernel_ends_before_it_has_waited_for_the_one_before(name):
    """The kernel behind a dependent launch waits for that launch alone: one that ended without
    waiting would let it start while an older kernel still runs."""
    found = list(kernels(name))
    assert found
    for kernel, body in found:
        ends = [m.start() for m in re.finditer(r"\breturn\b", body)]
        # the lambdas of these kernels come after the wait
        assert body.index("pdl_wait()") < min(ends, default=len(body)), kernel


def enclosing_block(text, at):
    depth = 0
    for i in range(at - 1, -1, -1):
        depth += {"}": 1, "{": -1}.get(text[i], 0)
        if depth < 0:
            return text[i:at]
    raise AssertionError("no block")


def test_every_way_out_of_tree_attention_tells_the_join():
    """The join is launched whatever happens and reads a record per CTA of a workspace that
    nothing initialises: each early way out writes one, and so does the way through."""
    body = dict(kernels("tree_attention.cu"))["tree_attention_kernel"]
    outs = [m.start() for m in re.finditer(r"\breturn;", body)]
    assert len(outs) == 2
    for at in outs:
        assert re.search(r"a\.join\[[^]]+\]\.parts = 0;", enclosing_block(body, at))
    assert re.search(r"if \(t == 0\) a\.join\[plan->slot\]\.parts = 0;", body[outs[-1]:])
