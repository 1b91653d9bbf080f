"""What the token operators' sources have to hold that no run would show."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sign_muon_optimizer_momentum_b200", "csrc")


def kernels(name):
    """(name, parameters, body) of each __global__ function of a source."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())

    def closing(at, pair):
        depth = 0
        for i in range(at, len(text)):
            depth += (text[i] == pair[0]) - (text[i] == pair[1])
            if depth == 0:
                return i
        raise AssertionError("unbalanced")
    for m in re.finditer(r"__global__", text):
        at = m.end()
        bounds = re.compile(r"\s*void\s+__launch_bounds__\s*").match(text, at)
        if bounds:
            at = closing(bounds.end(), "()") + 1
        head = re.compile(r"\s*(?:void\s+)?(\w+)\s*\(").match(text, at)
        end = closing(head.end() - 1, "()")
        start = text.index("{", end)
        yield head.group(1), text[head.end():end], text[start:closing(start, "{}") + 1]


@pytest.mark.parametrize("source", ["embedding.cu", "layer_norm.cu", "distill.cu"])
def test_kernels_that_wait_read_by_ordinary_loads(source):
    """A kernel that is launched while the one before still writes its inputs
    must not take them as `const __restrict__` (which allows the read-only path
    and loads before the wait) nor by __ldg."""
    found = [k for k in kernels(source) if "wait_for_kernel_before()" in k[2]]
    assert found
    for name, params, body in found:
        assert "__restrict__" not in params, name
        assert "__ldg" not in body, name
