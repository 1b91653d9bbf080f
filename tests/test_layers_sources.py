"""What the token operators' sources have to hold that no run would show."""
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "sign_muon_optimizer_momentum_b200")
CSRC = os.path.join(PACKAGE, "csrc")


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


def run_build(tmp_path, *flags, code="print(build.build())"):
    """build() of a copy of the package, with a stand-in for nvcc, by a Python
    that is started with `flags`."""
    package = tmp_path / "sign_muon_optimizer_momentum_b200"
    shutil.copytree(CSRC, package / "csrc")
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    shutil.copy(os.path.join(PACKAGE, "build.py"), package)
    (package / "__init__.py").write_text("")
    tools = tmp_path / "tools"
    tools.mkdir()
    (tools / "nvcc").write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && : > "$2"; shift; done\n')
    (tools / "nvcc").chmod(0o755)
    env = dict(os.environ, PATH=f"{tools}:{os.environ['PATH']}")
    env.pop("PYTHONPATH", None)
    r = subprocess.run([sys.executable, *flags, "-c", f"import sys; sys.path.insert(0, {str(tmp_path)!r})\n"
                        f"from sign_muon_optimizer_momentum_b200 import build\n{code}"],
                       capture_output=True, text=True, env=env, timeout=300)
    return r, package


def test_library_is_built_without_pytorch(tmp_path):
    r, package = run_build(tmp_path, "-S")       # no site-packages: no PyTorch
    assert r.returncode == 0, r.stderr
    assert (package / "libsignmuon.so").exists() and not (package / "_layers_native.so").exists()
    assert "without the binding" in r.stderr


def test_library_is_built_where_the_binding_fails(tmp_path):
    fail = ("def fail(verbose):\n    raise RuntimeError('no binding')\n"
            "build._binding_can_be_built = lambda: True\nbuild._compile_binding = fail\nbuild.build()")
    r, package = run_build(tmp_path, "-S", code=fail)
    assert r.returncode != 0 and "no binding" in r.stderr
    assert (package / "libsignmuon.so").exists()
