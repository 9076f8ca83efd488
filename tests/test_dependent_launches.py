"""Kernels that are launched to start while the kernel ahead of them on the stream is still running read what that kernel
writes after griddepcontrol.wait.  The read-only path (ld.global.nc) is for memory that nothing writes while the kernel
runs, so they must not take it, neither by instruction nor by a const __restrict__ parameter, from which the compiler does."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_io_aware_17_gb300", "csrc")


def _sources():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path, encoding="utf-8") as f:
            yield os.path.basename(path), re.sub(r"//[^\n]*", "", f.read())


def _kernels(text):
    """(parameters, body) of each __global__ function."""
    for m in re.finditer(r"__global__", text):
        name = re.compile(r"(\w+_kernel)\s*\(").search(text, m.end())
        open_at, depth = text.index("{", name.end()), 0
        for end in range(open_at, len(text)):
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            if depth == 0:
                break
        yield name.group(1), text[name.end():open_at], text[open_at:end]


def test_no_read_only_loads():
    for name, text in _sources():
        assert ".nc." not in text and "__ldg(" not in text, name


def test_kernels_that_wait_have_no_read_only_parameters():
    waiting = 0
    for source, text in _sources():
        for name, parameters, body in _kernels(text):
            if "griddep_wait()" in body:
                waiting += 1
                assert not re.search(r"const [\w ]+\*\s*__restrict__", parameters), (source, name)
    assert waiting >= 8
