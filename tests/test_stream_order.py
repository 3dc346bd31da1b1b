"""Kernels that may start beside the one ahead of them on their stream (programmatic dependent launch) touch no memory of
a call before they have waited for it: a source check, since a kernel that reads too early is right most of the time."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_long_context_lightning_b200", "csrc")
# loads and stores of global memory as the sources write them: bulk and asynchronous copies, cached loads, atomics, and
# the pointers of a kernel's argument struct
ACCESS = re.compile(r"\b(tma_load\w*|cp_async\w*|__ldg|__ldcg|__ldcs|ld_global\w*|st_global\w*|atomic\w+|red_\w+)\s*\(|\ba\.\w+\s*\[|[=(,;{]\s*\*\s*a\.\w+")


def _source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def _kernels():
    """(file, kernel, body) of every __global__ function."""
    for name in sorted(f for f in os.listdir(CSRC) if f.endswith(".cu")):
        text = _source(name)
        for m in re.finditer(r"__global__[^;{]*?\b(k_\w+)\s*\(", text):
            at = text.index("{", text.index(")", m.end()))
            depth, end = 0, at
            for end in range(at, len(text)):
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                if depth == 0:
                    break
            yield name, m.group(1), text[at:end]


KERNELS = {k: (f, body) for f, k, body in _kernels()}
EARLY = sorted(k for k, (_, body) in KERNELS.items() if "pdl_wait()" in body)


def test_every_kernel_launched_early_waits():
    launched = set()
    for name in sorted(f for f in os.listdir(CSRC) if f.endswith(".cu")):
        for m in re.finditer(r"launch_pdl\(\s*([^;]*)", _source(name)):
            launched |= set(re.findall(r"\bk_\w+", m.group(1).split("dim3")[0]))
    assert launched and launched <= set(KERNELS)
    assert launched <= set(EARLY), sorted(launched - set(EARLY))


@pytest.mark.parametrize("kernel", EARLY)
def test_nothing_is_read_or_written_ahead_of_the_wait(kernel):
    name, body = KERNELS[kernel]
    ahead = body[: body.index("pdl_wait()")]
    found = ACCESS.search(ahead)
    assert found is None, f"{name}: {kernel} has {found.group(0)!r} ahead of pdl_wait()"
    trigger = body.find("pdl_launch_dependents()")
    assert trigger < 0 or trigger > body.index("pdl_wait()"), f"{name}: {kernel} lets the next kernel start before its own wait"
