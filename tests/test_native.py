"""Host checks in C++ of what the kernels' headers compute: built with nvcc,
run on the CPU (no GPU call is made)."""
import os
import subprocess

import pytest

from sparse_long_context_page_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def native(tmp_path_factory):
    """Builds and runs tests/native/<name>.cu; fails with its output where it ends with another status than 0."""
    out = tmp_path_factory.mktemp("native")

    def run(name, *args):
        exe = str(out / name)
        if not os.path.exists(exe):
            subprocess.run([build.nvcc()] + build.ARCH + ["-O2", "-std=c++17", "--expt-relaxed-constexpr", "-I", build.CSRC,
                            os.path.join(HERE, "native", name + ".cu"), "-o", exe, "-lpthread"], check=True)
        done = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=300)
        assert done.returncode == 0, done.stdout + done.stderr

    return run


def test_prefix_plan_stays_in_its_workspace(native):
    """Every partial slot of random group tables, empty prefixes among them, for every head count."""
    native("plan_bounds", 4000)


def test_what_stays_zero_lies_apart_from_every_calls_scratch(native):
    """Layouts of calls for different sizes on one workspace."""
    native("workspace_layout", 20000)


def test_a_kernels_shared_memory_limit_is_never_lowered(native):
    """Two threads' first calls with different sizes."""
    native("smem_limit")
