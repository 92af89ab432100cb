"""Sorts that need more than 48 KB of shared memory, also from several host threads."""
from __future__ import annotations

import os
import shutil
import subprocess

import numpy as np
import pytest

from conftest import ROOT
from gpu_util import ccl
from oracle import experts
from test_gpu_experts import host, run_sort


# CTAs of 8 to 32 warps, clusters up to 16 of them, up to 136 KB each
@pytest.mark.gpu
@pytest.mark.parametrize("tokens,k,num", [([100000], 2, 1024), ([9000, 70000], 1, 1000), ([40000, 10], 1, 500), ([300], 8, 1024)])
def test_large_sorts_of_many_experts(tokens, k, num):
    rng = np.random.default_rng(num)
    ids = [rng.integers(-1, num + 1, (t, k)).astype(np.int32) for t in tokens]
    offsets, rows = run_sort(ccl(), ids, num)
    for r, i in enumerate(ids):
        want = experts.sort(i, num)
        np.testing.assert_array_equal(host(offsets[r]), want[0])
        np.testing.assert_array_equal(host(rows[r]), want[1])


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    from a2a_ring_ordered_gb300 import build

    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc is not installed")
    lib, cuda = os.path.abspath(build.build()), os.path.dirname(os.path.dirname(build.nvcc()))
    out = str(tmp_path_factory.mktemp("c_abi") / "sort_threads")
    cmd = [gcc, "-std=c11", "-Wall", "-Wextra", "-Werror", "-O1", "-pthread", "-I", build.INCLUDE, "-I", os.path.join(cuda, "include"),
           os.path.join(ROOT, "tests", "c_abi", "sort_threads.c"), "-o", out, lib, f"-Wl,-rpath,{os.path.dirname(lib)}",
           "-L", os.path.join(cuda, "lib64"), "-lcudart", f"-Wl,-rpath,{os.path.join(cuda, 'lib64')}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out


def test_program_of_sorting_threads_links(exe):
    assert os.access(exe, os.X_OK)


@pytest.mark.gpu
def test_sorts_of_several_host_threads(exe):
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
