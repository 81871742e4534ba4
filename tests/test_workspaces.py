"""The scratch of decode calls on the CPU: its layout, and the sizes handed out."""

import os
import subprocess

import pytest

from paged_kv_cache_292_gb300 import binding
from paged_kv_cache_292_gb300 import build as pa_build


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return binding.load()


@pytest.mark.parametrize("check", ["workspace_check", "scaled_plan_check"])
def test_host_check(tmp_path, check):
    """Partials of no shape reach another's merge tickets, everything stays inside the size handed out; plans over int8
    pools hold their scales."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = tmp_path / check
    subprocess.run(["g++", "-O2", "-std=c++17", "-I" + os.path.join(root, "paged_kv_cache_292_gb300", "csrc"),
                    "-I" + os.path.join(root, "tests", "host", "fake"),
                    os.path.join(root, "tests", "host", check + ".cpp"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.startswith("ok")


@pytest.mark.parametrize("Q", [1, 4])
def test_sizes_grow_with_the_batch(lib, Q):
    """A buffer sized for the larger of two batches holds the smaller, whatever differs."""
    last = 0
    for S, R in ((1, 1), (4, 1), (4, 20), (300, 20), (300, 513), (300, 514), (5000, 514), (5000, 4096)):
        size = binding.pa_decode_mq_workspace_size(S, Q, 8, 8, 64, R)
        assert size >= last and size % 256 == 0
        last = size
