"""Index arithmetic that the kernels and the host share, checked on the host."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def host_check(tmp_path, name):
    """Build tests/host/<name>.cpp against the kernels' headers as plain C++ and run it."""
    exe = tmp_path / name
    subprocess.run(["g++", "-O2", "-std=c++17", "-I" + os.path.join(ROOT, "paged_kv_cache_292_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "host", name + ".cpp"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.startswith("ok")


def test_rows_of_an_allocation(tmp_path):
    host_check(tmp_path, "rows_check")


def test_walks_partials_and_cuts(tmp_path):
    """Tiles, partial slots and cuts of every walk, range by range, and the checks that the kernels make before they
    use a stage's sequence or a sequence's cut as an index."""
    host_check(tmp_path, "walk_check")


def test_scratch_of_the_librarys_own_under_threads(tmp_path):
    """pa_host.cu against a stand-in for the CUDA runtime: a call's buffer is its own up to its last launch."""
    exe = tmp_path / "scratch_check"
    here = os.path.join(ROOT, "tests", "host")
    csrc = os.path.join(ROOT, "paged_kv_cache_292_gb300", "csrc")
    subprocess.run(["g++", "-O1", "-std=c++17", "-pthread", "-I" + os.path.join(here, "fake"), "-I" + csrc, "-x", "c++",
                    os.path.join(here, "scratch_check.cpp"), os.path.join(csrc, "pa_host.cu"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.startswith("ok")


def test_plans_of_every_batch_shape(tmp_path):
    """No shape that the entry points take is refused for its launch plan, and every plan fits the SM."""
    exe = tmp_path / "plan_check"
    here = os.path.join(ROOT, "tests", "host")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I" + os.path.join(here, "fake"),
                    "-I" + os.path.join(ROOT, "paged_kv_cache_292_gb300", "csrc"), os.path.join(here, "plan_check.cpp"),
                    "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.startswith("ok")
