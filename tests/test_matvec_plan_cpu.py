"""The layout of lhcal_matvec's products over warps and shared memory, checked on the host over the sizes
that the call takes (tests/c/matvec_plan.cpp)."""
import os
import shutil
import subprocess

import pytest


@pytest.fixture(scope="module")
def program(tmp_path_factory, root_dir):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = tmp_path_factory.mktemp("plan") / "matvec_plan"
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(root_dir, "include"),
                        "-I", os.path.join(root_dir, "scale_calibration_lh_b200", "csrc"),
                        os.path.join(root_dir, "tests", "c", "matvec_plan.cpp"), "-o", str(exe)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    return str(exe)


@pytest.fixture(scope="module")
def report(program):
    r = subprocess.run([program], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "checked" in r.stdout, r.stdout + r.stderr
    return r.stdout


@pytest.mark.parametrize("what", [
    "warps", "channels", "passes", "stages", "shared memory", "room", "stage alignment", "weights read", "codes read", "sums",
    "list alignment", "scan alignment", "counts", "sums below the lists", "lists",
    "stage owners",  # a stage is always read by the same warps: a wait by parity needs a warp that saw the lap before
])
def test_plan(report, what):
    assert f"\n{what}: " not in "\n" + report, report


def test_the_gpu_tests_sizes_reach_every_share_of_rows(program):
    """Warps over the channels and over the rows, and stages, of sizes that the GPU tests multiply: rows that
    one warp takes, and that 2, 3, 5, 6 and 8 share."""
    sizes = {(0, 1, 1, 40000, 768): (3, 6, 12), (0, 2, 1, 40000, 1024): (4, 5, 10), (0, 8, 1, 40003, 1040): (5, 4, 8),
             (0, 1, 1, 40000, 1536): (6, 3, 9), (0, 1, 1, 40000, 2560): (10, 2, 8), (0, 2, 1, 40000, 512): (2, 8, 8),
             (0, 1, 1, 38000, 5120): (20, 1, 3), (1, 640, 32, 1280, 2560): (10, 2, 6), (1, 80, 40, 1280, 2560): (10, 2, 8),
             (1, 640, 64, 1280, 768): (3, 6, 12), (1, 10, 32, 37, 272): (2, 1, 2)}
    r = subprocess.run([program] + [str(v) for k in sizes for v in k], capture_output=True, text=True, timeout=60)
    got = [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]
    assert dict(zip(sizes, got)) == sizes
