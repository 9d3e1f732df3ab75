"""How the shared-prefix attention cuts its work (csrc/prefix_plan.cuh), on the
CPU: no tile is lost or done twice, no two partials share workspace rows, and
the shares are equal to within one tile."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    out = tmp_path_factory.mktemp("plan") / "libplan.so"
    inc = os.environ.get("CUDA_HOME", "/usr/local/cuda") + "/include"
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I" + inc,
                           "-I" + os.path.join(ROOT, "fp4_kv_cache_quantize_b200", "csrc"),
                           "-o", str(out), os.path.join(ROOT, "tests", "plan_ref.cpp")])
    f = ctypes.CDLL(str(out)).plan_check
    i64 = ctypes.POINTER(ctypes.c_int64)
    f.argtypes = [ctypes.c_int] * 4 + [ctypes.POINTER(ctypes.c_int32), ctypes.c_int, ctypes.c_int,
                                       i64, i64]

    def check(batch, nq, prefix, max_rows, n_rows, window, grid):
        most, mean = ctypes.c_int64(), ctypes.c_int64()
        rc = f(batch, nq, prefix, max_rows, (ctypes.c_int32 * batch)(*n_rows), window, grid,
               ctypes.byref(most), ctypes.byref(mean))
        assert rc == 0, (rc, batch, nq, prefix, max_rows, window, grid)
        return most.value, mean.value
    return check


@pytest.mark.parametrize("window", [0, 1])
@pytest.mark.parametrize("batch,nq,prefix,own", [
    (1, 1, 0, 0), (1, 1, 0, 1), (1, 1, 1, 0), (4, 1, 2048, 64), (7, 3, 5003, 300), (64, 1, 131072, 2000),
    (2, 256, 16384, 700), (5, 5, 100, 129), (1, 1024, 640, 1), (1024, 1, 128, 300), (3, 4, 1 << 19, 9)])
def test_plan_covers_every_tile_once(plan, batch, nq, prefix, own, window):
    rng = random.Random(batch * 1000 + nq)
    for grid in (1, 2, 7, 148, 192):
        n_rows = [prefix + rng.randint(0, own) for _ in range(batch)]
        most, mean = plan(batch, nq, prefix, prefix + own, n_rows, window, grid)
        assert most <= mean + 17  # a share plus at most one tile (of 16) and the rounding


def test_plan_with_counts_out_of_range(plan):
    """Negative and overlong counts are clamped; sequences may end inside the prefix."""
    for grid in (1, 13, 148):
        plan(4, 2, 1000, 1500, [-5, 200, 1 << 30, 1000], 1, grid)
        plan(3, 1, 0, 0, [0, 7, -1], 0, grid)
