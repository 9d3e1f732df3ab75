"""Which tokens the cache extension takes for which sequence (csrc/extend_runs.cuh),
on the CPU: a run in order owns each of its tokens and no other, whatever the
offsets of the others; a descent is never overlooked."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def runs(tmp_path_factory):
    out = tmp_path_factory.mktemp("runs") / "libruns.so"
    inc = os.environ.get("CUDA_HOME", "/usr/local/cuda") + "/include"
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I" + inc,
                           "-I" + os.path.join(ROOT, "fp4_kv_cache_quantize_b200", "csrc"),
                           "-o", str(out), os.path.join(ROOT, "tests", "runs_ref.cpp")])
    lib = ctypes.CDLL(str(out))

    def both(cu, total):
        """({sequence: its tokens} of the runs in order, [sequence of each token])."""
        n = len(cu) - 1
        c, lo, hi = (ctypes.c_int32 * len(cu))(*cu), ctypes.c_int32(), ctypes.c_int32()
        ok = {}
        for b in range(n):
            r = lib.run_of(c, n, total, b, ctypes.byref(lo), ctypes.byref(hi))
            assert r != 2, "one thread and 32 lanes disagree"
            if r:
                ok[b] = list(range(lo.value, hi.value))
        return ok, [lib.seq_of(c, n, total, i) for i in range(total)]
    return both


def whole(ok, seq):
    for b, tokens in ok.items():
        assert all(seq[i] == b for i in tokens), (b, tokens)
    assert all(b == -1 or i in ok[b] for i, b in enumerate(seq)), (ok, seq)


def test_offsets_in_order(runs):
    """Every run is taken, empty ones and a padded tail included."""
    rng = random.Random(1)
    for _ in range(300):
        counts = [rng.choice([0, 0, 1, 2, 7, 40]) for _ in range(rng.randint(1, 70))]
        cu = [0]
        for c in counts:
            cu.append(cu[-1] + c)
        ok, seq = runs(cu, cu[-1] + 5)
        assert ok == {b: list(range(cu[b], cu[b + 1])) for b in range(len(counts))}
        assert seq == [b for b, c in enumerate(counts) for _ in range(c)] + [-1] * 5


@pytest.mark.parametrize("cu,total,want", [
    ([0, 10, 4, 12], 12, [0]),         # [4, 12) would share 4..9 with [0, 10)
    ([0, 4, 20, 6, 12], 12, [0]),      # a search for 6..11 ends at the second, [4, 20)
    ([0, 10, 5, 12], 12, [0]),
    ([0, 3, 2, 2, 9], 9, [2, 3]),      # token 2 is the last one's: the search meets offset 2 first
    ([3, 5, 9], 9, [1]),               # does not start at 0
    ([0, -2, 9], 9, []),
    ([0, 4, 10], 9, [0]),              # ends behind the tokens
])
def test_runs_that_cross(runs, cu, total, want):
    ok, seq = runs(cu, total)
    assert sorted(ok) == want
    whole(ok, seq)


def test_any_offsets(runs):
    """Random disorder: whole runs or none, never a token twice, and the sequence at
    each descent is refused."""
    rng = random.Random(2)
    refused = 0
    for _ in range(20000):
        n, total = rng.randint(1, 12), rng.randint(1, 40)
        cu = sorted(rng.randint(0, total) for _ in range(n + 1))
        cu[0] = 0
        for _ in range(rng.randint(1, 3)):
            cu[rng.randrange(n + 1)] = rng.randint(-3, total + 3)
        ok, seq = runs(cu, total)
        whole(ok, seq)
        assert all(b not in ok for b in range(n) if cu[b + 1] < cu[b] or cu[b + 1] > total or cu[b] < 0)
        refused += any(cu[b] <= cu[b + 1] <= total and cu[b] >= 0 and b not in ok for b in range(1, n))
    assert refused > 100  # runs that only the others' offsets rule out
