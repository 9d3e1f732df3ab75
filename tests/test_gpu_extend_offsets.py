"""csa2_cache_extend with token offsets that descend: a sequence is extended by its
whole run or left as it was (rows, windows, counters), and the rest is extended."""
import pytest
import torch

from dense_ref import PAGE
from test_gpu_extend import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp4_kv_cache_quantize_b200 import csa2
    return csa2


def owner(cu, i):
    """Where a binary search for token i in the offsets ends."""
    lo, hi = 0, len(cu) - 1
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if cu[mid] <= i else (lo, mid)
    return lo if cu[lo] <= i < cu[lo + 1] else -1


def left_alone(cu, total):
    """Sequences whose run is not theirs as a whole."""
    own = [owner(cu, i) for i in range(total)]
    return {b for b in range(len(cu) - 1)
            if not 0 <= cu[b] <= cu[b + 1] <= total or any(own[i] != b for i in range(cu[b], cu[b + 1]))}


FEW = [([10, 0, 8], {2: 4}), ([4, 2, 0, 6], {2: 20}), ([10, 0, 7], {2: 5}), ([3, 4, 5], {1: 9, 2: 1})]
MANY = [([700, 0, 300], {2: 350}), ([40, 500, 0, 90, 20], {2: 900, 4: 545}), ([1] * 600, {301: 250, 77: 79}),
        ([2] * 200 + [300, 1], {50: 99, 200: 10}), ([400, 1, 400], {2: 0})]


@pytest.mark.parametrize("kw", [dict(L=2), dict(L=1, entries=False), dict(L=0, paged=False)])
@pytest.mark.parametrize("counts,moved", FEW + MANY)
def test_descending_offsets(lib, orc, counts, moved, kw):
    c = Case(lib, orc, counts, [(37 * b) % 90 for b in range(len(counts))], pos="given", **kw)
    for b, v in moved.items():
        c.cu[b] = v
    c.d["cu"].copy_(c.cu)
    cu = c.cu.tolist()
    alone = left_alone(cu, c.T)
    room = PAGE * c.page_table.shape[1] if c.page_table is not None else c.stride
    if c.entries:  # a run that grew may not fit: then it is left alone too
        alone |= {b for b in range(c.B) if c.n0[b] + cu[b + 1] - cu[b] > room}
    assert 0 < len(alone) < c.B
    c.counts = [max(0, cu[b + 1] - cu[b]) for b in range(c.B)]
    c.run()
    with pytest.raises(lib.Csa2Error) as e:
        lib.csa2_sync_status(c.ws)
    assert e.value.status == 7
    c.check(refused=alone)
