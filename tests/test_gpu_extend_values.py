"""csa2_cache_extend of entries that hold infinities and NaN: few tokens and many give
the bits of csa2_rope_rows followed by csa2_quantize_fp4, and the other tokens get what
they would without them."""
import pytest
import torch

from dense_ref import D, W, rows_of
from test_gpu_extend import Case

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
# token, channel: in front of the rotated channels, among them, and last
BAD = [(0, 0, NAN), (1, 17, INF), (2, 18, -INF), (3, 100, NAN), (3, 101, INF), (4, 448, NAN), (5, 449, -INF),
       (6, 511, INF), (7, 447, -NAN), (9, 200, -INF), (9, 460, NAN), (11, 510, INF), (11, 511, -INF)]


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp4_kv_cache_quantize_b200 import csa2
    return csa2


@pytest.mark.parametrize("dims", [0, 64])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("T", [40, 700])
def test_rows_that_are_not_finite(lib, orc, T, halves, dims):
    c = Case(lib, orc, [T], [10], L=0, dims=dims, halves=halves)
    for tok, ch, v in BAD:
        c.x[tok, ch] = c.x[T - 1 - tok, ch] = v
    c.x[8] = NAN
    c.x[10, :16] = NAN  # a whole group
    c.d["x"].copy_(c.x)
    x = c.d["x"].clone()
    if dims:
        rope = lib.Rope(c.d["tab"], lib.ROPE_HALVES if halves else lib.ROPE_PAIRS)
        lib.csa2_rope_rows(rope, x.view(T, 1, D), c.at.int().cuda(), x.view(T, 1, D), c.ws)
    codes = torch.empty((T, 256), dtype=torch.uint8, device="cuda")
    scales = torch.empty((T, 32), dtype=torch.uint8, device="cuda")
    lib.csa2_quantize_fp4(x, codes, scales)
    c.run()
    lib.csa2_sync_status(c.ws)
    row = rows_of(0, 10, 10 + T, c.stride, c.page_table)
    assert torch.equal(c.d["codes"][row.cuda()], codes)
    assert torch.equal(c.d["scales"][row.cuda()], scales)
    # the keys: NaN or infinite for those tokens, as ever for the others
    keys = c.d["idx_k"].cpu()[row]
    bad = ~torch.isfinite(c.x.float()).all(-1)
    assert (~torch.isfinite(keys[bad].float())).all()
    exact, bound, _ = c.expect()
    assert ((keys[~bad].double() - exact[~bad]).abs() <= bound[~bad]).all()


@pytest.mark.parametrize("T", [40, 700])
def test_window_entries_that_are_not_finite(lib, orc, T):
    """Infinities saturate, NaN stays NaN, few tokens and many."""
    c = Case(lib, orc, [T], [10], L=2, dims=0, entries=False)
    c.x_swa[1, T - 5, 3], c.x_swa[1, T - 5, 4], c.x_swa[0, T - 1, 511] = INF, -INF, NAN
    c.d["x_swa"].copy_(c.x_swa)
    c.run()
    lib.csa2_sync_status(c.ws)
    c.x_swa[0, T - 1, 511] = 0.0
    p = int(c.swa_pos[0])
    c.expect()
    got = c.d["swa"].cpu()
    slot = (p + T - 1) % W
    assert int(got[0, 0, slot, 511]) & 0x7F == 0x7F
    got[0, 0, slot, 511] = c.swa[0, 0, slot, 511]
    assert torch.equal(got, c.swa)
