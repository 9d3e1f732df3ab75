"""csa2_prefix_attn where the prefix is worked through in several bands (few row blocks
over images of a long prefix), against its 64-bit definition."""
import pytest
import torch

from dense_ref import D, H, PAGE
from test_gpu_prefix import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp4_kv_cache_quantize_b200 import csa2
    return csa2


def bands(c):
    """Bands of a call, out of its workspace: 515 floats a partial's row, 65,600 bytes an
    image; a partial of 64 rows per row block and band, and per CTA, then the own ones."""
    ctas = min(torch.cuda.get_device_properties(0).multi_processor_count, 192)
    tiles, blocks = -(-c.prefix // 64), -(-c.B * c.nq * H // 64)
    own = (c.B * -(-c.nq // 4) + ctas) * H * min(c.nq, 4)
    rows = (c.attn.workspace_size() - 256 - tiles * 65600) // (515 * 4) - own
    assert rows > 0 and rows % 64 == 0
    n = rows // 64 - ctas
    assert n % blocks == 0
    return n // blocks


# 64 sequences with one query each (some end inside the prefix, one is empty); sequences
# with several queries, rows contiguous, a prefix that ends inside a tile
WIDE = dict(n_rows=[12230 + 7 * b if b % 5 else 12230 - 150 * b for b in range(63)] + [0], prefix=12224)


@pytest.mark.parametrize("window", [None, [(13 * b) % 129 for b in range(64)]])
def test_one_query_each(lib, orc, window):
    c = Case(lib, orc, window=window, seed=41, **WIDE)
    assert bands(c) > 4
    c.check()


@pytest.mark.parametrize("n_rows,prefix,nq,window,paged", [
    ([12500, 12400, 12340, 12333, 12000, 9, 12600, 12700], 12333, 8, [135, 8, 0, 100, 77, 3, 128, 60], False),
    ([2700] * 8 + [2559 + b for b in range(8)], 2550, 16, [143] * 16, True),
    ([3000, 2900, 2800, 2720], 2710, 64, None, False),
])
def test_several_queries(lib, orc, n_rows, prefix, nq, window, paged):
    c = Case(lib, orc, n_rows, prefix, nq, window=window, paged=paged, seed=42)
    assert bands(c) > 1
    c.check()


def test_nan_and_unmapped_pages_of_later_bands(lib, orc):
    """A NaN row is met by the queries that see it, a page that is not mapped by none; the
    next call, without them, finds nothing of either."""
    c = Case(lib, orc, [2700, 2690, 2400, 2650], 2624, 64, seed=43)
    assert bands(c) > 1
    clean = c.reference()
    at = c.page_table[0].long()[2500 // PAGE] * PAGE + 2500 % PAGE
    d, keep = c.d, c.d["scales"].clone()
    d["scales"][at, 9] = 0x7F
    first = c.run().clone()
    d["scales"].copy_(keep)
    table = d["page_table"][0, 30].clone()
    d["page_table"][0, 30] = -1
    second = c.run().clone()
    d["page_table"][0, 30] = table
    third = c.run().clone()
    with pytest.raises(lib.Csa2Error) as e:
        lib.csa2_sync_status(c.ws)
    assert e.value.status == 7
    clean.check(third)
    out = first.view(4, 64, H, D).float().cpu().double()
    sees = (torch.tensor([2700, 2690, 2400, 2650])[:, None] - 63 + torch.arange(64) > 2500)
    assert out[sees].isnan().all()
    want, tol = clean.out.view(4, 64, H, D), clean.tol.view(4, 64, H, D)
    assert ((out - want)[~sees].abs() <= tol[~sees] + 1e-30).all()
    c.page_table = torch.cat([c.page_table[:, :30], c.page_table[:, 31:]], 1)
    c.n_rows, c.prefix = c.n_rows - PAGE, c.prefix - PAGE
    c.reference().check(second)


def test_the_same_every_time(lib, orc):
    c = Case(lib, orc, window=[128] * 64, seed=44, **WIDE)
    first = c.run().clone()
    for _ in range(5):
        c.attn.out.zero_()
        assert torch.equal(c.run(), first)
    lib.csa2_sync_status(c.ws)
