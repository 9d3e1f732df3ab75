"""GPU parity of csa2_rope_rows and csa2_cache_extend.

Rotated rows, FP4 rows, window rings and counters are compared bit for bit with
the 64-bit reference rounded as the header says (the reference's two products
and one sum differ from a fused sum by 2^-53, which no rounding to bf16 sees
outside of a 2^-29 share of cases).  Indexer keys lie within half a bf16 step
(2^-8 relative) plus the fp32 summation bound of their exact value."""
import numpy as np
import pytest
import torch

from dense_ref import D, DI, PAGE, W, dequant, rotate, rows_of, table, to_bf16

pytestmark = pytest.mark.gpu
PROJ_ERR = 520 * 2.0 ** -24  # a sum of 512 products in fp32, in any order


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp4_kv_cache_quantize_b200 import csa2
    return csa2


def ws_of(lib):
    return lib.workspace(lib.WS_HEADER)


# ------------------------------------------------------------------ rotation
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("rows,heads,ch,dims", [
    (1, 1, 32, 32), (1, 16, 512, 64), (37, 8, 64, 64), (5, 3, 200, 96), (2, 1, 512, 512), (300, 16, 512, 64),
    (4096, 1, 64, 32)])
def test_rope_rows(lib, rows, heads, ch, dims, halves, inverse):
    g = torch.Generator().manual_seed(rows * 7 + dims)
    x = torch.randn((rows, heads, ch), generator=g).bfloat16()
    x[0, 0, -1] = 0.0
    tab = table(5000, dims)
    pos = torch.randint(0, 5000, (rows,), generator=g, dtype=torch.int32)
    pos[0] = 4999
    want = to_bf16(rotate(x, tab[pos.long()], halves, inverse))
    rope = lib.Rope(tab.cuda(), lib.ROPE_HALVES if halves else lib.ROPE_PAIRS)
    xd, ws = x.cuda(), ws_of(lib)
    y = torch.full_like(xd, 7.0)
    lib.csa2_rope_rows(rope, xd, pos.cuda(), y, ws, inverse=inverse)
    lib.csa2_sync_status(ws)
    assert torch.equal(xd.cpu(), x)
    assert torch.equal(y.cpu(), want)
    lib.csa2_rope_rows(rope, xd, pos.cuda(), xd, ws, inverse=inverse)  # in place
    lib.csa2_sync_status(ws)
    assert torch.equal(xd.cpu(), want)


def test_rope_there_and_back(lib):
    """The inverse undoes the rotation to one rounding of each turn."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn((64, 16, 512), generator=g).bfloat16().cuda()
    rope = lib.Rope(table(1000, 64).cuda())
    pos, ws = torch.arange(64, dtype=torch.int32).cuda() * 13, ws_of(lib)
    y, z = torch.empty_like(x), torch.empty_like(x)
    lib.csa2_rope_rows(rope, x, pos, y, ws)
    lib.csa2_rope_rows(rope, y, pos, z, ws, inverse=True)
    a, b = x.double().cpu().view(-1, 512), z.double().cpu().view(-1, 512)
    assert torch.equal(a[:, :448], b[:, :448])
    pair = a[:, 448:].view(-1, 32, 2).norm(dim=-1, keepdim=True)  # a turn rounds each channel by 2^-8 of itself
    assert ((a - b)[:, 448:].view(-1, 32, 2).abs() <= pair * (2.0 ** -8 * 1.5 + 2.0 ** -8)).all()


def test_rope_positions_outside_the_table(lib):
    x = torch.randn((4, 1, 64)).bfloat16()
    tab, ws = table(10, 64), ws_of(lib)
    rope, y = lib.Rope(tab.cuda()), torch.empty_like(x).cuda()
    lib.csa2_rope_rows(rope, x.cuda(), torch.tensor([0, -3, 10, 9], dtype=torch.int32).cuda(), y, ws)
    with pytest.raises(lib.Csa2Error) as e:
        lib.csa2_sync_status(ws)
    assert e.value.status == 7
    assert torch.equal(y.cpu(), to_bf16(rotate(x, tab[[0, 0, 9, 9]], False)))


# ----------------------------------------------------------------- extension
class Case:
    """A cache, windows and one extension of them, on the device and on the host."""

    def __init__(self, lib, orc, counts, n0, *, paged=True, L=2, dims=64, idx_dims=32, halves=False, pos="own",
                 tail=0, entries=True, seed=0, cu=True, shuffle_extra=3):
        self.lib, self.orc, self.halves = lib, orc, halves
        g = torch.Generator().manual_seed(seed)
        B = len(counts)
        self.B, self.L, self.counts, self.n0 = B, L, list(counts), list(n0)
        T = sum(counts) + tail
        self.T = T
        ends = [n + c for n, c in zip(n0, counts)]
        if paged:
            mp = max(-(-e // PAGE) for e in ends) + 1
            pages = B * mp + shuffle_extra
            self.page_table = torch.randperm(pages, generator=g)[:B * mp].int().view(B, mp)
            self.stride, self.pool = 0, pages * PAGE
        else:
            self.page_table, self.stride = None, -(-max(ends) // PAGE) * PAGE + PAGE
            self.pool = B * self.stride
        r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.x = (r(T, D) * 10 ** (torch.rand((T, 1), generator=g) * 6 - 3)).bfloat16()
        self.w = (r(D, DI) * D ** -0.5).bfloat16()
        self.codes = torch.randint(0, 256, (self.pool, 256), generator=g, dtype=torch.uint8)
        self.scales = torch.randint(0, 120, (self.pool, 32), generator=g, dtype=torch.uint8)
        self.idx_k = r(self.pool, DI).bfloat16()
        self.n_rows = torch.tensor(n0, dtype=torch.int32)
        self.swa_pos = torch.tensor([n * 2 + 5 for n in n0], dtype=torch.int32)
        self.swa_len = self.swa_pos.clamp(max=W)
        self.x_swa = (r(L, T, D) * 100).bfloat16()  # some beyond E4M3's 448
        self.swa = torch.randint(0, 120, (L, B, W, D), generator=g, dtype=torch.uint8)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
        start = torch.repeat_interleave(self.n_rows, torch.tensor(counts))
        swa_start = torch.repeat_interleave(self.swa_pos, torch.tensor(counts))
        off = torch.cat([torch.arange(c, dtype=torch.int32) for c in counts]) if counts else None
        n_pos = 3 * (max(ends) + 200)
        pad = lambda v: torch.cat([v, torch.zeros(tail, dtype=torch.int32)]).int()  # noqa: E731
        if pos == "own":
            self.pos, self.at, self.at_swa = None, start + off, swa_start + off
        else:
            self.pos = pad((start + off) * 2 + 1)
            self.at = self.at_swa = self.pos[:sum(counts)]
        self.tab = table(n_pos, dims) if dims else None
        self.tab_idx = table(n_pos, idx_dims, base=1000.0) if idx_dims else None
        self.entries = entries
        d = {}
        for k in ("x", "w", "codes", "scales", "idx_k", "n_rows", "swa_pos", "swa_len", "x_swa", "swa", "cu", "pos",
                  "tab", "tab_idx", "page_table"):
            v = getattr(self, k)
            d[k] = None if v is None else v.cuda()
        self.d = d
        style = lib.ROPE_HALVES if halves else lib.ROPE_PAIRS
        kv = lib.KVCache(d["codes"], d["scales"], d["idx_k"], d["n_rows"], max_rows=max(ends),
                         seq_stride=self.stride, page_table=d["page_table"])
        rope = lib.Rope(d["tab"], style) if dims else None
        win = dict(x_swa=d["x_swa"], swa=d["swa"], swa_pos=d["swa_pos"], swa_len=d["swa_len"],
                   rope_swa=rope) if L else {}
        self.ext = lib.CacheExtend(kv, d["x"] if entries else None, d["w"] if entries else None,
                                   cu_tokens=d["cu"] if cu else None, pos=d["pos"],
                                   rope=rope, rope_idx=lib.Rope(d["tab_idx"], style) if idx_dims else None, **win)
        self.ws = ws_of(lib)

    def run(self, stream=None):
        self.lib.csa2_cache_extend(self.ext, self.ws, stream=stream)

    def expect(self, refused=()):
        """Applies the extension to the host copies; returns the indexer keys'
        exact values and bounds at the rows written."""
        exact, bound, at = [], [], []
        for b, c in enumerate(self.counts):
            if b in refused or c == 0:
                continue
            t = slice(int(self.cu[b]), int(self.cu[b]) + c)
            if self.entries:
                n0 = int(self.n_rows[b])
                row = rows_of(b, n0, n0 + c, self.stride, self.page_table)
                x = self.x[t]
                if self.tab is not None:
                    x = to_bf16(rotate(x, self.tab[self.at[t].long()], self.halves))
                codes, scales = self.orc.quantize_fp4(x.view(torch.int16).numpy().view(np.uint16))
                self.codes[row], self.scales[row] = torch.from_numpy(codes), torch.from_numpy(scales)
                xd, wd = self.x[t].double(), self.w.double()
                k, err = xd @ wd, PROJ_ERR * (xd.abs() @ wd.abs())
                if self.tab_idx is not None:
                    cs = self.tab_idx[self.at[t].long()]
                    k = rotate(k, cs, self.halves)
                    # |c| e1 + |s| e2, and the rounding of the rotated sum to fp32
                    err = rotate(err, torch.stack((cs[..., 0].abs(), -cs[..., 1].abs()), -1), self.halves).maximum(
                        rotate(err, cs.abs(), self.halves)) + k.abs() * 2.0 ** -23
                exact.append(k), bound.append(err + k.abs() * 2.0 ** -8), at.append(row)
                self.n_rows[b] += c
            if self.L:
                keep = slice(max(t.start, t.stop - W), t.stop)
                v = self.x_swa[:, keep]
                if self.tab is not None:
                    v = to_bf16(rotate(v.transpose(0, 1), self.tab[self.at_swa[keep].long()], self.halves)).transpose(0, 1)
                slot = (int(self.swa_pos[b]) + torch.arange(keep.start - t.start, c)) % W
                self.swa[:, b, slot] = v.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                self.swa_pos[b] += c
                self.swa_len[b] = min(int(self.swa_pos[b]), W)
        return [torch.cat(v) if v else None for v in (exact, bound, at)]

    def check(self, refused=()):
        before = self.idx_k.clone()
        exact, bound, at = self.expect(refused)
        for k in ("codes", "scales", "n_rows", "swa", "swa_pos", "swa_len"):
            assert torch.equal(self.d[k].cpu(), getattr(self, k)), k
        got = self.d["idx_k"].cpu()
        if at is not None:
            assert ((got[at].double() - exact).abs() <= bound).all()
            self.idx_k[at] = got[at]
        assert torch.equal(got, self.idx_k), "other rows' keys changed"
        assert at is None or not torch.equal(before, self.idx_k)


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("counts,n0,kw", [
    ([1], [0], dict(cu=False)),
    ([1, 1, 1], [63, 64, 1000], dict(cu=False, pos="given", L=5)),
    ([3, 0, 130, 1], [62, 10, 0, 127], dict()),
    ([300, 17], [1, 63], dict(dims=128, idx_dims=64, pos="given", tail=9)),
    ([65, 64, 63], [63, 0, 1], dict(dims=512, idx_dims=0, L=0)),
    ([40, 200], [5, 0], dict(dims=0, idx_dims=64, L=1)),
    ([129, 127, 128], [0, 0, 0], dict(dims=32, idx_dims=0, entries=False)),
    ([700, 1], [123, 77], dict(dims=64, idx_dims=64, L=1, tail=50)),
    ([513], [0], dict(dims=512, idx_dims=64, L=0, pos="given")),
    ([1, 0, 1500, 63, 64, 65, 0, 0, 2], [64, 9, 100, 0, 1, 63, 5, 0, 200], dict(dims=32, idx_dims=32, tail=70)),
    ([0, 0, 900, 0], [0, 1, 2, 3], dict(dims=0, idx_dims=0, pos="given", tail=1)),
    ([600, 300], [5, 0], dict(dims=96, idx_dims=0, entries=False, L=3)),
])
def test_extend(lib, orc, counts, n0, kw, paged, halves):
    c = Case(lib, orc, counts, n0, paged=paged, halves=halves, **kw)
    c.run()
    lib.csa2_sync_status(c.ws)
    c.check()


def test_extend_many_sequences(lib, orc):
    rng = np.random.default_rng(5)
    counts = [int(v) for v in rng.integers(0, 9, 333)]
    n0 = [int(v) for v in rng.integers(0, 200, 333)]
    c = Case(lib, orc, counts, n0, L=1, pos="given")
    c.run()
    lib.csa2_sync_status(c.ws)
    c.check()


@pytest.mark.parametrize("dims", [0, 32])
def test_extend_packs_every_finite_bf16(lib, orc, dims):
    """Both encoders (few and many tokens, rotated by position 0 or not) against
    the oracle's on every finite bf16 value, next to group maxima that put the
    scale anywhere, ties of every kind included."""
    bits = torch.arange(1 << 16, dtype=torch.int32)
    bits = bits[(bits & 0x7F80) != 0x7F80].to(torch.int16)  # finite
    g = torch.Generator().manual_seed(1)
    vals = bits[torch.randperm(len(bits), generator=g)][:65024 // 15 * 15].view(-1, 15)
    big = torch.randint(0, 0x7F80, (len(vals), 1), generator=g).to(torch.int16)
    x = torch.cat([vals, big], 1)
    small = torch.randint(0x3C00, 0x4300, (len(vals), 16), generator=g).to(torch.int16)  # ties near 1
    x = torch.cat([x, small]).view(-1)
    x = x[:x.numel() // D * D].view(-1, D)
    for part in (x, x[:300]):  # more than, and no more than, the few tokens' limit
        T = len(part)
        c = Case(lib, orc, [T], [0], L=0, dims=dims, idx_dims=0, pos="given")
        c.x = part.view(torch.bfloat16)
        c.d["x"].copy_(c.x)
        c.pos.zero_()
        c.d["pos"].zero_()
        c.run()
        lib.csa2_sync_status(c.ws)
        codes, scales = orc.quantize_fp4(part.numpy().view(np.uint16))
        row = rows_of(0, 0, T, c.stride, c.page_table)
        assert torch.equal(c.d["codes"].cpu()[row], torch.from_numpy(codes))
        assert torch.equal(c.d["scales"].cpu()[row], torch.from_numpy(scales))


def test_extend_every_group_maximum(lib, orc):
    """The many tokens' encoder with every positive finite bf16 as a group's maximum:
    each scale, ties between two of them included."""
    top = torch.arange(1, 0x7F80, dtype=torch.int32)
    top = torch.cat([top, top[:32 * 1020 - len(top)]]).to(torch.int16).view(-1, 1)
    g = torch.Generator().manual_seed(2)
    part = (torch.rand((len(top), 15), generator=g) * 2 - 1) * top.view(torch.bfloat16).float()
    x = torch.cat([part.bfloat16(), top.view(torch.bfloat16)], 1).view(-1, D)
    c = Case(lib, orc, [len(x)], [0], L=0, dims=0, idx_dims=0)
    c.x = x
    c.d["x"].copy_(x)
    c.run()
    lib.csa2_sync_status(c.ws)
    codes, scales = orc.quantize_fp4(x.view(torch.int16).numpy().view(np.uint16))
    row = rows_of(0, 0, len(x), c.stride, c.page_table)
    assert torch.equal(c.d["codes"].cpu()[row], torch.from_numpy(codes))
    assert torch.equal(c.d["scales"].cpu()[row], torch.from_numpy(scales))


@pytest.mark.parametrize("counts,L", [
    ([400] + [3] * 199, 2),    # one long run among short ones: its windows by few CTAs
    ([1] * 300, 20),           # more tokens than CTAs per layer: a token's layers in a loop
    ([2] * 290 + [1], 5),      # short runs of more than 512 tokens
    ([1] * 600, 1),            # counters of more sequences than one CTA advances
])
def test_extend_spreads_runs_and_layers(lib, orc, counts, L):
    n0 = [(37 * b) % 190 for b in range(len(counts))]
    c = Case(lib, orc, counts, n0, L=L, pos="given")
    c.run()
    lib.csa2_sync_status(c.ws)
    c.check()


@pytest.mark.parametrize("many", [3, 700])
def test_extend_behind_4_gib(lib, orc, many):
    """Rows whose byte offset in the codes passes 32 bits: the same bits as in a
    small pool."""
    c = Case(lib, orc, [many, 1], [60, 5], L=0)
    pages = 17 * (1 << 20) // PAGE + 64  # of 256 code bytes a row: 4.25 GiB
    d = c.d
    far = d["page_table"] + (pages - c.pool // PAGE)
    big = {k: torch.empty((pages * PAGE, d[k].shape[1]), dtype=d[k].dtype, device="cuda")
           for k in ("codes", "scales", "idx_k")}
    for k in big:
        big[k][-c.pool:] = d[k]
    n_rows = d["n_rows"].clone()
    kv = lib.KVCache(big["codes"], big["scales"], big["idx_k"], n_rows, max_rows=2000, page_table=far)
    style = lib.ROPE_PAIRS
    ext = lib.CacheExtend(kv, d["x"], d["w"], cu_tokens=d["cu"], rope=lib.Rope(d["tab"], style),
                          rope_idx=lib.Rope(d["tab_idx"], style))
    lib.csa2_cache_extend(ext, c.ws)
    lib.csa2_sync_status(c.ws)
    c.run()
    lib.csa2_sync_status(c.ws)
    for k in big:
        assert torch.equal(big[k][-c.pool:], d[k]), k
    assert torch.equal(n_rows, d["n_rows"])
    c.check()


def test_extend_nothing(lib, orc):
    """No tokens at all: counters stay, nothing is written."""
    c = Case(lib, orc, [0, 0], [5, 6])
    c.run()
    lib.csa2_sync_status(c.ws)
    c.check()


def test_extend_far_position_of_a_long_cache(lib, orc):
    """The position is the last of a 1M-row sequence."""
    c = Case(lib, orc, [2], [(1 << 20) - 70], L=1, pos="given", dims=64, idx_dims=64, shuffle_extra=0)
    c.run()
    lib.csa2_sync_status(c.ws)
    c.check()


@pytest.mark.parametrize("many", [0, 700])
@pytest.mark.parametrize("what", ["unmapped", "page_out_of_pool", "capacity", "negative_rows", "negative_window",
                                  "offsets"])
def test_extend_refuses_a_run_as_a_whole(lib, orc, what, many):
    """The sequence stays as it was, the others are extended (few tokens, and
    many)."""
    counts = [10 + many, 200, 5]
    c = Case(lib, orc, counts, [60, 30, 3], paged=what != "capacity", L=1)
    d, bad = c.d, 1
    if what == "unmapped":
        c.page_table[1, 2] = d["page_table"][1, 2] = -1
    elif what == "page_out_of_pool":
        c.page_table[1, 1] = d["page_table"][1, 1] = c.pool // PAGE
    elif what == "capacity":
        n = c.stride - 199
        c.n_rows[1] = d["n_rows"][1] = n
    elif what == "negative_rows":
        c.n_rows[1] = d["n_rows"][1] = -1
    elif what == "negative_window":
        c.swa_pos[1] = d["swa_pos"][1] = -7
    else:  # the last run would end behind the tokens
        c.cu[3] = d["cu"][3] = sum(counts) + 1
        bad = 2
    # rotation positions stay those that the case was made with
    d["pos"] = torch.cat([c.at, torch.zeros(c.T - len(c.at), dtype=torch.int32)]).cuda()
    c.at_swa = c.at
    c.ext.keep += (d["pos"],)
    c.ext.desc.pos = d["pos"].data_ptr()
    c.run()
    with pytest.raises(lib.Csa2Error) as e:
        lib.csa2_sync_status(c.ws)
    assert e.value.status == 7
    c.check(refused=(bad,))


def test_extend_is_the_append_of_one_unrotated_entry(lib, orc):
    """Same FP4 rows, rings, counters and keys as csa2_cache_append."""
    a = Case(lib, orc, [1, 1, 1, 1], [0, 63, 64, 200], L=6, dims=0, idx_dims=0, cu=False)
    b = Case(lib, orc, [1, 1, 1, 1], [0, 63, 64, 200], L=6, dims=0, idx_dims=0, cu=False)
    a.run()
    d = b.d
    kv = lib.KVCache(d["codes"], d["scales"], d["idx_k"], d["n_rows"], max_rows=300, page_table=d["page_table"])
    lib.csa2_cache_append(kv, d["x"], d["w"], b.ws, d["x_swa"], d["swa"], d["swa_pos"], d["swa_len"])
    lib.csa2_sync_status(b.ws)
    for k in ("codes", "scales", "n_rows", "swa", "swa_pos", "swa_len"):
        assert torch.equal(a.d[k], b.d[k]), k
    lib.csa2_sync_status(a.ws)
    a.check()


def test_extend_is_rotation_then_quantiser(lib, orc):
    c = Case(lib, orc, [77], [10], L=0, idx_dims=0)
    c.run()
    y = torch.empty_like(c.d["x"])
    lib.csa2_rope_rows(lib.Rope(c.d["tab"]), c.d["x"].view(77, 1, D), c.at.int().cuda(), y.view(77, 1, D), c.ws)
    codes = torch.empty((77, 256), dtype=torch.uint8, device="cuda")
    scales = torch.empty((77, 32), dtype=torch.uint8, device="cuda")
    lib.csa2_quantize_fp4(y, codes, scales)
    row = rows_of(0, 10, 87, 0, c.page_table).cuda()
    assert torch.equal(c.d["codes"][row], codes) and torch.equal(c.d["scales"][row], scales)


def test_extend_captured_and_replayed(lib, orc):
    """Two replays append two runs; the counters on the device lead the way."""
    c = Case(lib, orc, [70, 3], [10, 60], L=2, pos="given", shuffle_extra=50)
    mp = 8  # room for both runs
    c.page_table = torch.randperm(c.pool // PAGE)[:2 * mp].int().view(2, mp)
    c.d["page_table"] = c.page_table.cuda()
    kv = c.ext.keep[0]
    kv.page_table = c.d["page_table"]
    c.ext.desc.kv.page_table, c.ext.desc.kv.max_pages = kv.page_table.data_ptr(), mp
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.run()
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        lib.csa2_sync_status(c.ws)
        c.check()


def test_extend_on_another_stream(lib, orc):
    c = Case(lib, orc, [150, 9], [1, 63], L=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    lib.csa2_sync_status(c.ws, stream=s)
    c.check()


def test_stored_rows_read_back(lib, orc):
    """What the cache holds after an extension is what csa2_dequantize_fp4 reads."""
    c = Case(lib, orc, [33], [0], L=0)
    c.run()
    y = torch.empty((c.pool, D), dtype=torch.bfloat16, device="cuda")
    lib.csa2_dequantize_fp4(c.d["codes"], c.d["scales"], y)
    assert torch.equal(y.cpu().double(), dequant(c.d["codes"].cpu(), c.d["scales"].cpu()))
