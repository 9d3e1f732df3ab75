"""GPU parity of csa2_prefix_attn with its 64-bit definition (dense_ref.py says
how far each value may be off, and why), its masks and its place between the
extension, the rotation and the sparse attention."""
import pytest
import torch

from dense_ref import D, H, PAGE, W, Attention, rotate, table, to_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp4_kv_cache_quantize_b200 import csa2
    return csa2


class Case:
    def __init__(self, lib, orc, n_rows, prefix, nq=1, *, paged=True, window=None, seed=0, sharp=1.0, q=None,
                 max_rows=None):
        g = torch.Generator().manual_seed(seed)
        B = len(n_rows)
        self.lib, self.B, self.nq, self.prefix = lib, B, nq, prefix
        most = max(max(n_rows), prefix, 1)
        r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        if paged:
            mp = -(-most // PAGE)
            sp = prefix // PAGE  # pages that every sequence shares
            own = mp - sp
            perm = torch.randperm(sp + B * own + 2, generator=g).int()
            self.page_table = torch.cat([perm[:sp].expand(B, sp), perm[sp:sp + B * own].view(B, own)], 1).contiguous()
            self.stride, self.pool = 0, len(perm) * PAGE
        else:
            self.page_table, self.stride = None, -(-most // PAGE) * PAGE
            self.pool = B * self.stride
        self.codes = torch.randint(0, 256, (self.pool, 256), generator=g, dtype=torch.uint8)
        self.scales = (r(self.pool, 32).abs() * 0.3).to(torch.float8_e4m3fn).view(torch.uint8)
        self.n_rows = torch.tensor(n_rows, dtype=torch.int32)
        self.q = (r(B * nq, H, D) * sharp).bfloat16() if q is None else q
        self.swa = self.swa_len = None
        if window is not None:
            self.swa = r(B, W + nq - 1, D).to(torch.float8_e4m3fn).view(torch.uint8)
            self.swa_len = torch.tensor(window, dtype=torch.int32)
        self.max_rows = most if max_rows is None else max_rows
        self.build()

    def build(self):
        lib = self.lib
        self.d = {k: None if getattr(self, k) is None else getattr(self, k).cuda()
                  for k in ("codes", "scales", "page_table", "n_rows", "q", "swa", "swa_len")}
        d = self.d
        self.kv = lib.KVCache(d["codes"], d["scales"], None, d["n_rows"], max_rows=self.max_rows,
                              seq_stride=self.stride, page_table=d["page_table"])
        self.attn = lib.PrefixAttn(self.kv, d["q"], self.prefix, swa=d["swa"], swa_len=d["swa_len"], n_query=self.nq)
        self.attn.out.fill_(99.0)
        self.ws = lib.workspace(self.attn.workspace_size())

    def run(self, **kw):
        self.lib.csa2_prefix_attn(self.attn, self.ws, **kw)
        return self.attn.out

    def reference(self):
        return Attention(self.codes, self.scales, self.page_table, self.stride, self.n_rows, self.prefix, self.q,
                         self.nq, self.swa, self.swa_len)

    def check(self):
        out = self.run()
        self.lib.csa2_sync_status(self.ws)
        self.reference().check(out)


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("n_rows,prefix,nq,window", [
    ([1], 0, 1, None),
    ([1], 1, 1, [0]),
    ([64, 65], 64, 1, None),
    ([127, 128, 129], 0, 1, [1, 128, 127]),
    ([130, 200, 129, 128, 140], 128, 1, [128, 0, 5, 127, 64]),
    ([700, 513, 640], 513, 1, [128, 128, 128]),
    ([1000, 900], 896, 3, [130, 3]),
    ([600, 601, 700, 602, 603, 604, 605], 600, 2, [129] * 7),
    ([300, 450], 256, 5, [132, 60]),
    ([2500], 2048, 1, [128]),
    ([200, 260], 128, 70, [197, 100]),
    ([1300] * 17, 1280, 1, None),
])
def test_prefix_attn(lib, orc, n_rows, prefix, nq, window, paged):
    if not paged and prefix % PAGE:
        pass  # a contiguous prefix may end anywhere
    Case(lib, orc, n_rows, prefix, nq, paged=paged, window=window, seed=len(n_rows) + nq).check()


def test_rows_that_see_nothing(lib, orc):
    """No keys gives zeros: empty sequences, queries in front of the first entry,
    sequences shorter than the prefix, an empty window."""
    c = Case(lib, orc, [0, 1, 2, 70, 0], 64, 3, window=[0, 0, 1, 0, 2])
    c.check()
    out = c.attn.out.view(5, 3, H, D)
    assert not out[0].any() and not out[1, :2].any() and not out[4, 0].any()
    assert out[1, 2].any() and out[4, 2].any()
    Case(lib, orc, [0], 0, 1).check()
    Case(lib, orc, [0, 0], 0, 1, window=[0, 128]).check()


def test_a_batch_without_own_rows(lib, orc):
    Case(lib, orc, [512] * 6, 512, 1).check()


@pytest.mark.parametrize("sharp", [0.0, 1e-6, 30.0, 1e4])
def test_query_magnitudes(lib, orc, sharp):
    """Flat rows, and rows where one key takes all and appears late (the
    reference is raised many times on the way)."""
    Case(lib, orc, [900, 1000], 640, 1, window=[128, 9], sharp=sharp, seed=2).check()


def test_logits_that_keep_rising(lib, orc):
    """Each key tile's logits exceed the last tile's by more than the slack."""
    c = Case(lib, orc, [1500, 1400], 1280, 1, sharp=1.0, seed=4)
    pos = torch.arange(1500)
    q0 = c.q[0, 0].double()
    step = (q0.sign() * 2).clamp(-6, 6)  # rows along the sign of one query, growing with the position
    nib = torch.where(step > 0, 4, 12).to(torch.uint8)
    code = nib.view(-1, 2)[:, 0] | (nib.view(-1, 2)[:, 1] << 4)
    for b in range(2):
        rows = c.page_table[b].long()[pos // PAGE] * PAGE + pos % PAGE
        c.codes[rows] = code
        c.scales[rows] = (0.01 + pos[:, None] / 1500.0).float().expand(-1, 32).to(torch.float8_e4m3fn).view(torch.uint8)
    c.build()
    c.check()


def test_nan_in_masked_places(lib, orc):
    """Rows behind the last entry, window rows outside of it and entries of later
    drafts may hold NaN: only the queries that see one turn NaN."""
    c = Case(lib, orc, [300, 260], 256, 3, window=[100, 130], seed=6)
    pos = torch.arange(300, 320)
    rows = c.page_table[0].long()[pos // PAGE] * PAGE + pos % PAGE
    c.scales[rows] = 0x7F
    c.swa[0, 100:] = 0x7F
    clean = c.reference()
    c.build()
    out = c.run()
    lib.csa2_sync_status(c.ws)
    clean.check(out)
    # the newest entry (position 259 of sequence 1) is seen by its last query only
    row = c.page_table[1].long()[259 // PAGE] * PAGE + 259 % PAGE
    c.scales[row, 3] = 0xFF
    c.swa[0, 99, 77] = 0xFF  # and the newest window row of sequence 0
    c.build()
    out = c.run().view(2, 3, H, D).float().cpu().double()
    lib.csa2_sync_status(c.ws)
    want, tol = clean.out.view(2, 3, H, D), clean.tol.view(2, 3, H, D)
    for b in (0, 1):
        assert out[b, 2].isnan().all()
        assert ((out[b, :2] - want[b, :2]).abs() <= tol[b, :2] + 1e-30).all()


def test_infinite_query_head_stays_alone(lib, orc):
    c = Case(lib, orc, [400, 300], 256, 1, seed=8)
    want = c.reference()
    c.q[1, 3, 5] = float("inf")
    c.build()
    out = c.run().float().cpu().double()
    lib.csa2_sync_status(c.ws)
    assert out[1, 3].isnan().all()
    out[1, 3] = want.out[1, 3]
    assert ((out - want.out).abs() <= want.tol + 1e-30).all()


def test_unmapped_pages_are_skipped_and_reported(lib, orc):
    c = Case(lib, orc, [500, 400], 256, 1, seed=9)
    keep = c.page_table.clone()
    c.page_table[1, 5] = -1            # positions 320..383 of sequence 1
    c.page_table[0, 7] = c.pool        # positions 448..499 of sequence 0
    c.build()
    out = c.run()
    with pytest.raises(lib.Csa2Error) as e:
        lib.csa2_sync_status(c.ws)
    assert e.value.status == 7
    # the same without those rows: sequence 0 ends in front of its hole, and
    # sequence 1's page 6 moves into the place of page 5
    c.page_table = keep
    c.n_rows = torch.tensor([448, 336], dtype=torch.int32)
    c.page_table[1, 5] = keep[1, 6]
    c.reference().check(out)


def test_counts_out_of_range_are_clamped(lib, orc):
    c = Case(lib, orc, [200, 300], 64, 1, window=[10, 20])
    want = c.reference()
    c.d["n_rows"][1] = 301  # beyond max_rows = 300
    out = c.run()
    with pytest.raises(lib.Csa2Error):
        lib.csa2_sync_status(c.ws)
    want.check(out)
    c.d["n_rows"][1] = 300
    c.d["swa_len"][0] = -4
    out = c.run()
    with pytest.raises(lib.Csa2Error):
        lib.csa2_sync_status(c.ws)
    c.swa_len[0] = 0
    c.reference().check(out)


def test_pool_behind_4_gib(lib, orc):
    """Rows whose byte offset in the codes passes 32 bits: the same bits as from a
    small pool."""
    c = Case(lib, orc, [700, 650], 600, 2, window=[129, 40], seed=9)
    near = c.run().clone()
    lib.csa2_sync_status(c.ws)
    pages = 17 * (1 << 20) // PAGE + 64  # of 256 code bytes a row: 4.25 GiB
    d = c.d
    codes = torch.empty((pages * PAGE, 256), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages * PAGE, 32), dtype=torch.uint8, device="cuda")
    codes[-c.pool:], scales[-c.pool:] = d["codes"], d["scales"]
    kv = lib.KVCache(codes, scales, None, d["n_rows"], max_rows=c.max_rows,
                     page_table=d["page_table"] + (pages - c.pool // PAGE))
    far = lib.PrefixAttn(kv, d["q"], c.prefix, swa=d["swa"], swa_len=d["swa_len"], n_query=c.nq)
    lib.csa2_prefix_attn(far, c.ws)
    lib.csa2_sync_status(c.ws)
    assert torch.equal(far.out, near)
    c.check()


def test_the_largest_batch(lib, orc):
    """As many sequences as a call may have, each of its own length, empty ones among
    them; one more is refused (on the host)."""
    Case(lib, orc, [(7 * b) % 40 for b in range(1024)], 5, paged=False, seed=4).check()


# Many row blocks over a prefix of some length: its fp16 tiles are made first.
MANY = dict(nq=256, seed=21)


@pytest.mark.parametrize("n_rows,prefix,window,paged", [
    ([1400, 1290], 1100, [383, 200], True),
    ([1300, 1000], 1088, None, False),
])
def test_many_row_blocks(lib, orc, n_rows, prefix, window, paged):
    Case(lib, orc, n_rows, prefix, paged=paged, window=window, **MANY).check()


def test_many_row_blocks_nan_in_masked_places(lib, orc):
    """A NaN in a prefix row behind a sequence's end reaches only the others' queries
    that see the row; so does one in a window."""
    c = Case(lib, orc, [1000, 1300], 1100, **MANY)
    clean = c.reference()
    row = c.page_table[0].long()[1050 // PAGE] * PAGE + 1050 % PAGE
    c.scales[row, 17] = 0x7F
    c.build()
    out = c.run().view(2, 256, H, D).float().cpu().double()
    lib.csa2_sync_status(c.ws)
    want, tol = clean.out.view(2, 256, H, D), clean.tol.view(2, 256, H, D)
    sees = 1300 - 255 + torch.arange(256) > 1050
    assert out[1, sees].isnan().all()
    out[1, sees] = want[1, sees]
    assert ((out - want).abs() <= tol + 1e-30).all()


def test_many_row_blocks_unmapped_page(lib, orc):
    """Skipped and reported: as if the page's positions were not there at all."""
    c = Case(lib, orc, [1400, 1290], 1100, **MANY)
    c.page_table[0, 5] = -1
    c.build()
    out = c.run()
    with pytest.raises(lib.Csa2Error) as e:
        lib.csa2_sync_status(c.ws)
    assert e.value.status == 7
    c.page_table = torch.cat([c.page_table[:, :5], c.page_table[:, 6:]], 1)
    c.n_rows, c.prefix = c.n_rows - PAGE, c.prefix - PAGE
    c.reference().check(out)


def test_many_row_blocks_captured(lib, orc):
    """A replayed graph reads the rows that are there then, on any stream; two graphs
    with a workspace each do not meet."""
    cases = [Case(lib, orc, [1400, 1290], 1100, **MANY), Case(lib, orc, [1200, 1300], 1090, nq=300, seed=22)]
    graphs = []
    for c in cases:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run()
        graphs.append(g)
    for c in cases:
        c.codes = (c.codes.int() * 7 + 3).to(torch.uint8)
        c.d["codes"].copy_(c.codes)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for c in cases:
        lib.csa2_sync_status(c.ws)
        c.reference().check(c.attn.out)


def test_shared_rows_are_sequence_zeros(lib, orc):
    """Positions below prefix_rows come from sequence 0's pages for everyone."""
    a = Case(lib, orc, [300, 290], 128, 1, seed=11)
    first = a.run().clone()
    a.page_table[1, :2] = -1  # never looked at
    a.build()
    assert torch.equal(a.run(), first)
    lib.csa2_sync_status(a.ws)


def test_same_result_every_time_and_on_another_stream(lib, orc):
    c = Case(lib, orc, [3000, 2900, 3100], 2500, 2, window=[129, 60, 2], seed=12)
    first = c.run().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        c.attn.out.fill_(0)
        s.wait_stream(torch.cuda.current_stream())
        c.run(stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(c.attn.out, first)


def test_captured_with_growing_sequences(lib, orc):
    """One graph serves every length up to max_rows: the counts are on the device."""
    c = Case(lib, orc, [400, 390], 256, 1, window=[128, 128], seed=13)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.run()
    for n in ([256, 256], [300, 257], [400, 399], [3, 0]):
        c.n_rows = torch.tensor(n, dtype=torch.int32)
        c.d["n_rows"].copy_(c.n_rows)
        g.replay()
        torch.cuda.synchronize()
        c.reference().check(c.attn.out)
        lib.csa2_sync_status(c.ws)


def test_two_workspaces_two_streams(lib, orc):
    a = Case(lib, orc, [2000, 1900], 1500, 1, seed=14)
    b = Case(lib, orc, [1800, 1700, 1600], 1536, 1, seed=15)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        a.run(stream=s1)
        b.run(stream=s2)
    torch.cuda.synchronize()
    a.reference().check(a.attn.out)
    b.reference().check(b.attn.out)


def test_short_contexts_equal_the_sparse_attention(lib, orc):
    """With at most 512 entries the sparse attention selects them all: both
    compute the same sum, each to its own rounding."""
    c = Case(lib, orc, [512, 300], 256, 1, window=[128, 77], seed=16)
    out = c.run()
    ref = c.reference()
    ref.check(out)
    idx = torch.arange(512, dtype=torch.int32).repeat(2, 1)
    idx[1, 300:] = -1
    other = torch.empty_like(out)
    ws = lib.workspace(lib.csa2_attn_workspace_size(2))
    # sparse rows are looked up per sequence: both map the prefix to the same pages
    k = torch.zeros((c.pool, 64), dtype=torch.bfloat16, device="cuda")
    kv = lib.KVCache(c.d["codes"], c.d["scales"], k, c.d["n_rows"], max_rows=512, page_table=c.d["page_table"])
    lib.csa2_sparse_attn_decode(c.d["q"], kv, idx.cuda(), c.d["n_rows"], 512, c.d["swa"], c.d["swa_len"], D ** -0.5,
                                other, ws)
    lib.csa2_sync_status(ws)
    rel = (out.double() - other.double()).norm() / out.double().norm()
    assert rel < 2 * 2.0 ** -8 + 2.0 ** -10  # two bf16 roundings, two fp16 weights


def test_extend_rotate_attend_turn_back(lib, orc):
    """The run that a server makes of a step: drafts appended with rotation, the
    queries rotated, attention over shared prefix, own rows and window, and the
    outputs turned back by the query's position, against 64 bits throughout."""
    nq, B, prefix, dims = 2, 3, 640, 64
    n0 = [650, 700, 641]
    c = Case(lib, orc, [n + nq for n in n0], prefix, nq, seed=17)
    g = torch.Generator().manual_seed(18)
    tab = table(2000, dims)
    x = torch.randn((B * nq, D), generator=g).bfloat16()
    w = torch.randn((D, 64), generator=g).bfloat16()
    x_swa = torch.randn((1, B * nq, D), generator=g).bfloat16()
    swa = torch.zeros((1, B, W, D), dtype=torch.uint8)
    pos = torch.tensor([n + t for n in n0 for t in range(nq)], dtype=torch.int32)
    d = c.d
    n_rows = torch.tensor(n0, dtype=torch.int32).cuda()
    kv = lib.KVCache(d["codes"], d["scales"], torch.zeros((c.pool, 64), dtype=torch.bfloat16).cuda(), n_rows,
                     max_rows=c.max_rows, page_table=d["page_table"])
    rope = lib.Rope(tab.cuda())
    swa_pos, swa_len = torch.zeros(B, dtype=torch.int32).cuda(), torch.zeros(B, dtype=torch.int32).cuda()
    swa_d = swa.cuda()
    ext = lib.CacheExtend(kv, x.cuda(), w.cuda(), cu_tokens=torch.arange(0, B * nq + 1, nq, dtype=torch.int32).cuda(),
                          pos=pos.cuda(), rope=rope, rope_idx=rope, rope_swa=rope, x_swa=x_swa.cuda(), swa=swa_d,
                          swa_pos=swa_pos, swa_len=swa_len)
    win = torch.zeros((B, W + nq - 1, D), dtype=torch.uint8).cuda()
    q = torch.empty_like(d["q"])
    attn = lib.PrefixAttn(kv, q, prefix, swa=win, swa_len=swa_len, n_query=nq)
    ws = lib.workspace(max(attn.workspace_size(), lib.WS_HEADER))
    lib.csa2_cache_extend(ext, ws)
    win[:, :nq] = swa_d[0, :, :nq]
    lib.csa2_rope_rows(rope, d["q"], pos.cuda(), q, ws)
    lib.csa2_prefix_attn(attn, ws)
    turned = torch.empty_like(attn.out)
    lib.csa2_rope_rows(rope, attn.out, pos.cuda(), turned, ws, inverse=True)
    lib.csa2_sync_status(ws)
    # 64 bits, on the cache as stored
    c.codes, c.scales, c.n_rows = d["codes"].cpu(), d["scales"].cpu(), n_rows.cpu()
    assert c.n_rows.tolist() == [n + nq for n in n0]
    c.q = to_bf16(rotate(c.q, tab[pos.long()], False))
    assert torch.equal(q.cpu(), c.q)
    c.swa, c.swa_len = win.cpu(), swa_len.cpu()
    want = to_bf16(rotate(x_swa[0], tab[pos.long()], False)).float().to(torch.float8_e4m3fn)
    assert torch.equal(win[:, :nq].cpu().view(B * nq, D), want.view(torch.uint8))
    ref = c.reference()
    ref.check(attn.out)
    assert torch.equal(turned.cpu(), to_bf16(rotate(attn.out.cpu(), tab[pos.long()], False, True)))
