"""Draft verification with windows: entries that may be rejected are appended without
them, their window rows go to scratch rings, and only the accepted ones to the rings."""
import pytest
import torch

from dense_ref import D, W, rotate, table, to_bf16
from test_gpu_prefix import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp4_kv_cache_quantize_b200 import csa2
    return csa2


def i32(*v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def test_drafts_behind_full_rings(lib, orc):
    """Three steps of four drafts: rings that are full and wrapped, filling and empty;
    all drafts accepted, some, or one. Every query sees its 128 newest window rows."""
    nq, B, prefix, dims, steps = 4, 4, 640, 64, 3
    n, taken = [650, 700, 641, 660], [[4, 1, 2, 4], [1, 4, 3, 1], [2, 2, 4, 4]]
    c = Case(lib, orc, [v + nq * steps for v in n], prefix, nq, seed=51)
    g = torch.Generator().manual_seed(52)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    tab = table(3000, dims)
    rope, ws = lib.Rope(tab.cuda()), lib.workspace(lib.WS_HEADER)
    w = r(D, 64).bfloat16().cuda()
    n_rows = i32(*n)
    kv = lib.KVCache(c.d["codes"], c.d["scales"], torch.zeros((c.pool, 64), dtype=torch.bfloat16).cuda(), n_rows,
                     max_rows=c.max_rows, page_table=c.d["page_table"])
    start = [1000, 127, 50, 0]  # window rows written so far
    old = [r(v, D).to(torch.float8_e4m3fn).view(torch.uint8) for v in start]
    ring = torch.zeros((1, B, W, D), dtype=torch.uint8)
    for b in range(B):
        for j in range(max(0, start[b] - W), start[b]):
            ring[0, b, j % W] = old[b][j]
    ring, ring_pos, ring_len = ring.cuda(), i32(*start), i32(*[min(v, W) for v in start])
    cu = torch.arange(0, B * nq + 1, nq, dtype=torch.int32).cuda()
    for step in range(steps):
        x, x_swa = r(B * nq, D).bfloat16(), r(1, B * nq, D).bfloat16()
        at = n_rows.tolist()
        pos = torch.tensor([v + t for v in at for t in range(nq)], dtype=torch.int32)
        # the drafts' entries, and their window rows into scratch rings
        lib.csa2_cache_extend(lib.CacheExtend(kv, x.cuda(), w, cu_tokens=cu, pos=pos.cuda(), rope=rope), ws)
        scratch, zero, zero2 = torch.zeros_like(ring), i32(*[0] * B), i32(*[0] * B)
        lib.csa2_cache_extend(lib.CacheExtend(kv, cu_tokens=cu, pos=pos.cuda(), rope_swa=rope, x_swa=x_swa.cuda(),
                                              swa=scratch, swa_pos=zero, swa_len=zero2), ws)
        win, length = torch.zeros((B, W + nq - 1, D), dtype=torch.uint8).cuda(), []
        rp, rl = ring_pos.tolist(), ring_len.tolist()
        for b in range(B):
            keep = min(rl[b], W - 1)
            win[b, :keep] = ring[0, b, [(rp[b] - keep + i) % W for i in range(keep)]]
            win[b, keep:keep + nq] = scratch[0, b, :nq]
            length.append(keep + nq)
        q = r(B * nq, 16, D).bfloat16().cuda()
        attn = lib.PrefixAttn(kv, q, prefix, swa=win, swa_len=i32(*length), n_query=nq)
        aws = lib.workspace(attn.workspace_size())
        lib.csa2_prefix_attn(attn, aws)
        lib.csa2_sync_status(aws)
        lib.csa2_sync_status(ws)
        # what the queries saw, from the rows' own history
        new = to_bf16(rotate(x_swa[0], tab[pos.long()], False)).float().to(torch.float8_e4m3fn).view(torch.uint8)
        for b in range(B):
            for t in range(nq):
                f = length[b] - (nq - 1 - t)
                want = torch.cat([old[b], new[b * nq:b * nq + t + 1]])[-W:]
                assert torch.equal(win[b, max(0, f - W):f].cpu(), want)
        c.codes, c.scales, c.n_rows = c.d["codes"].cpu(), c.d["scales"].cpu(), n_rows.cpu()
        c.q, c.swa, c.swa_len = q.cpu(), win.cpu(), torch.tensor(length, dtype=torch.int32)
        assert c.n_rows.tolist() == [v + nq for v in at]
        c.reference().check(attn.out)
        # the accepted drafts stay: the entries' count goes back, their window rows are added
        kept = [b * nq + t for b in range(B) for t in range(taken[step][b])]
        n_rows.copy_(i32(*[v + k for v, k in zip(at, taken[step])]))
        cu_kept = i32(0, *torch.tensor(taken[step]).cumsum(0).tolist())
        lib.csa2_cache_extend(lib.CacheExtend(kv, cu_tokens=cu_kept, pos=pos[kept].cuda(), rope_swa=rope,
                                              x_swa=x_swa[:, kept].cuda(), swa=ring, swa_pos=ring_pos,
                                              swa_len=ring_len), ws)
        lib.csa2_sync_status(ws)
        for b in range(B):
            old[b] = torch.cat([old[b], new[b * nq:b * nq + taken[step][b]]])
            k = len(old[b])
            assert ring_pos[b] == k and ring_len[b] == min(k, W)
            for j in range(max(0, k - W), k):
                assert torch.equal(ring[0, b, j % W].cpu(), old[b][j])
