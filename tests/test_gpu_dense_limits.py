"""The extension, the rotation and the shared-prefix attention where calls are largest or
follow one another without a pause: offsets that pass 32 bits, the most sequences and
queries, whole decode loops in one graph."""
import pytest
import torch

from dense_ref import D, DI, H, PAGE, W, Attention, rotate, table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp4_kv_cache_quantize_b200 import csa2
    return csa2


def randn(gen, *shape, dtype=torch.bfloat16, chunk=1 << 27):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), chunk):
        flat[i:i + chunk] = torch.randn(min(chunk, flat.numel() - i), generator=gen, device="cuda").to(dtype)
    return out


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def packed(lib, x, rope, pos, ws):
    """Codes and scales of rotated rows, by the rotation and the quantiser."""
    y = torch.empty_like(x)
    lib.csa2_rope_rows(rope, x.view(-1, 1, D), pos, y.view(-1, 1, D), ws)
    codes = torch.empty((len(x), D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((len(x), D // 16), dtype=torch.uint8, device="cuda")
    lib.csa2_quantize_fp4(y, codes, scales)
    return codes, scales, y


def test_rotation_of_rows_behind_4_gib(lib):
    """In place and into another buffer; both pairings."""
    rows = 270000  # 4.4 GB
    g = gen_of(1)
    x = randn(g, rows, H, D)
    pos = torch.randint(0, 1000, (rows,), generator=g, device="cuda", dtype=torch.int32)
    tab, ws = table(1000, 64).cuda(), lib.workspace(lib.WS_HEADER)
    tail, tail_pos = x[-300:].clone(), pos[-300:].clone()
    for style in (lib.ROPE_PAIRS, lib.ROPE_HALVES):
        rope, want = lib.Rope(tab, style), torch.empty_like(tail)
        lib.csa2_rope_rows(rope, tail, tail_pos, want, ws)
        y = torch.empty_like(x)
        lib.csa2_rope_rows(rope, x, pos, y, ws)
        assert torch.equal(y[-300:], want)
        y.copy_(x)
        lib.csa2_rope_rows(rope, y, pos, y, ws)
        assert torch.equal(y[-300:], want)
        del y
    lib.csa2_sync_status(ws)


def test_extension_of_a_run_behind_4_gib(lib):
    """More than 2^22 tokens of one sequence: entries and keys to the end."""
    total, n0 = (1 << 22) + 5000, 3
    g = gen_of(2)
    x = randn(g, total, D)
    w = (randn(g, D, DI).float() * D ** -0.5).bfloat16()
    pool = -(-(total + n0) // PAGE) * PAGE
    codes = torch.zeros((pool, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((pool, D // 16), dtype=torch.uint8, device="cuda")
    idx_k = torch.zeros((pool, DI), dtype=torch.bfloat16, device="cuda")
    n_rows = torch.tensor([n0], dtype=torch.int32).cuda()
    pos = torch.arange(total, dtype=torch.int32, device="cuda") % 1000
    rope, ws = lib.Rope(table(1000, 64).cuda()), lib.workspace(lib.WS_HEADER)
    kv = lib.KVCache(codes, scales, idx_k, n_rows, max_rows=1 << 20, seq_stride=pool)
    cu = torch.tensor([0, total], dtype=torch.int32).cuda()
    lib.csa2_cache_extend(lib.CacheExtend(kv, x, w, cu_tokens=cu, pos=pos, rope=rope, rope_idx=rope), ws)
    lib.csa2_sync_status(ws)
    assert n_rows.item() == total + n0 and not codes[:n0].any() and not codes[total + n0:].any()
    for at in (0, total // 2 - 77, total - 700):
        want = packed(lib, x[at:at + 700], rope, pos[at:at + 700], ws)
        assert torch.equal(codes[n0 + at:n0 + at + 700], want[0])
        assert torch.equal(scales[n0 + at:n0 + at + 700], want[1])
        k = rotate(x[at:at + 700].cpu().double() @ w.cpu().double(), table(1000, 64)[pos[at:at + 700].cpu().long()], False)
        err = (x[at:at + 700].cpu().double().abs() @ w.cpu().double().abs()) * 2 * 520 * 2.0 ** -24
        assert ((idx_k[n0 + at:n0 + at + 700].cpu().double() - k).abs() <= err + k.abs() * 2.0 ** -8).all()


@pytest.mark.parametrize("counts", ["one", "few", "more"])
def test_extension_of_the_most_sequences(lib, counts):
    """65,535 sequences (rings of 4.3 GB): one token each, none to three, two to five."""
    B, g = 65535, gen_of(3)
    n = {"one": torch.ones(B, dtype=torch.long, device="cuda"),
         "few": torch.randint(0, 4, (B,), generator=g, device="cuda"),
         "more": torch.randint(2, 6, (B,), generator=g, device="cuda")}[counts]
    total, stride = int(n.sum()), 64
    x, x_swa, w = randn(g, total, D), randn(g, 1, total, D), randn(g, D, DI)
    codes = torch.zeros((B * stride, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((B * stride, D // 16), dtype=torch.uint8, device="cuda")
    idx_k = torch.zeros((B * stride, DI), dtype=torch.bfloat16, device="cuda")
    n0 = torch.randint(0, 50, (B,), generator=g, device="cuda", dtype=torch.int32)
    sp = n0 + 100
    n_rows, swa_pos, swa_len = n0.clone(), sp.clone(), sp.clamp(max=W)
    swa = torch.zeros((1, B, W, D), dtype=torch.uint8, device="cuda")
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), n.cumsum(0)]).int()
    rope, ws = lib.Rope(table(1000, 64).cuda()), lib.workspace(lib.WS_HEADER)
    kv = lib.KVCache(codes, scales, idx_k, n_rows, max_rows=64, seq_stride=stride)
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), n)
    off = torch.arange(total, device="cuda") - cu[:-1].long()[seq]
    pos = (n0[seq] + off).int()
    lib.csa2_cache_extend(lib.CacheExtend(
        kv, x, w, cu_tokens=None if counts == "one" else cu, pos=pos, rope=rope, rope_idx=rope, rope_swa=rope,
        x_swa=x_swa, swa=swa, swa_pos=swa_pos, swa_len=swa_len), ws)
    lib.csa2_sync_status(ws)
    assert torch.equal(n_rows, (n0 + n).int()) and torch.equal(swa_pos, (sp + n).int())
    assert torch.equal(swa_len, swa_pos.clamp(max=W))
    c, s, _ = packed(lib, x, rope, pos, ws)
    row = seq * stride + pos.long()
    assert torch.equal(codes[row], c) and torch.equal(scales[row], s)
    codes[row], scales[row], idx_k[row] = 0, 0, 0
    assert not codes.any() and not scales.any() and not idx_k.any()
    y = packed(lib, x_swa[0], rope, pos, ws)[2].float().to(torch.float8_e4m3fn).view(torch.uint8)
    slot = (sp.long()[seq] + off) % W
    assert torch.equal(swa[0, seq, slot], y)
    swa[0, seq, slot] = 0
    assert not swa.any()


def test_attention_of_the_most_queries(lib):
    """257 sequences x 255 queries, rows contiguous; a sample of them against 64 bits."""
    B, nq, prefix, g = 257, 255, 777, gen_of(4)
    stride = 1152
    codes = torch.randint(0, 256, (B * stride, 256), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.randn((B * stride, 32), generator=g, device="cuda").abs() * 0.3).to(torch.float8_e4m3fn).view(torch.uint8)
    n_rows = (prefix + nq + torch.arange(B) % 100).int()
    q = randn(g, B * nq, H, D)
    swa = torch.randn((B, W + nq - 1, D), generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    swa_len = (nq + torch.arange(B) % 128 - 1).int()
    kv = lib.KVCache(codes, scales, None, n_rows.cuda(), max_rows=int(n_rows.max()), seq_stride=stride)
    attn = lib.PrefixAttn(kv, q, prefix, swa=swa, swa_len=swa_len.cuda(), n_query=nq)
    ws = lib.workspace(attn.workspace_size())
    lib.csa2_prefix_attn(attn, ws)
    lib.csa2_sync_status(ws)
    out = attn.out.view(B, nq, H, D)
    assert torch.isfinite(attn.out).all()
    shared = [codes[:prefix].cpu(), scales[:prefix].cpu()]
    for b, t in [(0, 0), (0, 254), (1, 3), (100, 128), (128, 60), (255, 254), (256, 0), (256, 254)]:
        later = nq - 1 - t
        n, f = int(n_rows[b]) - later, int(swa_len[b]) - later
        own = slice(b * stride + prefix, b * stride + max(n, prefix))
        rows = [torch.cat([a[:n], v[own].cpu()]) for a, v in zip(shared, (codes, scales))]
        pad = -len(rows[0]) % PAGE
        rows = [torch.cat([v, torch.zeros((pad, v.shape[1]), dtype=torch.uint8)]) for v in rows]
        win = torch.zeros((1, W, D), dtype=torch.uint8)
        k = max(0, min(f, W))
        win[0, :k] = swa[b, max(0, f - W):max(0, f)].cpu()
        ref = Attention(rows[0], rows[1], None, len(rows[0]), [n], 0, q.view(B, nq, H, D)[b, t].cpu(), 1, win, [k])
        ref.check(out[b, t])


class Loop:
    """A decode loop: append rotated entries, rotate queries, attend, turn back."""

    def __init__(self, lib, seed, B=5, prefix=640, steps=12):
        g, self.lib, self.steps = gen_of(seed), lib, steps
        n0 = [prefix + 7 * b for b in range(B)]
        mp = -(-(max(n0) + steps) // PAGE)
        sp = prefix // PAGE
        perm = torch.randperm(sp + B * (mp - sp), generator=g, device="cuda").int()
        pages = torch.cat([perm[:sp].expand(B, sp), perm[sp:].view(B, mp - sp)], 1).contiguous()
        pool = len(perm) * PAGE
        self.state = dict(
            codes=torch.randint(0, 256, (pool, 256), generator=g, device="cuda", dtype=torch.uint8),
            scales=(torch.randn((pool, 32), generator=g, device="cuda").abs() * 0.3).to(torch.float8_e4m3fn).view(torch.uint8),
            idx_k=randn(g, pool, DI), n_rows=torch.tensor(n0, dtype=torch.int32).cuda(),
            swa=torch.randint(0, 120, (1, B, W, D), generator=g, device="cuda", dtype=torch.uint8),
            swa_pos=torch.tensor(n0, dtype=torch.int32).cuda(), swa_len=torch.full((B,), W, dtype=torch.int32).cuda())
        self.begin = {k: v.clone() for k, v in self.state.items()}
        s = self.state
        kv = lib.KVCache(s["codes"], s["scales"], s["idx_k"], s["n_rows"], max_rows=mp * PAGE, page_table=pages)
        self.rope, w = lib.Rope(table(2000, 64).cuda()), randn(g, D, DI)
        self.pos = [torch.tensor([n + i for n in n0], dtype=torch.int32).cuda() for i in range(steps)]
        self.q = [randn(g, B, H, D) for _ in range(steps)]
        x, xs = [randn(g, B, D) for _ in range(steps)], [randn(g, 1, B, D) for _ in range(steps)]
        self.ext = [lib.CacheExtend(kv, x[i], w, rope=self.rope, rope_idx=self.rope, rope_swa=self.rope, x_swa=xs[i],
                                    swa=s["swa"], swa_pos=s["swa_pos"], swa_len=s["swa_len"]) for i in range(steps)]
        self.rq = [torch.empty_like(v) for v in self.q]
        self.attn = [lib.PrefixAttn(kv, self.rq[i], prefix, swa=s["swa"][0], swa_len=s["swa_len"]) for i in range(steps)]
        self.out = [torch.empty_like(v) for v in self.q]
        self.ws = lib.workspace(max(a.workspace_size() for a in self.attn))

    def reset(self):
        for k, v in self.state.items():
            v.copy_(self.begin[k])
        for o in self.out:
            o.fill_(7.0)

    def run(self, wait=False, stream=None):
        for i in range(self.steps):
            for call in (lambda: self.lib.csa2_cache_extend(self.ext[i], self.ws, stream=stream),
                         lambda: self.lib.csa2_rope_rows(self.rope, self.q[i], self.pos[i], self.rq[i], self.ws, stream=stream),
                         lambda: self.lib.csa2_prefix_attn(self.attn[i], self.ws, stream=stream),
                         lambda: self.lib.csa2_rope_rows(self.rope, self.attn[i].out, self.pos[i], self.out[i], self.ws,
                                                         inverse=True, stream=stream)):
                call()
                if wait:
                    torch.cuda.synchronize()

    def result(self):
        torch.cuda.synchronize()
        self.lib.csa2_sync_status(self.ws)
        return [v.clone() for v in (*self.out, *self.state.values())]


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


def test_decode_loops_without_a_pause(lib):
    """Twelve steps call after call, in one graph, and two loops at once on two streams,
    give the bits of the same steps with a wait behind every call."""
    loops = [Loop(lib, 5), Loop(lib, 6, B=3, prefix=704)]
    want = []
    for lp in loops:
        lp.reset()
        lp.run(wait=True)
        want.append(lp.result())
        lp.reset()
        lp.run()
        assert same(lp.result(), want[-1])
    streams = [torch.cuda.Stream() for _ in loops]
    for lp in loops:
        lp.reset()
    torch.cuda.synchronize()
    for lp, st in zip(loops, streams):
        lp.run(stream=st)
    assert all(same(lp.result(), v) for lp, v in zip(loops, want))
    graphs = []
    for lp, st in zip(loops, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            lp.run()
        graphs.append(graph)
    for _ in range(3):
        for lp in loops:
            lp.reset()
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        assert all(same(lp.result(), v) for lp, v in zip(loops, want))


@pytest.mark.parametrize("tokens", [3, 40, 1500])
def test_extensions_without_a_pause(lib, tokens):
    """Runs of the same sequences call after call: each begins where the last one ended
    (few and many tokens, with windows)."""
    B, calls, g = 3, 20, gen_of(7)
    cut = torch.tensor([0, tokens // 3, tokens // 3, tokens], dtype=torch.int32).cuda()
    room = -(-calls * tokens // PAGE) * PAGE + PAGE
    x, xs = randn(g, calls, tokens, D), randn(g, calls, 1, tokens, D)
    w, rope = randn(g, D, DI), lib.Rope(table(calls * tokens + 10, 64).cuda())
    results = []
    for wait in (True, False):
        codes = torch.zeros((B * room, 256), dtype=torch.uint8, device="cuda")
        scales = torch.zeros((B * room, 32), dtype=torch.uint8, device="cuda")
        idx_k = torch.zeros((B * room, DI), dtype=torch.bfloat16, device="cuda")
        n_rows, pos, length = [torch.zeros(B, dtype=torch.int32).cuda() for _ in range(3)]
        swa = torch.zeros((1, B, W, D), dtype=torch.uint8, device="cuda")
        kv, ws = lib.KVCache(codes, scales, idx_k, n_rows, max_rows=room, seq_stride=room), lib.workspace(lib.WS_HEADER)
        ext = [lib.CacheExtend(kv, x[i], w, cu_tokens=cut, rope=rope, rope_idx=rope, rope_swa=rope, x_swa=xs[i],
                               swa=swa, swa_pos=pos, swa_len=length) for i in range(calls)]
        torch.cuda.synchronize()
        for e in ext:
            lib.csa2_cache_extend(e, ws)
            if wait:
                torch.cuda.synchronize()
        lib.csa2_sync_status(ws)
        results.append([codes, scales, idx_k, n_rows, pos, length, swa])
    assert same(*results)
    assert n_rows.tolist() == [calls * (tokens // 3), 0, calls * (tokens - tokens // 3)]
    at = torch.arange(calls * tokens, device="cuda").view(calls, tokens)
    mine = at % tokens >= tokens // 3
    rows = x[mine].view(-1, D)
    where = torch.arange(len(rows), device="cuda").int()
    want = packed(lib, rows, rope, where, ws)
    assert torch.equal(codes[2 * room:2 * room + len(rows)], want[0])
