"""The cache-filling and dense-attention operators, as measured cases.

Three operators work on one FP4 main-KV cache (E2M1 codes, one E4M3 scale per
16 channels, rows of 512 channels, a 64-channel bf16 indexer key per row):

  extend  append a ragged run of entries per sequence, rotated by position
  rope    rotate query or output rows by position, forward or back
  attn    dense attention of a batch whose sequences share a long prefix

`own` selects the framework's entry points; otherwise run() computes the same
with elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

D, H, DI, W, PAGE = 512, 16, 64, 128, 64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one new token of one long sequence, windows of a 20-layer decoder: pure latency
        dict(name="extend_1_token_20_layers", op="extend", batch=1, tokens=1, start=1000000, layers=20,
             dims=64, idx_dims=32, halves=False, paged=True, ratio=1),
        # a decode step of 64 ragged paged sequences, ratio-2 entries, 20 window layers
        dict(name="extend_64_seq_20_layers", op="extend", batch=64, tokens=64, start=131072, layers=20,
             dims=64, idx_dims=64, halves=False, paged=True, ratio=2),
        # prompt chunks of unequal length from 11 sequences, pages that end inside a run
        dict(name="extend_ragged_chunks", op="extend", batch=11, tokens=5003, start=30000, layers=2,
             dims=128, idx_dims=64, halves=True, paged=True, ratio=1),
        # one large prefill chunk into a contiguous cache
        dict(name="extend_prefill_32k", op="extend", batch=1, tokens=32768, start=77, layers=0,
             dims=64, idx_dims=64, halves=False, paged=False, ratio=1),
        # the queries of a 64-sequence decode step
        dict(name="rope_q_64", op="rope", rows=64, heads=16, ch=512, dims=64, halves=False, inverse=False,
             in_place=False),
        # the indexer queries of a chunk: short rows, rotated as a whole
        dict(name="rope_idx_q_chunk", op="rope", rows=4099, heads=8, ch=64, dims=64, halves=True, inverse=False,
             in_place=False),
        # the outputs of a prefill chunk turned back, in place
        dict(name="rope_out_back_8k", op="rope", rows=8192, heads=16, ch=512, dims=64, halves=False, inverse=True,
             in_place=True),
        # a small batch with a short system prompt: latency
        dict(name="attn_4x1_prefix_2k", op="attn", batch=4, queries=1, prefix=2048, own_rows=64, paged=True,
             window=True),
        # draft verification over an odd prefix, contiguous rows
        dict(name="attn_7x3_prefix_5003", op="attn", batch=7, queries=3, prefix=5003, own_rows=300, paged=False,
             window=True),
        # few sequences over a million-token document
        dict(name="attn_4x1_prefix_1m", op="attn", batch=4, queries=1, prefix=1000000, own_rows=500, paged=True,
             window=False),
        # a serving batch behind one long document, ragged continuations
        dict(name="attn_64x1_prefix_128k", op="attn", batch=64, queries=1, prefix=131072, own_rows=2000, paged=True,
             window=True),
        # a prompt chunk of two sequences over their shared prefix
        dict(name="attn_2x256_prefix_16k", op="attn", batch=2, queries=256, prefix=16384, own_rows=700, paged=True,
             window=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "extend", "rope", "attn", "attn"])
    if op == "extend":
        batch = _log(rng, 1, 64)
        tokens = batch if rng.random() < 0.4 else max(batch, _log(rng, batch, 16000))
        return dict(op=op, batch=batch, tokens=tokens, start=_log(rng, 1, 400000),
                    layers=rng.choice([0, 1, 2, 5, 20]) if tokens <= 2000 else rng.choice([0, 1, 2]),
                    dims=rng.choice([32, 64, 128, 512]), idx_dims=rng.choice([0, 32, 64]),
                    halves=rng.random() < 0.5, paged=rng.random() < 0.7, ratio=rng.choice([1, 2]))
    if op == "rope":
        heads, ch = rng.choice([(16, 512), (8, 64), (1, 512), (5, 192)])
        return dict(op=op, rows=_log(rng, 1, 8000), heads=heads, ch=ch, dims=rng.choice([32, 64]),
                    halves=rng.random() < 0.5, inverse=rng.random() < 0.5, in_place=rng.random() < 0.5)
    batch = _log(rng, 1, 64)
    queries = rng.choice([1, 1, 1, 2, 3, 4, 8, _log(rng, 5, 100)])
    queries = min(queries, max(1, 1000 // batch))
    most = min(900000, 120000000 // (batch * queries * 16) + 500)
    return dict(op=op, batch=batch, queries=queries, prefix=_log(rng, 200, max(300, most)),
                own_rows=queries + _log(rng, 1, 1000), paged=rng.random() < 0.7, window=rng.random() < 0.7)


# ----------------------------------------------------------------- inputs
def _spread(parts, total, least):
    """`parts` unequal whole numbers >= least that sum to `total`, by the case alone."""
    r = np.random.RandomState((parts * 7919 + total) % (1 << 31))
    cut = np.sort(r.randint(0, total - parts * least + 1, parts - 1)) if parts > 1 else np.zeros(0, int)
    return [int(v) + least for v in np.diff(np.concatenate([[0], cut, [total - parts * least]]))]


def _pack(x):
    """bf16 rows [n][512] -> (codes, scales): E2M1 with one E4M3 scale per 16 channels."""
    g = x.float().view(x.shape[0], -1, 16)
    scale = (g.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    q = torch.where(s > 0, g / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(g))
    a = q.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * torch.signbit(q).to(torch.uint8)
    code = code.view(x.shape[0], -1, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4), scale.view(torch.uint8)


def _unpack(codes, scales):
    """The values that codes and scales stand for, fp32 [n][512]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).view(codes.shape[0], -1, 16)
    return (v * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)).view(codes.shape[0], -1)


def _table(n_pos, dims):
    """(cos, sin) of every position, angles in 64 bits, rounded once: fp32 [n_pos][dims / 2][2]."""
    if dims == 0:
        return None
    f = 10000.0 ** (-torch.arange(0, dims, 2, device="cuda", dtype=torch.float64) / dims)
    a = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.stack((a.cos(), a.sin()), -1).float().contiguous()


def _ints(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_extend(case, gen, rnd):
    B, T, L = case["batch"], case["tokens"], case["layers"]
    counts = _spread(B, T, 1)
    if case["paged"]:
        n0 = [case["start"] - (i * 997) % max(1, case["start"] // 2) for i in range(B)]
        need = [(n + c - 1) // PAGE - n // PAGE + 1 for n, c in zip(n0, counts)]
        pages = sum(need) + 5
        mp = max((n + c - 1) // PAGE + 1 for n, c in zip(n0, counts)) + 2
        order = torch.randperm(pages - 1, generator=gen, device="cuda").add_(1).int().cpu()
        table, at = torch.zeros((B, mp), dtype=torch.int32), 0  # pages before the run are not touched: page 0
        for b in range(B):
            table[b, n0[b] // PAGE:n0[b] // PAGE + need[b]] = order[at:at + need[b]]
            at += need[b]
        page_table, stride, pool = table.cuda(), 0, pages * PAGE
    else:
        n0 = [min(case["start"], 200) - i % max(1, min(case["start"], 200)) for i in range(B)]
        stride = -(-max(n + c for n, c in zip(n0, counts)) // PAGE) * PAGE
        page_table, pool = None, stride * B
    swa_pos = [n + 13 for n in n0]
    pad = -(-B // 4) * 4
    begin = torch.zeros((3, pad), dtype=torch.int32)
    begin[0, :B], begin[1, :B] = torch.tensor(n0), torch.tensor(swa_pos)
    begin[2, :B] = torch.tensor(swa_pos).clamp(max=W)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    offs = torch.arange(T) - torch.repeat_interleave(cu[:-1].cpu().long(), torch.tensor(counts))
    start = torch.repeat_interleave(torch.tensor(n0), torch.tensor(counts))
    s = dict(
        case=case, cu=cu, begin=begin.cuda(), counters=begin.cuda(), page_table=page_table, stride=stride,
        pos=((start + offs) * case["ratio"]).int().cuda(),
        x=rnd(T, D).bfloat16(), w_idx=(rnd(D, DI) * D ** -0.5).bfloat16(),
        codes=torch.randint(0, 256, (pool, D // 2), generator=gen, device="cuda", dtype=torch.uint8),
        scales=rnd(pool, D // 16).abs().to(torch.float8_e4m3fn).view(torch.uint8),
        idx_k=rnd(pool, DI).bfloat16(), values=torch.empty((pool, D), dtype=torch.bfloat16, device="cuda"),
        x_swa=rnd(L, T, D).bfloat16() if L else None,
        swa=rnd(L, B, W, D).to(torch.float8_e4m3fn).view(torch.uint8) if L else None)
    most = (max(n + c for n, c in zip(n0, counts))) * case["ratio"] + 1
    s["table"], s["table_idx"] = _table(most, case["dims"]), _table(most, case["idx_dims"])
    c = s["counters"]
    s["n_rows"], s["swa_pos"], s["swa_len"] = c[0, :B], c[1, :B], c[2, :B]
    if own:
        from fp4_kv_cache_quantize_b200 import csa2
        style = csa2.ROPE_HALVES if case["halves"] else csa2.ROPE_PAIRS
        kv = csa2.KVCache(s["codes"], s["scales"], s["idx_k"], s["n_rows"],
                          max_rows=max(n + c for n, c in zip(n0, counts)), seq_stride=stride, page_table=page_table)
        rope = csa2.Rope(s["table"], style)
        rope_idx = csa2.Rope(s["table_idx"], style) if case["idx_dims"] else None
        more = dict(x_swa=s["x_swa"], swa=s["swa"], swa_pos=s["swa_pos"], swa_len=s["swa_len"], rope_swa=rope) if L else {}
        s["extend"] = csa2.CacheExtend(kv, s["x"], s["w_idx"], cu_tokens=cu, pos=s["pos"], rope=rope,
                                       rope_idx=rope_idx, **more)
        s["ws"] = csa2.workspace(csa2.WS_HEADER)
    return s


def _prepare_rope(case, gen, rnd):
    R, heads, ch = case["rows"], case["heads"], case["ch"]
    n_pos = 200000
    x = rnd(R, heads, ch).bfloat16()
    s = dict(case=case, x=x, table=_table(n_pos, case["dims"]),
             pos=torch.randint(0, n_pos, (R,), generator=gen, device="cuda", dtype=torch.int32),
             y=x.clone() if case["in_place"] else torch.empty_like(x))
    if own:
        from fp4_kv_cache_quantize_b200 import csa2
        s["rope"] = csa2.Rope(s["table"], csa2.ROPE_HALVES if case["halves"] else csa2.ROPE_PAIRS)
        s["ws"] = csa2.workspace(csa2.WS_HEADER)
    return s


def _prepare_attn(case, gen, rnd):
    B, Q, P = case["batch"], case["queries"], case["prefix"]
    lens = [max(Q, case["own_rows"] - (i * 131) % max(1, case["own_rows"])) for i in range(B)]
    shared = P // PAGE * PAGE if case["paged"] else P  # whole pages are shared
    n_rows = [P + n for n in lens]
    if case["paged"]:
        sp = shared // PAGE
        need = [(n + PAGE - 1) // PAGE - sp for n in n_rows]
        pages = sp + sum(need)
        order = torch.randperm(pages, generator=gen, device="cuda").int()
        table = torch.zeros((B, sp + max(need)), dtype=torch.int32, device="cuda")
        table[:, :sp] = order[:sp]
        at = sp
        for b in range(B):
            table[b, sp:sp + need[b]] = order[at:at + need[b]]
            at += need[b]
        page_table, stride, pool = table, 0, pages * PAGE
    else:
        page_table, stride = None, -(-max(n_rows) // PAGE) * PAGE
        pool = stride * B
    codes = torch.empty((pool, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pool, D // 16), dtype=torch.uint8, device="cuda")
    for r in range(0, pool, 65536):
        n = min(65536, pool - r)
        codes[r:r + n], scales[r:r + n] = _pack(rnd(n, D).bfloat16())
    # heads from flat to sharp: the logits' deviation runs from 0.5 to 3
    sharp = torch.rand((B * Q, H, 1), generator=gen, device="cuda") * 2.5 + 0.5
    rows_w = W + Q - 1
    win = [min(rows_w, Q + (i * 37) % W) for i in range(B)]
    s = dict(case=case, codes=codes, scales=scales, page_table=page_table, stride=stride, shared=shared,
             n_rows=_ints(*n_rows), max_rows=max(n_rows), q=(rnd(B * Q, H, D) * sharp).bfloat16(),
             swa=rnd(B, rows_w, D).to(torch.float8_e4m3fn).view(torch.uint8) if case["window"] else None,
             swa_len=_ints(*win) if case["window"] else None)
    if own:
        from fp4_kv_cache_quantize_b200 import csa2
        kv = csa2.KVCache(codes, scales, None, s["n_rows"], max_rows=s["max_rows"], seq_stride=stride,
                          page_table=page_table)
        s["attn"] = csa2.PrefixAttn(kv, s["q"], shared, swa=s["swa"], swa_len=s["swa_len"], n_query=Q)
        s["ws"] = csa2.workspace(s["attn"].workspace_size())
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def rnd(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    return dict(extend=_prepare_extend, rope=_prepare_rope, attn=_prepare_attn)[case["op"]](case, gen, rnd)


# ------------------------------------------------------------ plain forms
def _rotate(x, cs, halves, inverse=False):
    """Rotates the last channels of x [..., ch] by cs [..., pairs, 2], in 64 bits."""
    n = cs.shape[-2] * 2
    t, c, s = x[..., x.shape[-1] - n:].double(), cs[..., 0].double(), cs[..., 1].double()
    if inverse:
        s = -s
    a, b = (t[..., :n // 2], t[..., n // 2:]) if halves else (t[..., 0::2], t[..., 1::2])
    u, v = a * c - b * s, a * s + b * c
    t = torch.cat((u, v), -1) if halves else torch.stack((u, v), -1).flatten(-2)
    return torch.cat((x[..., :x.shape[-1] - n].double(), t), -1)


def _run_extend(s):
    case, B = s["case"], s["case"]["batch"]
    s["counters"].copy_(s["begin"])  # the run is taken back first, as rejected drafts are
    if own:
        from fp4_kv_cache_quantize_b200 import csa2
        csa2.csa2_cache_extend(s["extend"], s["ws"])
        csa2.csa2_dequantize_fp4(s["codes"], s["scales"], s["values"])
    else:
        token = torch.arange(case["tokens"], device="cuda")
        seq = torch.searchsorted(s["cu"][1:].long(), token, right=True)
        off = token - s["cu"].long()[seq]
        p = s["n_rows"].long()[seq] + off
        row = seq * s["stride"] + p if s["page_table"] is None else s["page_table"].long()[seq, p // PAGE] * PAGE + p % PAGE
        cs = s["table"][s["pos"].long()]
        s["codes"][row], s["scales"][row] = _pack(_rotate(s["x"], cs, case["halves"]).float().bfloat16())
        k = s["x"].float() @ s["w_idx"].float()
        if case["idx_dims"]:
            k = _rotate(k, s["table_idx"][s["pos"].long()], case["halves"]).float()
        s["idx_k"][row] = k.bfloat16()
        counts = (s["cu"][1:] - s["cu"][:-1])
        if case["layers"]:
            kept = (off >= counts.long()[seq] - W).nonzero()[:, 0]
            slot = (s["swa_pos"].long()[seq] + off) % W
            v = _rotate(s["x_swa"][:, kept], cs[kept], case["halves"]).float().bfloat16()
            s["swa"][:, seq[kept], slot[kept]] = v.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s["swa_pos"] += counts
            s["swa_len"].copy_(s["swa_pos"].clamp(max=W))
        s["n_rows"] += counts
        s["values"].copy_(_unpack(s["codes"], s["scales"]))
    out = dict(values=s["values"], idx_k=s["idx_k"], n_rows=s["n_rows"])
    if case["layers"]:
        out.update(swa=s["swa"].view(torch.float8_e4m3fn), swa_pos=s["swa_pos"], swa_len=s["swa_len"])
    return out


def _run_rope(s):
    case = s["case"]
    src = s["x"]
    if case["in_place"]:
        s["y"].copy_(s["x"])  # the rows as the attention left them
        src = s["y"]
    if own:
        from fp4_kv_cache_quantize_b200 import csa2
        csa2.csa2_rope_rows(s["rope"], src, s["pos"], s["y"], s["ws"], inverse=case["inverse"])
    else:
        cs = s["table"][s["pos"].long()].unsqueeze(1)
        s["y"].copy_(_rotate(src, cs, case["halves"], case["inverse"]).float())
    return s["y"]


def _run_attn(s):
    case = s["case"]
    if own:
        from fp4_kv_cache_quantize_b200 import csa2
        csa2.csa2_prefix_attn(s["attn"], s["ws"])
        return s["attn"].out
    B, Q, P = case["batch"], case["queries"], s["shared"]
    n = s["n_rows"].long()
    pos = torch.arange(P, device="cuda")
    row = pos if s["page_table"] is None else s["page_table"].long()[0, pos // PAGE] * PAGE + pos % PAGE
    shared = _unpack(s["codes"][row], s["scales"][row])
    most = s["max_rows"] - P
    pos = (P + torch.arange(most, device="cuda")).expand(B, most)
    seq = torch.arange(B, device="cuda")[:, None]
    inside = pos < n[:, None]
    if s["page_table"] is None:
        row = seq * s["stride"] + pos
    else:
        row = s["page_table"].long()[seq, (pos // PAGE).clamp(max=s["page_table"].shape[1] - 1)] * PAGE + pos % PAGE
    row = torch.where(inside, row, torch.zeros_like(row))
    mine = _unpack(s["codes"][row.flatten()], s["scales"][row.flatten()]).view(B, most, D)
    later = (Q - 1 - torch.arange(Q, device="cuda"))[None, :]
    see = pos[:, None, :] < (n[:, None] - later)[:, :, None]
    q = s["q"].float().view(B, Q * H, D) * D ** -0.5
    parts = [(q.reshape(-1, D) @ shared.t()).view(B, Q, H, P),
             torch.where(see[:, :, None], (q @ mine.transpose(1, 2)).view(B, Q, H, most), -torch.inf)]
    if case["window"]:
        win = s["swa"].view(torch.float8_e4m3fn).float()
        end = (s["swa_len"].long()[:, None] - later)[:, :, None]
        j = torch.arange(win.shape[1], device="cuda")[None, None, :]
        see = (j < end) & (j >= end - W)
        parts.append(torch.where(see[:, :, None], (q @ win.transpose(1, 2)).view(B, Q, H, -1), -torch.inf))
    top = torch.stack([t.amax(-1) for t in parts]).amax(0).unsqueeze(-1)
    parts = [(t - top).exp_() for t in parts]
    total = torch.stack([t.sum(-1) for t in parts]).sum(0).view(B, Q * H, 1)
    out = (parts[0].view(-1, P) @ shared).view(B, Q * H, D) + parts[1].view(B, Q * H, most) @ mine
    if case["window"]:
        out = out + parts[2].view(B, Q * H, -1) @ win
    return (out / total).view(B * Q, H, D).bfloat16()


def run(state):
    return dict(extend=_run_extend, rope=_run_rope, attn=_run_attn)[state["case"]["op"]](state)


# ------------------------------------------------------------------- work
def _shape_extend(case):
    counts = _spread(case["batch"], case["tokens"], 1)
    if case["paged"]:
        n0 = [case["start"] - (i * 997) % max(1, case["start"] // 2) for i in range(case["batch"])]
        pool = (sum((n + c - 1) // PAGE - n // PAGE + 1 for n, c in zip(n0, counts)) + 5) * PAGE
    else:
        n0 = [min(case["start"], 200) - i % max(1, min(case["start"], 200)) for i in range(case["batch"])]
        pool = -(-max(n + c for n, c in zip(n0, counts)) // PAGE) * PAGE * case["batch"]
    return counts, pool


def work(case):
    if case["op"] == "extend":
        counts, pool = _shape_extend(case)
        T, L = case["tokens"], case["layers"]
        kept = sum(min(c, W) for c in counts)
        a_token = D * 2 + 4 + case["dims"] * 4 + case["idx_dims"] * 4 + 288 + DI * 2
        read_back = pool * (288 + D * 2)  # the whole cache, as the values that it stands for
        return {"bytes": T * a_token + D * DI * 2 + L * kept * (D * 2 + D) + read_back, "flops": T * 2 * D * DI}
    if case["op"] == "rope":
        n = case["rows"] * case["heads"]
        copy = n * case["ch"] * 4 if case["in_place"] else 0
        turned = n * (case["dims"] if case["in_place"] else case["ch"]) * 4
        return {"bytes": copy + turned + case["rows"] * (4 + case["dims"] * 4), "flops": n * case["dims"] * 3}
    B, Q = case["batch"], case["queries"]
    shared = case["prefix"] // PAGE * PAGE if case["paged"] else case["prefix"]
    rest = sum(case["prefix"] + max(Q, case["own_rows"] - (i * 131) % max(1, case["own_rows"])) - shared for i in range(B))
    win = sum(min(W + Q - 1, Q + (i * 37) % W) for i in range(B)) if case["window"] else 0
    keys = B * shared + rest + (min(W, win / B) * B if win else 0)
    return {"bytes": (shared + rest) * 288 + win * D + B * Q * H * D * 4, "flops": keys * Q * H * D * 4}


# ------------------------------------------- the definitions in 64 bits
def _levels(v, levels):
    """The nearest of ascending `levels` to v >= 0, ties to the even index, the last for all above."""
    lv = torch.tensor(levels, dtype=torch.float64, device=v.device)
    hi = torch.searchsorted(lv, v.contiguous()).clamp(1, len(levels) - 1)
    lo = hi - 1
    a, b = v - lv[lo], lv[hi] - v
    return lv[torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)]


def _e4m3_levels():
    return [k * 2.0 ** -9 for k in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)
                                                if not (e == 15 and m == 7)]


def _turn(x, angle_cs, halves, sign):
    """The same rotation as products of complex numbers; x [..., ch] in 64 bits."""
    z = torch.complex(angle_cs[..., 0].double(), sign * angle_cs[..., 1].double())
    n = 2 * z.shape[-1]
    keep, t = x.double().split((x.shape[-1] - n, n), -1)
    w = t.unflatten(-1, (2, n // 2)).transpose(-1, -2) if halves else t.unflatten(-1, (n // 2, 2))
    w = torch.view_as_real(torch.view_as_complex(w.contiguous()) * z)
    return torch.cat((keep, (w.transpose(-1, -2) if halves else w).flatten(-2)), -1)


def _exact_extend(case, s):
    pool = s["codes"].shape[0]
    nib = torch.stack((s["codes"] % 16, s["codes"] // 16), -1).view(pool, D).long()
    mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[nib % 8]
    value = torch.where(nib < 8, mag, -mag) * s["scales"].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
    idx_k = s["idx_k"].double()
    swa = s["swa"].view(torch.float8_e4m3fn).double() if case["layers"] else None
    cu, n0 = s["cu"].tolist(), s["n_rows"].tolist()
    for b in range(case["batch"]):
        t = slice(cu[b], cu[b + 1])
        p = torch.arange(n0[b], n0[b] + cu[b + 1] - cu[b], device="cuda")
        row = b * s["stride"] + p if s["page_table"] is None else s["page_table"][b].long()[p // PAGE] * PAGE + p % PAGE
        at = s["pos"][t].long()
        x = _turn(s["x"][t], s["table"][at], case["halves"], 1.0).float().bfloat16()
        g = x.double().view(len(p), -1, 16)
        step = _levels((g.abs().amax(-1).float() / 6.0).double(), _e4m3_levels())[..., None]
        level = _levels((g / step.clamp(min=1e-30)).abs(), E2M1)
        value[row] = (torch.copysign(level, g) * step).view(len(p), D)
        k = s["x"][t].double() @ s["w_idx"].double()
        idx_k[row] = _turn(k, s["table_idx"][at], case["halves"], 1.0) if case["idx_dims"] else k
        if case["layers"]:
            last = slice(max(0, len(p) - W), len(p))
            v = _turn(s["x_swa"][:, t][:, last], s["table"][at[last]], case["halves"], 1.0).float().bfloat16().double()
            slot = (s["swa_pos"][b].long() + torch.arange(last.start, last.stop, device="cuda")) % W
            swa[:, b, slot] = torch.copysign(_levels(v.abs(), _e4m3_levels()), v)
    out = dict(values=value, idx_k=idx_k, n_rows=None)
    if case["layers"]:
        out.update(swa=swa, swa_pos=None, swa_len=None)
    return out


def _exact_attn(case, s):
    B, Q = case["batch"], case["queries"]

    def rows_of(b, lo, hi):
        p = torch.arange(lo, hi, device="cuda")
        r = b * s["stride"] + p if s["page_table"] is None else s["page_table"][b].long()[p // PAGE] * PAGE + p % PAGE
        c = s["codes"][r]
        nib = torch.stack((c % 16, c // 16), -1).view(len(p), D).long()
        mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[nib % 8]
        return torch.where(nib < 8, mag, -mag) * s["scales"][r].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)

    P, out = s["shared"], torch.empty((B * Q, H, D), dtype=torch.float64, device="cuda")
    shared = rows_of(0, 0, P)
    for b in range(B):
        n = int(s["n_rows"][b])
        mine = rows_of(b, P, n)
        t = torch.arange(Q, device="cuda").repeat_interleave(H)[:, None]
        see = [torch.arange(P, n, device="cuda")[None] <= n - Q + t]
        keys = [mine]
        if case["window"]:
            w = int(s["swa_len"][b])
            j = torch.arange(w, device="cuda")[None]
            keys.append(s["swa"][b, :w].view(torch.float8_e4m3fn).double())
            see.append((j <= w - Q + t) & (j > w - Q + t - W))
        for r in range(0, Q * H, 1024):
            q = s["q"].view(B, Q * H, D)[b, r:r + 1024].double()
            logit = [q @ shared.T] + [(q @ k.T).masked_fill(~m[r:r + 1024], -math.inf) for k, m in zip(keys, see)]
            a = torch.softmax(torch.cat(logit, -1) / math.sqrt(D), -1)
            o = a[:, :P] @ shared
            at = P
            for k in keys:
                o += a[:, at:at + len(k)] @ k
                at += len(k)
            out.view(B, Q * H, D)[b, r:r + 1024] = o
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "extend":
        return _exact_extend(case, s)
    if case["op"] == "rope":
        return _turn(s["x"], s["table"][s["pos"].long()].unsqueeze(1), case["halves"], -1.0 if case["inverse"] else 1.0)
    return _exact_attn(case, s)
