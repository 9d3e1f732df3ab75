"""Refusals of csa2_rope_rows, csa2_cache_extend and csa2_prefix_attn: found on
the host, before any CUDA call (this file needs no GPU)."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, ALIGN, WS = 0, 1, 2, 3, 4
P16, P4, P2 = 256, 260, 258


@pytest.fixture(scope="module")
def lib():
    from fp4_kv_cache_quantize_b200 import csa2
    return csa2


def rope(lib, **kw):
    r = dict(table=P16, n_pos=10, dims=64, style=0)
    r.update(kw)
    return lib.RopeStruct(r["table"], r["n_pos"], r["dims"], r["style"])


def rope_call(lib, r=None, x=P16, pos=P16, rows=4, heads=16, ch=512, y=1 << 30, ws=P16, ws_bytes=256):
    r = rope(lib) if r is None else r
    return lib._lib.csa2_rope_rows(ctypes.byref(r), ctypes.c_void_p(x), ctypes.c_void_p(pos),
                                   ctypes.c_int64(rows), heads, ch, 0, ctypes.c_void_p(y),
                                   ctypes.c_void_p(ws), ctypes.c_size_t(ws_bytes), None)


def test_rope_refusals(lib):
    assert lib._lib.csa2_rope_rows(None, None, None, ctypes.c_int64(0), 1, 64, 0, None, None,
                                   ctypes.c_size_t(0), None) == INVALID
    assert rope_call(lib, rope(lib, table=None)) == INVALID
    assert rope_call(lib, rope(lib, table=P4)) == ALIGN
    assert rope_call(lib, rope(lib, n_pos=0)) == SHAPE
    assert rope_call(lib, rope(lib, dims=0)) == SHAPE
    assert rope_call(lib, rope(lib, dims=48)) == SHAPE
    assert rope_call(lib, rope(lib, dims=544)) == SHAPE       # more than the row
    assert rope_call(lib, rope(lib, style=2)) == INVALID
    assert rope_call(lib, ch=516) == SHAPE
    assert rope_call(lib, ch=0) == SHAPE
    assert rope_call(lib, rows=-1) == SHAPE
    assert rope_call(lib, heads=-1) == SHAPE
    assert rope_call(lib, rows=1 << 40) == SHAPE
    assert rope_call(lib, x=None) == INVALID
    assert rope_call(lib, x=P4) == ALIGN
    assert rope_call(lib, pos=None) == INVALID
    assert rope_call(lib, pos=P2) == ALIGN
    assert rope_call(lib, ws=None) == INVALID
    assert rope_call(lib, ws_bytes=255) == WS
    # half overlapping rows: 4 x 16 x 512 x 2 bytes each
    assert rope_call(lib, x=1 << 20, y=(1 << 20) + 65520) == INVALID
    assert b"overlap" in lib._last_error()
    assert rope_call(lib, rows=0, x=None, y=None, pos=None, ws=None) == OK
    assert rope_call(lib, heads=0, x=None, y=None, pos=None, ws=None) == OK


def extend_desc(lib, **kw):
    kv = lib.KVView(P16, P16, P16, None, 64, 0, P16, 4, 128, 128, 512)
    d = lib.ExtendDesc(kv=kv, total=4, cu_tokens=P16, pos=P16, x=P16, w_idx=P16,
                       rope=rope(lib), rope_idx=rope(lib), rope_swa=rope(lib), n_layers=2, x_swa=P16,
                       swa=P16, swa_pos=P16, swa_len=P16)
    for k, v in kw.items():
        if k in ("codes", "scales", "idx_k", "page_table", "page_rows", "max_pages", "n_rows", "batch",
                 "max_rows", "seq_stride", "pool_rows"):
            setattr(d.kv, k, v)
        else:
            setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw,want", [
    (dict(batch=0), SHAPE), (dict(batch=65536), SHAPE), (dict(total=-1), SHAPE),
    (dict(total=1 << 24), SHAPE), (dict(n_layers=-1), SHAPE), (dict(n_layers=1025), SHAPE),
    (dict(x=None, n_layers=0), INVALID), (dict(cu_tokens=P2), ALIGN),
    (dict(cu_tokens=None, total=5), SHAPE), (dict(pos=P2), ALIGN), (dict(codes=None), INVALID),
    (dict(codes=P4), ALIGN), (dict(scales=None), INVALID), (dict(idx_k=None), INVALID),
    (dict(n_rows=None), INVALID), (dict(pool_rows=-1), SHAPE), (dict(seq_stride=100), ALIGN),
    (dict(seq_stride=-64), ALIGN), (dict(page_table=P16, page_rows=32), SHAPE),
    (dict(page_table=P16, max_pages=-1), SHAPE), (dict(x=P4), ALIGN), (dict(w_idx=None), INVALID),
    (dict(x_swa=None), INVALID), (dict(swa=P4), ALIGN), (dict(swa_pos=None), INVALID),
    (dict(swa_len=P2), ALIGN)])
def test_extend_refusals(lib, kw, want):
    d = extend_desc(lib, **kw)
    assert lib._lib.csa2_cache_extend(ctypes.byref(d), ctypes.c_void_p(P16), ctypes.c_size_t(256), None) == want


def test_extend_refuses_ropes_and_workspaces(lib):
    call = lambda d, ws=P16, n=256: lib._lib.csa2_cache_extend(  # noqa: E731
        ctypes.byref(d), ctypes.c_void_p(ws), ctypes.c_size_t(n), None)
    assert lib._lib.csa2_cache_extend(None, None, ctypes.c_size_t(0), None) == INVALID
    assert call(extend_desc(lib, rope=rope(lib, dims=33))) == SHAPE
    assert call(extend_desc(lib, rope_idx=rope(lib, dims=96))) == SHAPE   # a key has 64 channels
    assert call(extend_desc(lib, rope_swa=rope(lib, style=7))) == INVALID
    assert call(extend_desc(lib), ws=None) == INVALID
    assert call(extend_desc(lib), ws=P4) == ALIGN
    assert call(extend_desc(lib), n=128) == WS


def prefix_desc(lib, **kw):
    kv = lib.KVView(P16, P16, None, None, 64, 0, P16, 4, 1024, 1024, 4096)
    d = lib.PrefixDesc(kv=kv, prefix_rows=512, n_query=1, q=P16, swa=P16, swa_len=P16, sm_scale=0.04, out=P16)
    for k, v in kw.items():
        setattr(d.kv if hasattr(d.kv, k) else d, k, v)
    return d


@pytest.mark.parametrize("kw,want", [
    (dict(batch=0), SHAPE), (dict(batch=1025), SHAPE), (dict(n_query=-1), SHAPE), (dict(n_query=1025), SHAPE),
    (dict(batch=1024, n_query=64), SHAPE), (dict(max_rows=-1), SHAPE), (dict(max_rows=(1 << 20) + 1), SHAPE),
    (dict(prefix_rows=-1), SHAPE), (dict(prefix_rows=1025), SHAPE), (dict(codes=None), INVALID),
    (dict(scales=P4), ALIGN), (dict(n_rows=None), INVALID), (dict(seq_stride=960), SHAPE),
    (dict(page_table=P16, max_pages=15), SHAPE), (dict(page_table=P16, max_pages=16, page_rows=16), SHAPE),
    (dict(q=None), INVALID), (dict(q=P4), ALIGN), (dict(out=None), INVALID), (dict(swa=None), INVALID),
    (dict(swa_len=None), INVALID), (dict(swa=P4), ALIGN), (dict(sm_scale=float("nan")), INVALID),
    (dict(sm_scale=float("inf")), INVALID)])
def test_prefix_refusals(lib, kw, want):
    d = prefix_desc(lib, **kw)
    assert lib._lib.csa2_prefix_attn(ctypes.byref(d), ctypes.c_void_p(P16), ctypes.c_size_t(1 << 40), None) == want


def test_prefix_workspace(lib):
    f = lib._prefix_ws
    small, big = prefix_desc(lib), prefix_desc(lib, n_query=8)
    a, b = f(ctypes.byref(small)), f(ctypes.byref(big))
    assert 256 < a < b
    assert f(ctypes.byref(prefix_desc(lib, batch=0))) == 0
    call = lambda n: lib._lib.csa2_prefix_attn(  # noqa: E731
        ctypes.byref(small), ctypes.c_void_p(P16), ctypes.c_size_t(n), None)
    assert call(a - 1) == WS
    assert lib._lib.csa2_prefix_attn(None, None, ctypes.c_size_t(0), None) == INVALID


def test_binding_refuses_wrong_dtypes_and_shapes(lib):
    with pytest.raises(ValueError, match="dtype"):
        lib.Rope(torch.zeros(4, 32, 2, dtype=torch.float64))
    with pytest.raises(ValueError, match="n_pos"):
        lib.Rope(torch.zeros(4, 64))
    with pytest.raises(ValueError, match="CUDA"):
        lib.Rope(torch.zeros(4, 32, 2))

    class Kv:  # of the cache, the wrappers look at the batch first
        batch = 2
    x = torch.zeros(5, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="required"):
        lib.CacheExtend(Kv)
    with pytest.raises(ValueError, match="w_idx"):
        lib.CacheExtend(Kv, x)
    with pytest.raises(ValueError, match="x has shape"):
        lib.CacheExtend(Kv, x[:, :256], x)
    with pytest.raises(ValueError, match="w_idx has shape"):
        lib.CacheExtend(Kv, x, x)
    w = torch.zeros(512, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cu_tokens has dtype"):
        lib.CacheExtend(Kv, x, w, cu_tokens=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="pos has shape"):
        lib.CacheExtend(Kv, x, w, pos=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="swa"):
        lib.CacheExtend(Kv, x, w, x_swa=torch.zeros(1, 5, 512, dtype=torch.bfloat16))
    q = torch.zeros(2, 16, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q has"):
        lib.PrefixAttn(Kv, q, 0, n_query=2)
    with pytest.raises(ValueError, match="together"):
        lib.PrefixAttn(Kv, q, 0, swa=torch.zeros(2, 128, 512, dtype=torch.uint8))
    with pytest.raises(ValueError, match="q has dtype"):
        lib.PrefixAttn(Kv, q.float(), 0)


def test_rope_refuses_too_many_heads(lib):
    assert rope_call(lib, rows=1, heads=65537, ch=64, r=rope(lib, dims=32)) == SHAPE


class OnDevice:
    """Looks like a CUDA tensor to the binding; nothing is ever read through it."""

    def __init__(self, device, *shape, dtype=torch.bfloat16):
        self.device_index, self.shape, self.dtype, self.is_cuda = device, shape, dtype, True

    def get_device(self):
        return self.device_index

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return P16


def test_binding_refuses_other_devices(lib, monkeypatch):
    """Tensors, a workspace or a stream of another device than the current one:
    the launch would go to the current device with the other one's addresses."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    on = lambda d, *s, **kw: OnDevice(d, *s, **kw)  # noqa: E731
    table = {d: lib.Rope(on(d, 4, 32, 2, dtype=torch.float32)) for d in (0, 1)}
    ws = {d: on(d, 256, dtype=torch.uint8) for d in (0, 1)}

    def rope(t=0, x=0, pos=0, y=0, w=0, stream=None):
        lib.csa2_rope_rows(table[t], on(x, 3, 16, 512), on(pos, 3, dtype=torch.int32), on(y, 3, 16, 512), ws[w],
                           stream=stream)
    for kw in (dict(t=1), dict(x=1), dict(pos=1), dict(y=1)):
        with pytest.raises(ValueError, match="different devices"):
            rope(**kw)

    class Stream:
        device_index, cuda_stream = 1, 0
    for kw in (dict(t=1, x=1, pos=1, y=1, w=1), dict(w=1), dict(stream=Stream)):
        with pytest.raises(ValueError, match="the current one is 0"):
            rope(**kw)

    class Kv:
        batch, view, idx_k, page_table = 2, lib.KVView(), None, None
        codes, scales, n_rows = on(1, 64, 256), on(1, 64, 32), on(1, 2)
    with pytest.raises(ValueError, match="different devices"):
        lib.PrefixAttn(Kv, on(0, 2, 16, 512), 0, out=on(0, 2, 16, 512))
    attn = lib.PrefixAttn(Kv, on(1, 2, 16, 512), 0, out=on(1, 2, 16, 512))
    with pytest.raises(ValueError, match="the current one is 0"):
        lib.csa2_prefix_attn(attn, ws[0])
    with pytest.raises(ValueError, match="different devices"):
        lib.CacheExtend(Kv, on(0, 5, 512), on(0, 512, 64))
    ext = lib.CacheExtend(Kv, on(1, 5, 512), on(1, 512, 64))
    with pytest.raises(ValueError, match="the current one is 0"):
        lib.csa2_cache_extend(ext, ws[1])
