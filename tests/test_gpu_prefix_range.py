"""csa2_prefix_attn over the whole range of queries and scales: logits far below and
beyond fp32's range, rows where one key takes all, against the 64-bit definition with a
tolerance that stays small there."""
import pytest
import torch

from dense_ref import D, H, W, Attention, dequant, rows_of
from test_gpu_prefix import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp4_kv_cache_quantize_b200 import csa2
    return csa2


class Sharp(Attention):
    """Attention with a tolerance for logits that are off by more than a weight can be.
    Each logit may be off by d.  Then w_j' = w_j e^(t_j) / sum_k w_k e^(t_k), |t| <= d,
    so w_j' <= min(1, w_j e^(2 d)); and as the weights sum to 1, a weight falls by no
    more than the others rise together, nor by more than 1 - e^(-2 d) of itself.  What
    else rounds is as in Attention."""

    def __init__(self, c, sm_scale):
        B, nq = c.B, c.nq
        vals = dequant(c.codes, c.scales)
        q = c.q.double().view(B, nq, H, D)
        self.out, self.tol = torch.zeros((B, nq, H, D), dtype=torch.float64), None
        self.tol = torch.zeros_like(self.out)
        for b in range(B):
            n = int(c.n_rows[b])
            rows = rows_of(0, 0, min(n, c.prefix), c.stride, c.page_table)
            if n > c.prefix:
                rows = torch.cat([rows, rows_of(b, c.prefix, n, c.stride, c.page_table)])
            for t in range(nq):
                keys = vals[rows[:n - (nq - 1 - t)]]
                if c.swa is not None:
                    f = max(0, int(c.swa_len[b]) - (nq - 1 - t))
                    keys = torch.cat([keys, c.swa[b, max(0, f - W):f].view(torch.float8_e4m3fn).double()])
                x = q[b, t] @ keys.T * sm_scale
                logw = torch.log_softmax(x, -1)
                w = logw.exp()
                d = ((q[b, t].abs() @ keys.abs().T) * abs(sm_scale) * 520 * 2.0 ** -24
                     + x.abs() * 8 * 2.0 ** -24).amax(-1, keepdim=True)
                up = (logw + 2 * d).clamp(max=0.0).exp() - w
                down = torch.minimum(w * -torch.expm1(-2 * d), up.sum(-1, keepdim=True) - up)
                moved = torch.maximum(up, down)
                rel = 2.0 ** -10 + len(keys) * (2.0 ** -32 + 2.0 ** -24) + 2.0 ** -16
                self.out[b, t] = w @ keys
                self.tol[b, t] = (moved @ keys.abs() + rel * ((w + moved) @ keys.abs())
                                  + self.out[b, t].abs() * 2.0 ** -8
                                  + 2.0 ** -32 * (w + moved).amax(-1, keepdim=True) * keys.abs().sum(0))
        self.out, self.tol = self.out.view(B * nq, H, D), self.tol.view(B * nq, H, D)


def positive(c):
    """Keys without a sign: a query's logits all have its own."""
    c.codes &= 0x77
    c.swa &= 0x7F


def check(lib, c, sm_scale=D ** -0.5):
    c.build()
    c.attn = lib.PrefixAttn(c.kv, c.d["q"], c.prefix, swa=c.d["swa"], swa_len=c.d["swa_len"], n_query=c.nq,
                            sm_scale=sm_scale)
    ref = Sharp(c, sm_scale)
    # what is compared means something, but in a rare row whose two best keys are as good
    assert (ref.tol.norm(dim=-1) < 0.05 * ref.out.norm(dim=-1)).double().mean() > 0.9
    out = c.run()
    lib.csa2_sync_status(c.ws)
    ref.check(out)


SHAPES = [([900, 1000], 640, 1, [128, 9]), ([700, 650, 641], 600, 2, [129, 40, 2])]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("size", [1.0, 30.0, 1e4, 1e7, 1e10, 1e20, 1e31, 1e37])
def test_sharp_rows(lib, orc, shape, size):
    n_rows, prefix, nq, window = shape
    check(lib, Case(lib, orc, n_rows, prefix, nq, window=window, sharp=size, seed=31))


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("size", [1e4, 1e10, 1e31, 3e37])
def test_logits_of_one_sign(lib, orc, sign, size):
    """All logits far below zero are a softmax like any other; so are those above."""
    c = Case(lib, orc, [900, 1000], 640, 1, window=[128, 9], seed=32)
    positive(c)
    c.q = (sign * c.q.float().abs() * size).bfloat16()
    check(lib, c)


def test_rows_of_all_sizes_in_one_block(lib, orc):
    c = Case(lib, orc, [300, 400, 333], 256, 1, window=[128, 9, 77], seed=33)
    size = 10.0 ** torch.linspace(-38, 37, 3 * H).view(3, H, 1)
    c.q = (c.q.float().sign() * (0.5 + torch.rand(c.q.shape, generator=torch.Generator().manual_seed(1)))
           * size).bfloat16()
    c.q[1, 4] = 0.0
    check(lib, c)


@pytest.mark.parametrize("sm_scale", [0.0, -0.05, -30.0, 1e-38, 1e30, 3.4e38, -3.4e38])
@pytest.mark.parametrize("size", [1.0, 1e-30, 1e30])
def test_any_finite_scale(lib, orc, sm_scale, size):
    check(lib, Case(lib, orc, [900, 1000], 640, 1, window=[128, 9], sharp=size, seed=34), sm_scale)


def test_a_head_that_is_not_finite_is_nan(lib, orc):
    """Also where no logit of it would be: the others are as without it."""
    for bad in (float("inf"), float("-inf"), float("nan")):
        c = Case(lib, orc, [400, 300], 256, 1, window=[5, 128], seed=35)
        positive(c)
        want = Sharp(c, D ** -0.5)
        c.q[1, 3, 5] = bad
        c.build()
        out = c.run().float().cpu().double()
        lib.csa2_sync_status(c.ws)
        assert out[1, 3].isnan().all()
        out[1, 3] = want.out[1, 3]
        want.check(out)
