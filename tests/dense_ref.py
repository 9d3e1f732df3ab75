"""Plain 64-bit references of the rotation, the cache extension and the
attention over a shared prefix, for their GPU tests (host tensors)."""
import numpy as np
import torch

D, H, DI, W, PAGE = 512, 16, 64, 128, 64


def table(n_pos, dims, base=10000.0):
    """(cos, sin) fp32 [n_pos][dims / 2][2]."""
    f = base ** (-torch.arange(0, dims, 2, dtype=torch.float64) / dims)
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * f
    return torch.stack((a.cos(), a.sin()), -1).float()


def rotate(x, cs, halves, inverse=False):
    """x [n][..., ch] rotated by cs [n][pairs][2], in 64 bits, unrounded."""
    x, n = x.double(), 2 * cs.shape[1]
    c, s = cs[..., 0].double(), cs[..., 1].double() * (-1 if inverse else 1)
    while c.dim() < x.dim():
        c, s = c.unsqueeze(1), s.unsqueeze(1)
    y = x.clone()
    t = x[..., x.shape[-1] - n:]
    a, b = (t[..., :n // 2], t[..., n // 2:]) if halves else (t[..., ::2], t[..., 1::2])
    u, v = a * c - b * s, a * s + b * c
    y[..., x.shape[-1] - n:] = torch.cat((u, v), -1) if halves else torch.stack((u, v), -1).flatten(-2)
    return y


def to_bf16(x):
    return x.float().bfloat16()


def dequant(codes, scales):
    """fp64 [n][512] values of E2M1 codes and E4M3 scales (host uint8)."""
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
    nib = torch.stack((codes & 15, codes >> 4), -1).view(codes.shape[0], -1).long()
    return lut[nib] * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)


def rows_of(b, lo, hi, stride, page_table):
    p = torch.arange(lo, hi)
    if page_table is None:
        return b * stride + p
    return page_table[b].long()[p // PAGE] * PAGE + p % PAGE


class Attention:
    """One call's reference: out [batch * nq][16][512] in 64 bits, and for each
    value how far a correct kernel may be from it."""

    def __init__(self, codes, scales, page_table, stride, n_rows, prefix, q, nq, swa=None, swa_len=None,
                 sm_scale=D ** -0.5):
        B = len(n_rows)
        vals = dequant(codes, scales)
        q = q.double().view(B, nq, H, D)
        self.out = torch.zeros((B, nq, H, D), dtype=torch.float64)
        self.tol = torch.zeros_like(self.out)
        for b in range(B):
            n = int(n_rows[b])
            rows = torch.cat([rows_of(0, 0, min(n, prefix), stride, page_table),
                              rows_of(b, prefix, n, stride, page_table) if n > prefix else
                              torch.zeros(0, dtype=torch.long)])
            for t in range(nq):
                keys = vals[rows[:max(0, n - (nq - 1 - t))]]
                if swa is not None:
                    f = max(0, int(swa_len[b]) - (nq - 1 - t))
                    keys = torch.cat([keys, swa[b, max(0, f - W):f].view(torch.float8_e4m3fn).double()])
                if not len(keys):
                    continue
                x = q[b, t] @ keys.T * sm_scale
                w = torch.softmax(x, -1)
                self.out[b, t] = w @ keys
                # a logit is off by the fp32 sum of 512 products and the fp32
                # roundings around it (8 units of its own size), and a weight
                # by e^(2 d) - 1 (numerator and normaliser) and its fp16
                # rounding (2^-11 in each); the sums over the keys and partials
                # round in fp32; the result rounds once to bf16 (half a step:
                # 2^-8).  Those are relative to the weight.  Below fp16's normal
                # range the rounding is absolute: weights are held as 2^7 w / r
                # with r at most the row's largest weight, in steps of 2^-24, so
                # each is off by at most 2^-25 r / 2^7 <= 2^-32 max w, whatever
                # its own size, and the sum over keys by 2^-32 max w sum |v|
                # (and the normaliser by 2^-32 max w a key)
                d = ((q[b, t].abs() @ keys.abs().T) * abs(sm_scale) * 520 * 2.0 ** -24
                     + x.abs() * 8 * 2.0 ** -24).amax(-1, keepdim=True)
                rel = 2 * d + 2.0 ** -10 + len(keys) * (2.0 ** -32 + 2.0 ** -24) + 2.0 ** -16
                self.tol[b, t] = (rel * (w @ keys.abs()) + self.out[b, t].abs() * 2.0 ** -8
                                  + 2.0 ** -32 * w.amax(-1, keepdim=True) * keys.abs().sum(0))
        self.out, self.tol = self.out.view(B * nq, H, D), self.tol.view(B * nq, H, D)

    def check(self, got):
        got = got.float().cpu().double().view(self.out.shape)
        assert torch.isfinite(got).all()
        off = (got - self.out).abs() - self.tol
        assert (off <= 1e-30).all(), (float(off.max()), (off > 1e-30).sum(), off.argmax())
