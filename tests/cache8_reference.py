"""The 8-bit cache and its decode step in 64 bits, from their definitions (plain torch, one sequence at a time)."""
import math

import torch

TOP = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def nearest_code(y, dtype):
    """The code nearest to y (fp64), ties to even, saturating; NaN stays (e4m3) or is 0 (int8).  In fp64 values."""
    top = TOP[dtype]
    y = y.clamp(-top, top)
    if dtype == torch.int8:
        return y.nan_to_num(0.0).round() + 0.0   # a whole number has no -0
    _, e = torch.frexp(y.abs().nan_to_num(1.0))
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp_min(-6) - 3)
    return (y / step).round() * step


class Model:
    """What a cache holds after appends: the rows themselves, quantised block by block when asked for."""

    def __init__(self, B, Hkv, d, dtype, block):
        self.dtype, self.block = dtype, block
        self.rows = {x: [torch.empty(Hkv, 0, d, dtype=torch.bfloat16) for _ in range(B)] for x in "kv"}

    def append(self, b, start, k, v):
        for x, new in (("k", k), ("v", v)):
            self.rows[x][b] = torch.cat([self.rows[x][b][:, :start], new.cpu()], 1)

    def length(self, b):
        return self.rows["k"][b].shape[1]

    def quantised(self, x, b):
        """codes (fp64 values) [Hkv, n, d] and scales fp32 [Hkv, blocks] of sequence b."""
        r = self.rows[x][b].double()
        codes, scales = [], []
        for j in range(0, r.shape[1], self.block):
            part = r[:, j:j + self.block]
            a = torch.where(part.isfinite(), part.abs(), 0.0).amax((1, 2)).clamp_min(2.0 ** -100)
            codes.append(nearest_code(part * TOP[self.dtype] / a[:, None, None], self.dtype))
            scales.append(a.float() / TOP[self.dtype])
        return torch.cat(codes, 1), torch.stack(scales, 1)

    def values(self, x, b):
        c, s = self.quantised(x, b)
        return c * s.double().repeat_interleave(self.block, 1)[:, :c.shape[1], None]


def decode(q, k, v, gate, tau, W, scale=0.0):
    """One sequence: q [Hq, n, d], k, v [Hkv, L, d] fp64 (its L positions), gate [n] fp32.  Returns the output
    [Hq, n, d] and a bound on the kernel's error, both fp64.

    The bound.  Each probability p carries relative errors from the score and from its rounding.  A score is a sum
    of d products held in fp32, added 16 at a time, each addition off by at most 2^-22 of the sum of magnitudes
    (twice a truncation to 24 bits), and scaled by two more fp32 roundings; so |ds| <= (d / 16 + 1) 2^-22 S with
    S = scale sum |q k|, and the subtraction of the maximum adds 2^-23 |s| <= 2^-23 S at either end.  q in fp16
    drops bits below 2^-25 of the row's largest element only: 2^-25 S too.  ex2.approx is off by 2^-22.  Numerator
    and denominator both carry it: 2 (e + 2^-21) with e = (d / 16 + 3) 2^-22 S.  P in fp16 adds 2^-11 in the
    numerator (and 2^-40 of the largest, at most, for subnormals).  The sums over L positions are fp32: (L / 16 + 64)
    2^-22, taken for numerator and denominator.  All of it scales sum p |v|.  The result is rounded to bf16: half a
    step, 2^-8 of the value (and the smallest bf16 step near zero)."""
    Hq, n, d = q.shape
    Hkv, L, _ = k.shape
    G = Hq // Hkv
    sc = scale if scale > 0 else 1 / math.sqrt(d)
    out = torch.zeros(Hq, n, d, dtype=torch.float64)
    bound = torch.zeros_like(out)
    for i in range(n):
        t = L - n + i
        if t < 0:
            continue
        share = 1 / (1 + math.exp(-float(gate[i]))) if float(gate[i]) > tau else 0.0
        for first, w in ((max(0, t - W + 1), 1.0), (0, share)):
            if w == 0.0:
                continue
            kk, vv = k[:, first:t + 1], v[:, first:t + 1]
            qi = q[:, i].double().view(Hkv, G, d)
            p = torch.softmax(torch.einsum("hgd,hld->hgl", qi, kk) * sc, -1)
            S = (torch.einsum("hgd,hld->hgl", qi.abs(), kk.abs()) * sc).amax(-1, keepdim=True)
            out[:, i] += w * torch.einsum("hgl,hld->hgd", p, vv).reshape(Hq, d)
            rel = 2 * ((d / 16 + 3) * 2.0 ** -22 * S + 2.0 ** -21 + (L / 16 + 64) * 2.0 ** -22) + 2.0 ** -11
            bound[:, i] += w * (rel * torch.einsum("hgl,hld->hgd", p, vv.abs()) +
                                2.0 ** -39 * vv.abs().sum(1)[:, None]).reshape(Hq, d)
    return out, bound + 2.0 ** -8 * (out.abs() + bound) + 1e-38
