"""The E4M3 cache's definition in 64 bits, for the tests of the calls that
write and read it (torch, no code of the package)."""
import math

import torch

PAGE = 16
HALF_BF16 = 2.0 ** -8   # half a step of bf16, relative
HALF_E4M3 = 2.0 ** -4   # of E4M3's normal values
HALF_SUB = 2.0 ** -10   # of its subnormal ones, absolute


def values(codes):
    """fp64 value of every code: 4 exponent bits (bias 7), 3 mantissa bits, no infinities."""
    c = codes.view(torch.uint8).long()
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e.double() - 10))
    v = torch.where(c >= 128, -v, v)
    return torch.where((c & 127) == 127, torch.full_like(v, math.nan), v)


def powers(scale):
    """fp64 value of every exponent byte."""
    s = scale.view(torch.uint8).double()
    return torch.where(s == 255, torch.full_like(s, math.nan), torch.exp2(s - 127))


def exponent(amax):
    """Least integer e >= -100 with amax <= 448 * 2^e (fp64 amax, finite)."""
    e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -200))) - 9
    for _ in range(3):
        e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    return e.clamp(min=-100)


def quantize(y):
    """fp64 vectors -> (codes, scale bytes) by the rule; codes rounded by torch from exact quotients."""
    finite = torch.isfinite(y).all(-1)
    e = torch.where(finite, exponent(torch.where(torch.isfinite(y), y, 0.0).abs().amax(-1)), 0.0)
    q = torch.where(finite[..., None], y * torch.exp2(-e)[..., None], math.nan)
    codes = q.float().to(torch.float8_e4m3fn).view(torch.uint8)  # an fp32 quotient is exact up to 24 bits
    codes = torch.where(finite[..., None], codes, 0x7f)
    return codes.to(torch.uint8), torch.where(finite, e + 127, 255.0).to(torch.uint8)


def attention(q, k, ks, v, vs, table, start, kv_len):
    """-> (out, bound) in 64 bits: rows start[s] .. start[s + 1] of sequence s
    see its first kv_len[s] keys, causally at the end.  The bound of a kernel
    that sums exact products in fp32 (every add off by a whole step 2^-23), keeps
    the softmax in fp32 and rounds its weights to bf16 for their product:
      score  : d * 2^-23 * sum |q k| / sqrt(d) + 4 roundings 2^-24 |score|, and
               2^-21 for the exponentials; it acts on weights as a factor, above
               and below the fraction: twice
      weights: half a step of bf16, above the fraction
      sums   : n adds of a step 2^-23, above and below
    all of them relative to sum p |v|; then half a step of bf16 of the output."""
    T, n_q, d = q.shape
    n_kv = k.shape[1]
    grp = n_q // n_kv
    out, bound = torch.zeros(T, n_q, d, dtype=torch.float64), torch.zeros(T, n_q, d, dtype=torch.float64)
    q = q.double()
    for s, n in enumerate(kv_len):
        r0, r1 = start[s], start[s + 1]
        pages = torch.tensor(table[s][:-(-n // PAGE)])
        pos = torch.arange(n - (r1 - r0), n)
        hidden = torch.arange(n)[None] > pos[:, None]
        for g in range(n_kv):
            kk, vv = ((values(c[pages, g]) * powers(e[pages, g])[..., None]).reshape(-1, d)[:n]
                      for c, e in ((k, ks), (v, vs)))
            for h in range(g * grp, (g + 1) * grp):
                x = q[r0:r1, h] @ kk.T / math.sqrt(d)
                size = (q[r0:r1, h].abs() @ kk.abs().T / math.sqrt(d)).masked_fill(hidden, 0.0)
                delta = (d * 2.0 ** -23 * size + 4 * 2.0 ** -24 * x.abs()).masked_fill(hidden, 0.0).amax(1)
                p = torch.softmax(x.masked_fill(hidden, -math.inf), 1)
                out[r0:r1, h] = p @ vv
                rel = HALF_BF16 + 2 * (delta + 2.0 ** -21) + 2 * n * 2.0 ** -23
                bound[r0:r1, h] = rel[:, None] * (p @ vv.abs())
    return out.view(T, -1), (bound + HALF_BF16 * out.abs()).view(T, -1)
