"""Attention of rows that see some of a sequence's tokens, in 64 bits on the GPU, for the tests of
attention of prompts and of drafted tokens."""
import math

import torch


def attend(q, k, v, seen, scale, k_abs=None, v_abs=None, v_small=None):
    """q [n, Hq, D], k, v [m, H, D] float64, seen [n, m] -> o [n, Hq, D] and how far an fp16 result may
    be off.  Rows that see nothing: zeros, exactly.  A NaN in v is one in the rows that see it, and in no others.

    k_abs, v_abs: the magnitudes of the parts that K and V enter in (|s (q - z)| + |s z + b| of the cache's groups), where
    they are not one fp16 each.  With p the normalised weights the bound adds up
    - the result's rounding: half an fp16 step, 2^-11 |o|, and 2^-25 where that is subnormal;
    - each weight's rounding to fp16, 2^-11 of its term, and half a subnormal step where it is below fp16's
      normal range, 2^-25 against a largest weight of at least 2^11: sum v_small 2^-36 / total (v_small: |v|, or what
      a weight's own scale makes of it);
    - the weights' own error a_j = the fp32 score's (D / 16 matrix steps and one more of terms that add up to
      |q| . k_abs, each off by 2^-23, the factor scale log2(e) and the exponent's argument by 2^-22 of themselves) + 2^-20 of the
      exponential: p a on |v| and, through the normaliser, (p . a) |o|;
    - fp32 sums over the tokens, m / 16 + 64 steps of 2^-23 of v_abs, and 2^-21 of it where V enters in parts."""
    n, Hq, D = q.shape
    m, H, _ = k.shape
    o = torch.zeros_like(q)
    bound = torch.zeros_like(q)
    if m == 0 or n == 0:
        return o, bound
    some = seen.any(1)
    for h in range(Hq):
        kk, vv = k[:, h // (Hq // H)], v[:, h // (Hq // H)]
        nan = torch.isnan(vv)
        vv = vv.masked_fill(nan, 0.0)
        s = scale * (q[:, h] @ kk.T)
        s = s.masked_fill(~seen, -math.inf)
        top = s.amax(1, keepdim=True)
        e = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
        total = e.sum(1, keepdim=True)
        p = e / torch.where(some[:, None], total, torch.ones_like(total))
        o[:, h] = (p @ vv).masked_fill(seen.double() @ nan.double() > 0, math.nan)
        ka = kk.abs() if k_abs is None else k_abs[:, h // (Hq // H)]
        a = scale * (q[:, h].abs() @ ka.T) * (D / 16 + 1) * 2.0 ** -23 + s.masked_fill(~seen, 0.0).abs() * 2.0 ** -21 + 2.0 ** -20
        pa = p * a
        av = vv.abs()
        parts = av if v_abs is None else v_abs[:, h // (Hq // H)].masked_fill(nan, 0.0)
        tiny = av if v_small is None else v_small[:, h // (Hq // H)].masked_fill(nan, 0.0)
        small = 2.0 ** -36 * (seen.double() @ tiny) / torch.where(some[:, None], total, torch.ones_like(total))
        bound[:, h] = (2.0 ** -11 + pa.sum(1, keepdim=True)) * o[:, h].abs() + 2.0 ** -25 + small + (pa + 2.0 ** -11 * p) @ av + \
            ((m / 16 + 64) * 2.0 ** -23 + (0.0 if v_abs is None else 2.0 ** -21)) * (p @ parts)
    bound[~some] = 0
    return o, bound


def causal(n, m, device):
    return torch.arange(m, device=device)[None, :] <= torch.arange(n, device=device)[:, None] + (m - n)


def close(got, o, bound):
    """Whether got lies within its bound of o, NaN where that is."""
    nan = torch.isnan(o)
    return bool((torch.isnan(got) == nan).all()) and bool(((got.double() - o).abs() <= bound)[~nan].all())
