"""Plain 64-bit forms of the projection, KV-cache and attention calls, for their tests:
numpy on the CPU, written from the definitions in edge0.h."""
import numpy as np

GROUP = 64


def dequant_q4(q, s, b):
    """q [out, in/8] int32, s, b [out, in/64] fp16 -> W [out, in] float64."""
    q = q.astype(np.int64) & 0xFFFFFFFF
    nib = (q[:, :, None] >> (4 * np.arange(8))) & 15
    w = nib.reshape(q.shape[0], -1, GROUP).astype(np.float64)
    w = w * s.astype(np.float64)[..., None] + b.astype(np.float64)[..., None]
    return w.reshape(q.shape[0], -1)


def quantise(x, bits):
    """x [..., D] fp16 -> codes uint8 [..., D], s, b fp16 [..., D/64]."""
    top = 2 ** bits - 1
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    bad = ~np.isfinite(g).all(-1)
    w = np.where(bad[..., None], 0.0, g.astype(np.float64))
    mn, mx = w.min(-1), w.max(-1)
    s = ((mx - mn).astype(np.float32) / np.float32(top)).astype(np.float16)
    over = s.astype(np.float64) * top + mn >= 65520          # would round to infinity: the next fp16 below
    s = np.where(over, (s.view(np.uint16) - over).astype(np.uint16).view(np.float16), s)
    d = np.where(s == 0, 1.0, s.astype(np.float64))
    q = np.clip(np.rint((w - mn[..., None]) / d[..., None]), 0, top)
    q = np.where((s == 0)[..., None] | bad[..., None], 0, q).astype(np.uint8)
    nan = np.float16(np.nan)
    return q.reshape(x.shape), np.where(bad, nan, s), np.where(bad, nan, mn.astype(np.float16))


def values(codes, s, b, wide=np.float64):
    g = codes.reshape(*codes.shape[:-1], -1, GROUP).astype(wide)
    return (g * s.astype(wide)[..., None] + b.astype(wide)[..., None]).reshape(codes.shape)


def turn(R, r):
    return r & 7 if R >= 128 else (r * R // 128) & (R // 16 - 1)


def page_image(codes, s, b, bits):
    """Bytes of pages: codes [n, 2, page_tokens, H, D] (K, V), s, b [n, 2, page_tokens, H, D/64]."""
    n, _, P, H, D = codes.shape
    R, G = D * bits // 8, D // GROUP
    half = 16 * (R + 4 * G)
    out = np.zeros((n, H, P // 16, 2, half), np.uint8)
    rows = codes if bits == 8 else codes[..., 0::2] | (codes[..., 1::2] << 4)
    sb = np.stack([s, b], -1).astype(np.float16)                   # [n, 2, P, H, G, 2]
    for t in range(P):
        strip, r = divmod(t, 16)
        for c in range(R // 16):
            at = r * R + 16 * (c ^ turn(R, r))
            out[:, :, strip, :, at:at + 16] = rows[:, :, t, :, 16 * c:16 * c + 16].transpose(0, 2, 1, 3)
        at = 16 * R + r * 4 * G
        img = np.ascontiguousarray(sb[:, :, t]).view(np.uint8).reshape(n, 2, H, 4 * G)
        out[:, :, strip, :, at:at + 4 * G] = img.transpose(0, 2, 1, 3)
    return out.reshape(n, -1)


class Cache:
    """A pool of pages with what they stand for."""

    def __init__(self, n_pages, page_tokens, H, D, bits, rng, k_offset=0.0, v_scale=1.0):
        x = rng.standard_normal((n_pages, 2, page_tokens, H, D))
        x[:, 0] += k_offset
        x[:, 1] *= v_scale
        self.codes, self.s, self.b = quantise(x.astype(np.float16), bits)
        self.bits, self.page_tokens, self.n_pages = bits, page_tokens, n_pages
        self.image = page_image(self.codes, self.s, self.b, bits)
        self.x = values(self.codes, self.s, self.b)

    def tokens(self, pages, n):
        """Of n tokens in a list of pages: K, V [n, H, D]; the magnitudes of V's two parts
        |s (q - z)| + |s z + b|, z half the code range; and |s z|."""
        pages = np.asarray(pages, np.int64)
        z = 2.0 ** (self.bits - 1)
        s, b = (np.repeat(a[pages, 1].astype(np.float64), GROUP, -1) for a in (self.s, self.b))
        parts = np.abs(s * (self.codes[pages, 1].astype(np.float64) - z)) + np.abs(s * z + b)
        return tuple(a.reshape(-1, *self.x.shape[3:])[:n] for a in (self.x[pages, 0], self.x[pages, 1], parts, s * z))


def attention(q, k, v, parts, sz, scale):
    """One sequence: q [Hq, D]; k, v, parts, sz [n, H, D] -> o [Hq, D] and how far an fp16
    result may be off, [Hq, D].

    With p the normalised weights the bound adds up
    - the result's rounding: half an fp16 step, 2^-11 |o|, and 2^-24 where that is subnormal;
    - the rounding of each weight to fp16 when it meets a code: 2^-11 of its term of V's
      parts; where p s is below fp16's normal range half its subnormal step, 2^-25 of 2^e
      2^-7 (2^e the largest s, at most doubled to a power of two), times the code's distance
      from z, and, while s >= 2^-9 2^e (so that p < 2^-12 of the reference, which is within
      a factor 2^4 below the maximum), times r = b / s + z: |v| / s in all, 2^-23 |v|;
    - the weights' own error a_j = the fp32 score's (D / 16 matrix steps and D / 64 group sums
      of terms that add up to at most |q| (3 max |k| of the group), each off by 2^-23, and the
      exponent's argument by 2^-22 of itself) + 2^-20 of the exponential: p a on V's parts
      and, through the normaliser, (p . a) |o|;
    - fp32 sums over the tokens: n / 16 + 64 steps of 2^-23 of V's parts."""
    Hq, D = q.shape
    n, H, _ = k.shape
    G = Hq // H
    o, bound = np.zeros((Hq, D)), np.full((Hq, D), 2.0 ** -24)
    if n == 0:
        return o, bound
    for h in range(Hq):
        kk, vv, pp, big = (a[:, h // G] for a in (k, v, parts, sz))
        sc = scale * (kk @ q[h])
        p = np.exp(sc - sc.max())
        total = p.sum()
        p /= total
        o[h] = p @ vv
        mag = 3 * np.abs(kk).reshape(n, -1, GROUP).max(-1).repeat(GROUP, -1)
        a = scale * (mag @ np.abs(q[h])) * (D / 16 + D / 64) * 2.0 ** -23 + np.abs(sc) * 2.0 ** -22 + 2.0 ** -20
        bound[h] += (2.0 ** -11 + p @ a) * np.abs(o[h]) + (p * (2.0 ** -11 + a + (n / 16 + 64) * 2.0 ** -23)) @ pp
        bound[h] += n * 2.0 ** -32 * 2 * big.max(0) / total
        bound[h] += 2.0 ** -23 / total * (np.abs(vv) * (p * total <= 2.0 ** -12)[:, None]).sum(0)
    return o, bound
