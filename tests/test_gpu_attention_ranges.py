"""Decode attention over the whole range of its inputs: queries far below one, values of very
different magnitude side by side.  Against the 64-bit form, under bounds that go by the row's
own terms."""
import numpy as np
import pytest
import torch

import block_ref as ref
from int4_routed_expert_prerouter_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def i32(a):
    return dev(np.asarray(a, np.int32))


def call(c, q, lists, lens, pre, P, scale):
    """The call on the pages of `c` (ref.Cache): q [B, Hq, D] fp16, lists of pages -> [B, Hq, D]."""
    _, _, page, H, D = c.codes.shape
    W = max(1, max(len(p) for p in lists))
    table = np.full((len(lists), W), -1, np.int32)
    for b, p in enumerate(lists):
        table[b, :len(p)] = p
    cache = binding.KVCache(c.n_pages, page, H, D, c.bits, pages=dev(c.image))
    got = binding.attn_decode(cache, dev(q), i32(table), i32(lens), i32(pre) if P else None, P, scale)
    assert cache.error() == binding.EDGE0_OK
    return got.cpu().numpy().astype(np.float64)


def tokens_of(c, pages, n, pre, P):
    """K, V, V's two parts and |s z| of the prefix's and the sequence's own tokens."""
    return tuple(np.concatenate(x) for x in zip(c.tokens(pre, P), c.tokens(pages, n)))


SHAPES = [(4, 64, 2, 4), (4, 128, 2, 4), (4, 256, 1, 8), (8, 64, 2, 4), (8, 128, 2, 4), (8, 256, 1, 8), (4, 64, 1, 16), (4, 128, 1, 16),
          (4, 256, 1, 16), (8, 128, 1, 16)]


@pytest.mark.parametrize("size", [1e-3, 1e-4, 1e-5, 1e-6])
@pytest.mark.parametrize("bits,D,H,G", SHAPES)
def test_small_queries_over_own_contexts(bits, D, H, G, size):
    """Queries of that size, subnormal fp16 among them, with a scale that makes ordinary scores; the
    sequence's other heads are up to 2^12 larger and smaller."""
    rng = np.random.default_rng(D + G)
    c = ref.Cache(14, 64, H, D, bits, rng)
    lens, lists = [777, 40, 1], [list(range(13)), [13], [5]]
    q = rng.standard_normal((3, H * G, D)) * size
    q[2] *= 2.0 ** rng.integers(-12, 13, (H * G, 1))
    q = q.astype(np.float16)
    scale = D ** -0.5 / size
    got = call(c, q, lists, lens, [], 0, scale)
    for b in range(3):
        want, bound = ref.attention(q[b].astype(np.float64), *tokens_of(c, lists[b], lens[b], [], 0), scale)
        err = np.abs(got[b] - want)
        assert (err <= bound).all(), (b, (err / bound).max())


# (bits, D, H, G, sequences): from so many query rows per K/V head on the prefix runs on the fifth-generation tensor cores
PREFIX = [(4, 64, 1, 8, 9), (4, 128, 2, 4, 6), (4, 256, 1, 16, 3), (8, 64, 1, 8, 9), (8, 128, 2, 4, 6), (8, 256, 1, 16, 3)]
# fewer rows: the kernel of the own contexts, 8, 16 and 32 rows at a time
FEW = [(4, 64, 1, 4, 2), (8, 128, 1, 4, 3), (4, 128, 1, 4, 1), (8, 64, 1, 16, 1), (4, 64, 1, 8, 5), (8, 64, 1, 16, 3), (4, 256, 1, 8, 3)]


@pytest.mark.parametrize("size", [1e-3, 1e-4, 1e-5, 1e-6])
@pytest.mark.parametrize("bits,D,H,G,B", PREFIX + FEW)
def test_small_queries_over_a_shared_prefix(bits, D, H, G, B, size):
    """As above; K's mean over each 64 dims is far from zero, so that the queries' sums count."""
    rng = np.random.default_rng(D + G)
    c = ref.Cache(14, 64, H, D, bits, rng, k_offset=2.0)
    pre, P = list(range(13)), 777
    q = rng.standard_normal((B, H * G, D)) * size
    q[B - 1] *= 2.0 ** rng.integers(-12, 13, (H * G, 1))
    q = q.astype(np.float16)
    scale = D ** -0.5 / size
    lens = [5 * (b % 2) for b in range(B)]
    got = call(c, q, [[13]] * B, lens, pre, P, scale)
    for b in range(B):
        want, bound = ref.attention(q[b].astype(np.float64), *tokens_of(c, [13], lens[b], pre, P), scale)
        err = np.abs(got[b] - want)
        assert (err <= bound).all(), (b, (err / bound).max())


def row_bound(q, k, v, parts, sz, scale):
    """ref.attention with a bound that does not grow with the largest V: o [Hq, D], bound.  As there:
    the result's rounding, the weights' rounding to fp16, their own errors a_j, fp32 sums.  In place
    of its terms for weights below fp16's normal range, with p the softmax weights before they are
    normalised (the largest between 2^-4 and 1), es the power of two above the largest s so far (at
    most 2^17, as s <= 65504) and w = 128 p s / es the fp16 weight, whose rounding is off by no more
    than w itself:
    - s >= 2^-9 es, then p < 2^-12: half a subnormal step, 2^-25 es / 128 <= 2^-23 s, times |q - z| <= z
      and times r: min(p, 2^-23) (|s z| + |v|);
    - s below 2^-9 es: what the rounding leaves is carried in units of 2^-48, off by 2^-49 es / 128
      <= 2^-39 at most, times |q - z| <= 128."""
    Hq, D = q.shape
    n, H, _ = k.shape
    G = Hq // H
    o, bound = np.zeros((Hq, D)), np.full((Hq, D), 2.0 ** -24)
    for h in range(Hq):
        kk, vv, pp, big = (a[:, h // G] for a in (k, v, parts, sz))
        sc = scale * (kk @ q[h])
        p = np.exp(sc - sc.max())
        total = p.sum()
        o[h] = p @ vv / total
        mag = 3 * np.abs(kk).reshape(n, -1, 64).max(-1).repeat(64, -1)
        a = scale * (mag @ np.abs(q[h])) * (D / 16 + D / 64) * 2.0 ** -23 + np.abs(sc) * 2.0 ** -22 + 2.0 ** -20
        bound[h] += (2.0 ** -11 + p @ a / total) * np.abs(o[h]) + (p * (2.0 ** -11 + a + (n / 16 + 64) * 2.0 ** -23)) @ pp / total
        bound[h] += (np.where(p < 2.0 ** -8, np.minimum(p, 2.0 ** -23), 0) @ (big + np.abs(vv)) + n * 2.0 ** -32) / total
    return o, bound


def outlier_case(bits, D, H, G, size, rng, at, groups):
    """A cache of V's of `size` whose tokens `at` hold V's up to 30,000 in some groups of 64 dims and a
    key against all queries but the last of each group of heads, which sees nothing else."""
    c = ref.Cache(14, 64, H, D, bits, rng)
    x = c.x.astype(np.float16)                       # [pages, 2, tokens, H, D]
    x[:, 1] = (rng.standard_normal(x[:, 1].shape) * size).astype(np.float16)
    u = rng.standard_normal(D)
    u *= (40.0 * D ** 0.5 / (u @ u)) ** 0.5          # u . u / sqrt(D) = 40
    for t in at:
        x[t // 64, 0, t % 64] = (-u).astype(np.float16)
        for g in groups:
            x[t // 64, 1, t % 64, :, 64 * g:64 * g + 64] = (rng.uniform(-1, 1, (H, 64)) * 30000).astype(np.float16)
    c.codes, c.s, c.b = ref.quantise(x, bits)
    c.image, c.x = ref.page_image(c.codes, c.s, c.b, bits), ref.values(c.codes, c.s, c.b)
    q = u + 0.3 * rng.standard_normal((H * G, D))
    q[G - 1::G] = -u
    return c, q


@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 1e-4])
@pytest.mark.parametrize("bits,D,H,G", SHAPES)
def test_large_values_without_weight_in_own_contexts(bits, D, H, G, size):
    """Tokens of next to no weight and large values leave the small values of the others alone, before
    and behind them, also where another query sees those tokens only."""
    rng = np.random.default_rng(D + G + bits)
    c, q = outlier_case(bits, D, H, G, size, rng, range(3, 832, 24), range(D // 128 + 1))
    lens, lists = [777, 40, 330], [list(range(13)), [0], list(range(13))]
    qs = np.stack([q, q * 0.9, q * 1.1]).astype(np.float16)
    got = call(c, qs, lists, lens, [], 0, D ** -0.5)
    for b in range(3):
        want, bound = row_bound(qs[b].astype(np.float64), *tokens_of(c, lists[b], lens[b], [], 0), D ** -0.5)
        err = np.abs(got[b] - want)
        assert (err <= bound).all(), (b, (err / bound).max())


@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 1e-4])
@pytest.mark.parametrize("bits,D,H,G,B", PREFIX + FEW)
def test_large_values_without_weight_in_a_shared_prefix(bits, D, H, G, B, size):
    """As above, in the prefix (pages 0 to 12, in any order) and in the sequences' own tokens behind it."""
    rng = np.random.default_rng(D + G + bits)
    c, q = outlier_case(bits, D, H, G, size, rng, range(3, 896, 24), range(D // 128 + 1))
    pre, P = rng.permutation(13).tolist(), 12 * 64 + 9
    qs = np.stack([q * (1 + 0.02 * b) for b in range(B)]).astype(np.float16)
    lens = [17 * (b % 3) for b in range(B)]
    got = call(c, qs, [[13]] * B, lens, pre, P, D ** -0.5)
    for b in range(B):
        want, bound = row_bound(qs[b].astype(np.float64), *tokens_of(c, [13], lens[b], pre, P), D ** -0.5)
        err = np.abs(got[b] - want)
        assert (err <= bound).all(), (b, (err / bound).max())


@pytest.mark.parametrize("bits,D,H,G,B", PREFIX + FEW)
def test_zero_and_constant_groups_beside_large_values(bits, D, H, G, B):
    """Groups of zeros (a whole tile of them first) and constant ones beside tokens of every size."""
    rng = np.random.default_rng(D * bits + B)
    c = ref.Cache(14, 64, H, D, bits, rng)
    x = c.x.astype(np.float16)
    x[:, 1] = (rng.standard_normal(x[:, 1].shape) * 1e-3).astype(np.float16)
    x[:2, 1] = 0
    for i, v in enumerate((0.0, 1e-3, -1e-3, 2.0 ** -24, -300.0, 0.0)):
        x[2 + i::6, 1, i::7, :, :64] = v
    u = rng.standard_normal(D)
    u *= (40.0 * D ** 0.5 / (u @ u)) ** 0.5
    for t in range(3, 64, 24):
        x[2:, 0, t] = (-u).astype(np.float16)
        x[2:, 1, t] = (rng.uniform(-1, 1, (H, D)) * 30000).astype(np.float16)
    c.codes, c.s, c.b = ref.quantise(x, bits)
    c.image, c.x = ref.page_image(c.codes, c.s, c.b, bits), ref.values(c.codes, c.s, c.b)
    q = np.stack([u + 0.3 * rng.standard_normal((H * G, D))] * B).astype(np.float16)
    sw, bw = (np.repeat(a[:, 1].astype(np.float64), 64, -1) for a in (c.s, c.b))
    z = 2.0 ** (bits - 1)
    # a constant group's value b is |b| times (0 - z) + (z +- 1): its part that meets a code is z |b|
    parts = np.where(sw == 0, (2 * z + 1) * np.abs(bw), np.abs(sw * (c.codes[:, 1].astype(np.float64) - z)) + np.abs(sw * z + bw))
    big = np.where(sw == 0, np.abs(bw), sw) * z
    flat = lambda a, pages, m: a[np.asarray(pages)].reshape(-1, H, D)[:m]
    for P, n in ((777, 60), (0, 860), (128, 0)):
        pre, own = list(range(13)), [13] if P else list(range(14))
        got = call(c, q, [own] * B, [n] * B, pre, P, D ** -0.5)
        for b in range(B):
            k, v, pp, zz = (np.concatenate([flat(a, pre, P), flat(a, own, n)]) for a in (c.x[:, 0], c.x[:, 1], parts, big))
            want, bound = row_bound(q[b].astype(np.float64), k, v, pp, zz, D ** -0.5)
            err = np.abs(got[b] - want)
            assert (err <= bound).all(), (P, n, b, (err / bound).max())
