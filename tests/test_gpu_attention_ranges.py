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


@pytest.mark.parametrize("size", [1e-3, 1e-4, 1e-5, 1e-6])
@pytest.mark.parametrize("bits,D,H,G,B", PREFIX + [(4, 64, 1, 4, 2), (8, 128, 1, 4, 3)])
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
