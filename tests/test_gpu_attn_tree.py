"""Attention of drafted tokens over the cache on the GPU against its definition in 64 bits, and with the
calls around it: rotary positions, append, compaction, decode attention."""
import math
import threading

import numpy as np
import pytest
import torch

import block_ref as ref
import flash_ref
from int4_routed_expert_prerouter_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def i32(a):
    return torch.tensor(np.asarray(a, np.int64).astype(np.uint32).view(np.int32), device=DEV)


def rows(T, *shape):
    return torch.randn(T, *shape, device=DEV).half()


class Pool:
    """A pool of quantised tokens with what they stand for, on the GPU."""

    def __init__(self, n_pages, page, H, D, bits, seed=0, k_offset=0.0, v_scale=1.0, spread=1.0):
        rng = np.random.default_rng(seed)
        few = min(n_pages, 12)
        x = rng.standard_normal((few, 2, page, H, D)) * spread
        x[:, 0] += k_offset
        x[:, 1] *= v_scale
        codes, s, b = ref.quantise(x.astype(np.float16), bits)
        rep = -(-n_pages // few)
        tile = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV).repeat(rep, *[1] * (a.ndim - 1))[:n_pages].contiguous()
        self.page, self.bits = page, bits
        self.image = tile(ref.page_image(codes, s, b, bits))
        self.cache = binding.KVCache(n_pages, page, H, D, bits, pages=self.image)
        self.codes, self.s, self.b = tile(codes).double(), tile(s).double(), tile(b).double()

    def tokens(self, pages, n):
        """K, V [n, H, D]; |s (q - z)| + |s z + b| of K and of V; what V's terms lose to a subnormal weight, which
        meets V / m with s = m 2^e, m at least 1 where s is at least 2^-10 (twice: 2^10 instead of 2^11)."""
        z = 2.0 ** (self.bits - 1)
        pages = torch.as_tensor(np.asarray(pages)[:-(-n // self.page)], device=DEV)
        wide = lambda a: a[pages].repeat_interleave(64, -1)
        q, s, b = self.codes[pages], wide(self.s), wide(self.b)
        flat = lambda a: a.flatten(0, 1)[:n]
        x = s * q + b
        parts = (s * (q - z)).abs() + (s * z + b).abs()
        small = 2 * x[:, 1].abs() * torch.clamp(2.0 ** -10 / torch.where(s[:, 1] == 0, 1.0, s[:, 1]), min=1.0)
        return flat(x[:, 0]), flat(x[:, 1]), flat(parts[:, 0]), flat(parts[:, 1]), flat(small)


def visible(n, x, mask, device=DEV):
    """[x, n + x] of the context of n tokens and x drafted ones (mask: [x, words] numpy uint32, or None)."""
    if mask is None:
        tree = np.tril(np.ones((x, x), bool))
    else:
        bits = np.unpackbits(np.ascontiguousarray(mask).astype("<u4").view(np.uint8), axis=1, bitorder="little").astype(bool)
        tree = np.zeros((x, x), bool)
        w = min(x, bits.shape[1])
        tree[:, :w] = bits[:, :w]
    return torch.from_numpy(np.concatenate([np.ones((x, n), bool), tree], 1)).to(device)


def check(got, pool, q, table, lens, cu, mask=None, scale=None):
    D = q.shape[2]
    for b in range(len(lens)):
        x, n = cu[b + 1] - cu[b], lens[b]
        if n < 0 or x == 0:
            continue
        r = slice(cu[b], cu[b + 1])
        k, v, *parts = pool.tokens(table[b], n + x)
        o, bound = flash_ref.attend(q[r].double(), k, v, visible(n, x, None if mask is None else mask[r]), scale or D ** -0.5, *parts)
        assert flash_ref.close(got[r], o, bound), (b, n, x, ((got[r].double() - o).abs() - bound).nan_to_num(0.0).max().item())


def tree_words(counts, words, rng):
    """Ancestors and itself in random trees."""
    out = []
    for x in counts:
        mine = []
        for j in range(x):
            parent = int(rng.integers(max(0, j - 4), j + 1)) - 1
            mine.append((mine[parent] if parent >= 0 else 0) | 1 << j)
        out += [[(m >> 32 * w) & 0xFFFFFFFF for w in range(words)] for m in mine]
    return np.array(out, np.uint32).reshape(-1, words)


def case(bits, D, H, G, page, lens, counts, seed=0, chain=False, **kw):
    rng = np.random.default_rng(seed)
    need = [max(1, -(-(max(n, 0) + x) // page)) for n, x in zip(lens, counts)]
    W, total = max(need), sum(need) + 1
    pool = Pool(total, page, H, D, bits, seed, **kw)
    order, table, at = rng.permutation(total), np.full((len(lens), W), -1), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cu = [0] + [int(c) for c in np.cumsum(counts)]
    q = rows(cu[-1], H * G, D)
    mask = None if chain else tree_words(counts, -(-max(counts) // 32), rng)
    return pool, q, table, list(lens), cu, mask


def call(pool, q, table, lens, cu, mask, **kw):
    return binding.attn_tree(pool.cache, q, i32(table), i32(lens), i32(cu), None if mask is None else i32(mask), **kw)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 4), (3, 5), (1, 8), (1, 64)])
@pytest.mark.parametrize("lens,counts", [([5], [1]), ([0, 37, 300], [3, 1, 7]), ([100, 0, 129], [33, 64, 40])])
@pytest.mark.parametrize("chain", [False, True])
def test_heads_and_lengths(bits, D, H, G, lens, counts, chain):
    c = case(bits, D, H, G, 16, lens, counts, chain=chain)
    check(call(*c), *c)
    assert c[0].cache.error() == binding.EDGE0_OK


@pytest.mark.parametrize("bits,D", [(4, 128), (8, 64), (8, 256), (4, 64), (8, 128), (4, 256)])
@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("lens,counts", [([5000], [16]), ([2000, 1, 4097], [1, 200, 70]), ([130] * 5 + [1500], [12] * 6)])
@pytest.mark.parametrize("chain", [False, True])
def test_long_contexts(bits, D, page, lens, counts, chain):
    c = case(bits, D, 2, 4, page, lens, counts, chain=chain)
    check(call(*c), *c)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_scale,kw", [(1.0, dict(k_offset=30.0)), (1e-6, dict(k_offset=200.0)), (300.0, dict(spread=0.01)),
                                        (1.0, dict(k_offset=-1000.0)), (0.01, dict(spread=3000.0)), (1.0, dict(v_scale=3e4)),
                                        (3e4, dict(spread=1e-5))])
def test_magnitudes(bits, D, q_scale, kw):
    c = list(case(bits, D, 1, 4, 32, [700, 20], [10, 40], **kw))
    c[1] = (c[1].float() * q_scale).half()
    check(call(*c), *c)


def written(k, v, page, bits):
    """A cache of the rows k, v [n, H, D] in pages in reverse order, with their table, what its groups stand for (K, V in 64 bits) and the
    magnitudes of V's parts."""
    n, H, D = k.shape
    W = -(-n // page)
    cache = binding.KVCache(W, page, H, D, bits, device=DEV)
    table = i32(np.arange(W)[::-1].copy()[None])
    binding.kv_append(cache, k, v, table, i32([0]), i32([0, n]))
    out = []
    for x in (k, v):
        codes, s, b = (torch.from_numpy(np.ascontiguousarray(a)).to(DEV).double() for a in ref.quantise(x.cpu().numpy(), bits))
        s, b, z = s.repeat_interleave(64, -1), b.repeat_interleave(64, -1), 2.0 ** (bits - 1)
        out.append((s * codes + b, (s * (codes - z)).abs() + (s * z + b).abs()))
    return cache, table, out[0][0], *out[1]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_size,k_size,scale", [(2001.0, 1111.0, 1.0), (3001.0, 16008.0, None), (50016.0, 40032.0, None),
                                                 (1.375, 1.125, 1e6), (60000.0, 50016.0, 1e6), (513.0, 1025.0, 3.0)])
@pytest.mark.parametrize("n,x", [(250, 12), (100, 60), (3000, 9)])
def test_scores_beyond_what_fp32_tells_apart(bits, D, q_size, k_size, scale, n, x):
    """Queries and keys of one dim each that is not zero, of a few classes: the largest scores of a row weigh the same, all others
    nothing, whatever their size (exponents of 2^21 up to 2^50)."""
    H, G, gen = 2, 4, torch.Generator().manual_seed(D + n)
    size = lambda m, h, a: (torch.where(torch.rand(m, h, generator=gen) < 0.3, -a, a) * 0.5 ** torch.randint(0, 3, (m, h), generator=gen)).half().to(DEV)
    q, k, v = (torch.zeros(m, h, D, dtype=torch.float16, device=DEV) for m, h in ((x, H * G), (n + x, H), (n + x, H)))
    q[..., 3], k[..., 3], v = size(x, H * G, q_size), size(n + x, H, k_size), rows(n + x, H, D)
    cache, table, kk, vv, parts = written(k, v, 32, bits)
    mask = tree_words([x], 2, np.random.default_rng(n))
    for m in (None, mask):
        got = binding.attn_tree(cache, q, table, i32([n]), i32([0, x]), None if m is None else i32(m), scale=scale)
        s = torch.einsum("nhd,mhd->hnm", q.double(), kk.repeat_interleave(G, 1)).masked_fill(~visible(n, x, m), -float("inf"))
        p = (s == s.amax(2, keepdim=True)).double()
        p /= p.sum(2, keepdim=True)
        o, a, b = (torch.einsum("hnm,mhd->nhd", p, y.repeat_interleave(G, 1)) for y in (vv, vv.abs(), parts))
        # the result's rounding, each weight's (one number, so the sum's too), fp32 sums
        bound = 2.0 ** -11 * o.abs() + 2.0 ** -25 + 2.0 ** -11 * a + (((n + x) / 16 + 64) * 2.0 ** -23 + 2.0 ** -21) * b
        # Exponents below 2^22: a score less the reference is formed in one fused step, but in the tile that sets the reference, where
        # both are rounded sums, and by a set of warps whose reference is an older one, which adds their difference: two roundings
        # by half an fp32 step e of the exponent, so equal scores' weights differ by a factor of up to 2^e, and with w in (1 - t, 1 + t),
        # t = 2^e - 1, sum w p v / sum w p is off by at most t (sum p |v| + |o|).
        top = (s.amax(2).abs() * (scale or D ** -0.5) * math.log2(math.e)).T[:, :, None]
        e = torch.where(top < 2.0 ** 22, 2.0 ** (torch.floor(torch.log2(top)) - 23), 0.0)
        bound += (2.0 ** e - 1) * (a + o.abs())
        err = (got.double() - o).abs()
        assert (err <= bound).all(), (err - bound).nan_to_num(99.0).max().item()
    assert cache.error() == binding.EDGE0_OK


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_size,k_size,scale", [(20000.0, 10000.0, None), (3000.0, 3000.0, None), (3000.0, 10.0, 1e4), (1.0, 1.0, 1e6)])
@pytest.mark.parametrize("x", [12, 60])
def test_rows_of_huge_scores_beside_ordinary_ones(bits, D, q_size, k_size, scale, x):
    """Finite, between the values that they are means of, and nothing to the rows beside them."""
    n, H, G = 900, 2, 4
    k, v = (rows(n + x, H, D).float() * k_size).clamp(-60000, 60000).half(), rows(n + x, H, D)
    cache, table, kk, vv, _ = written(k, v, 16, bits)
    q = (rows(x, H * G, D).float() / (k_size * (scale or D ** -0.5) * D ** 0.5)).half()
    args = table, i32([n]), i32([0, x]), i32(tree_words([x], 2, np.random.default_rng(x)))
    clean = binding.attn_tree(cache, q, *args, scale=scale)
    far = torch.rand(x, H * G, device=DEV) < 0.3
    huge = torch.where(far[:, :, None], (rows(x, H * G, D).float() * q_size).clamp(-60000, 60000).half(), q)
    got = binding.attn_tree(cache, huge, *args, scale=scale)
    assert torch.equal(got[~far], clean[~far])
    wide = vv.repeat_interleave(G, 1)
    assert ((got >= wide.amin(0) - 0.01) & (got <= wide.amax(0) + 0.01)).all() and cache.error() == binding.EDGE0_OK
    # one token far ahead of the others is what a row gives
    s = (scale or D ** -0.5) * torch.einsum("nhd,mhd->hnm", huge.double(), kk.repeat_interleave(G, 1))
    s = s.masked_fill(~visible(n, x, args[3].cpu().numpy().view(np.uint32)), -float("inf"))
    two = s.topk(2, dim=2)
    ahead = (two.values[..., 0] - two.values[..., 1] > 40 + two.values.abs().amax(2) * 2.0 ** -14).T          # [x, heads]
    best = torch.gather(wide.permute(1, 0, 2), 1, two.indices[..., :1].expand(-1, -1, D)).transpose(0, 1)       # [x, heads, D]
    assert ahead[far].float().mean() > 0.2 and ((got.double() - best).abs() <= 2.0 ** -9 * best.abs() + 1e-4)[ahead].all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_size", [1.0, 300.0])
@pytest.mark.parametrize("n,x", [(0, 40), (150, 9)])
def test_groups_around_zero(bits, D, q_size, n, x):
    """Offsets that take off what the middle code stands for: most codes' values are a few steps, far smaller than the offset, and
    those of the middle code are zero."""
    H, G, page, z = 2, 4, 16, 2 ** (bits - 1)
    pool = Pool(-(-(n + x) // page), page, H, D, bits)
    rng, shape = np.random.default_rng(D), tuple(pool.codes.shape)
    codes = rng.integers(z - 2, z + 3, shape)
    s = (rng.uniform(0.01, 0.03, shape[:-1] + (D // 64,))).astype(np.float16)
    b = (-s.astype(np.float64) * z).astype(np.float16)          # (a power of two times s: exact)
    pool.image.copy_(torch.from_numpy(ref.page_image(codes.astype(np.uint8), s, b, bits)).to(DEV))
    pool.codes, pool.s, pool.b = (torch.from_numpy(np.ascontiguousarray(a)).to(DEV).double() for a in (codes, s, b))
    q, table = (rows(x, H * G, D).float() * q_size).half(), np.arange(shape[0])[None]
    args = pool, q, table, [n], [0, x], None
    # V's parts: every other token's codes are taken about z - 1.  Pool.tokens has them about z for all, where both parts of a middle
    # code are 0; about z - 1 they are s and -s, and fp32 sums of them are off by 2^-21 (s + s) at most, not by 0.
    tokens, odd = pool.tokens, torch.arange(n + x, device=DEV)[:, None, None] % 2
    wide = lambda a: a[:, 1].flatten(0, 1)[:n + x].repeat_interleave(64, -1)
    ws, wb, wq = wide(pool.s), wide(pool.b), pool.codes[:, 1].flatten(0, 1)[:n + x]
    pool.tokens = lambda pages, m: (*tokens(pages, m)[:3], (ws * (wq - (z - odd))).abs() + (ws * (z - odd) + wb).abs(), tokens(pages, m)[4])
    check(call(*args), *args)


def test_masks():
    """Rows that see nothing, drafted tokens behind the row, bits behind the sequence's tokens, words beyond need."""
    pool, q, table, lens, cu, _ = case(4, 128, 2, 4, 16, [0, 50, 0], [40, 40, 3])
    rng = np.random.default_rng(1)
    mask = rng.integers(0, 2 ** 32, (83, 5), dtype=np.uint64).astype(np.uint32)
    mask[0:10] = 0
    mask[80:] = 0xFFFFFFF8           # nothing but tokens that are not there
    got = call(pool, q, table, lens, cu, mask)
    check(got, pool, q, table, lens, cu, mask)
    assert not got[:10].any() and not got[80:].any()
    assert pool.cache.error() == binding.EDGE0_OK


@pytest.mark.parametrize("D,bits", [(64, 8), (128, 4), (256, 4)])
def test_slices_padding_and_scale(D, bits):
    H, G = 2, 3
    pool, _, table, lens, cu, mask = case(bits, D, H, G, 16, [100, 50, 20, 0], [5, 9, 4, 6])
    lens[1] = -1
    lead, T = 3, cu[-1] + 7
    cu = [c + lead for c in cu]
    wide = rows(T, (H * G + 2) * D)
    q = wide[:, D:D + H * G * D].unflatten(1, (H * G, D))
    words = np.zeros((T, mask.shape[1]), np.uint32)
    words[lead:lead + len(mask)] = mask
    room = torch.full((T, H * G * D + 16), 7.0, dtype=torch.float16, device=DEV)
    got = call(pool, q, table, lens, cu, words, scale=0.2, out=room[:, 8:8 + H * G * D].unflatten(1, (H * G, D)))
    check(got, pool, q, table, lens, cu, words, scale=0.2)
    assert (room[:, :8] == 7).all() and (room[:, 8 + H * G * D:] == 7).all()
    assert (room[:lead] == 7).all() and (room[cu[-1]:] == 7).all() and (room[cu[1]:cu[2]] == 7).all()


@pytest.mark.parametrize("bits,D", [(4, 128), (8, 256), (4, 64)])
@pytest.mark.parametrize("what", [0, 1])
def test_groups_of_nan_reach_the_rows_that_see_them(bits, D, what):
    """A non-finite K (what 0) or V (1) of one drafted token, and of tokens behind the last."""
    H, G, page, n, x = 2, 4, 16, 130, 20
    cache = binding.KVCache(12, page, H, D, bits, device=DEV)
    table, k, v = np.arange(12)[None], rows(180, H, D), rows(180, H, D)
    binding.kv_append(cache, k, v, i32(table), i32([0]), i32([0, 180]))
    q, rng = rows(x, H * G, D), np.random.default_rng(0)
    mask = tree_words([x], 1, rng)
    args = (i32(table), i32([n]), i32([0, x]), i32(mask))
    clean = binding.attn_tree(cache, q, *args)
    for at in (n + 3, n + 17, n + x, 179):
        bad = (k, v)[what][at:at + 1].clone()
        bad[0, 1, 5] = float("inf")
        kv = (bad, v[at:at + 1]) if what == 0 else (k[at:at + 1], bad)
        binding.kv_append(cache, *kv, i32(table), i32([at]))
        got = binding.attn_tree(cache, q, *args)
        sees = np.array([at < n + x and bool(m >> (at - n) & 1) for m in mask[:, 0]])
        hit = torch.zeros(x, H * G, D, dtype=torch.bool, device=DEV)
        hit[torch.from_numpy(sees).to(DEV), G:, :64 if what else D] = True
        assert torch.equal(got[~hit], clean[~hit]), at
        assert torch.isnan(got[hit]).all(), at
        binding.kv_append(cache, k[at:at + 1], v[at:at + 1], i32(table), i32([at]))
    assert torch.equal(binding.attn_tree(cache, q, *args), clean) and cache.error() == binding.EDGE0_OK


def test_what_lies_outside_is_reported():
    pool, q, table, lens, cu, mask = case(4, 128, 2, 4, 16, [100, 20], [10, 12])
    c = pool.cache
    clean = call(pool, q, table, lens, cu, mask)
    assert c.error() == binding.EDGE0_OK
    for bad in (-3, c.n_pages, 2 ** 31 - 1):
        t = table.copy()
        t[1, 0] = bad
        got = call(pool, q, t, lens, cu, mask)
        assert c.error() == binding.EDGE0_EINVAL and torch.equal(got[:10], clean[:10])
        t[1, 0] = 0                                        # page 0 stands in
        assert torch.equal(call(pool, q, t, lens, cu, mask), got) and c.error() == binding.EDGE0_OK
    cap = table.shape[1] * 16
    for n in (cap - 5, cap, cap + 100, 2 ** 31 - 1):
        got = call(pool, q, table, [n, 20], cu, mask)
        assert c.error() == binding.EDGE0_EINVAL and torch.equal(got[10:], clean[10:]) and torch.isfinite(got).all()
    # more drafted tokens than the mask names: those behind are seen by no row
    pool, q, table, lens, cu, mask = case(4, 128, 1, 2, 16, [30], [40])
    got = call(pool, q, table, lens, cu, mask[:, :1])
    assert pool.cache.error() == binding.EDGE0_EINVAL
    check(got, pool, q, table, lens, cu, mask[:, :1])


@pytest.mark.parametrize("bits,D", [(8, 128), (4, 256)])
def test_pages_behind_2_31_bytes(bits, D):
    H, G, page, lens, counts = 4, 4, 128, [1500, 60], [9, 40]
    pool, q, table, lens, cu, mask = case(bits, D, H, G, page, lens, counts)
    few = pool.image.shape[0]
    times = (5 << 30) // pool.image.numel()
    pool.cache = binding.KVCache(few * times, page, H, D, bits, pages=pool.image.repeat(times, 1))
    rng = np.random.default_rng(0)
    far = np.where(table < 0, -1, table + few * rng.integers(times // 2, times, table.shape))
    got = call(pool, q, far, lens, cu, mask)
    check(got, pool, q, table, lens, cu, mask)
    assert pool.cache.error() == binding.EDGE0_OK


def test_bounds_outside_the_rows_touch_nothing():
    pool, q, table, lens, _, _ = case(4, 128, 1, 2, 16, [30, 20, 10, 5], [10, 10, 10, 10])
    guard = torch.full((120, 2, 128), 9.0, dtype=torch.float16, device=DEV)
    binding.attn_tree(pool.cache, q, i32(table), i32(lens), torch.tensor([-50, 10, 1000, 7, 2 ** 31 - 1], dtype=torch.int32, device=DEV),
                      out=guard[40:80])
    torch.cuda.synchronize()
    assert (guard[:40] == 9).all() and (guard[80:] == 9).all()


def test_in_a_graph_lengths_and_masks_are_read_at_replay():
    pool, q, table, lens, cu, mask = case(4, 128, 2, 4, 64, [3000, 100], [20, 30])
    a = [i32(table), i32(lens), i32(cu), i32(mask)]
    g = torch.cuda.CUDAGraph()
    binding.attn_tree(pool.cache, q, *a)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = binding.attn_tree(pool.cache, q, *a)
        two = binding.attn_tree(pool.cache, out, *a)
    for n, c, m in (([3000, 100], [0, 20, 50], mask), ([1, 90], [0, 7, 50], mask[::-1].copy()), ([2900, 0], [0, 50, 50], mask)):
        for t, x in zip(a[1:], (n, c, m)):
            t.copy_(i32(x))
        g.replay()
        torch.cuda.synchronize()
        want = binding.attn_tree(pool.cache, q, *a)
        assert torch.equal(out, want) and torch.equal(two, binding.attn_tree(pool.cache, want, *a))


@pytest.mark.parametrize("bits,D", [(4, 128), (8, 256), (4, 64)])
@pytest.mark.parametrize("lens", [[300, 5], [9000, 70]])
def test_without_waiting(bits, D, lens):
    pool, q, table, lens, cu, mask = case(bits, D, 2, 4, 64, lens + [-1], [10, 7, 3])
    clean = call(pool, q, table, lens, cu, mask, out=torch.full_like(q, 5.0))
    assert pool.cache.error() == binding.EDGE0_OK
    for _ in range(3):
        binding.set_wait_limit(0)
        try:
            got = call(pool, q, table, lens, cu, mask, out=torch.full_like(q, 5.0))
        finally:
            binding.set_wait_limit()
        assert torch.isnan(got[:17]).all() and (got[17:] == 5).all()
        assert pool.cache.error() == binding.EDGE0_ETIMEOUT
        assert torch.equal(call(pool, q, table, lens, cu, mask, out=torch.full_like(q, 5.0)), clean) and pool.cache.error() == binding.EDGE0_OK


@pytest.mark.parametrize("bits,D", [(4, 64), (4, 128), (4, 256), (8, 64), (8, 128), (8, 256)])
@pytest.mark.parametrize("lens,counts", [([300, 5, -1], [10, 7, 3]), ([9000, 70, 0], [10, 30, 3]), ([40, 500, 900], [40, 5, 1])])
def test_waits_that_run_out_on_the_way(bits, D, lens, counts):
    """Limits shorter than the call: rows that lack something are NaN and reported, the others as they should be, and so is the next call."""
    c = case(bits, D, 2, 4, 64, lens, counts)
    pool, q = c[:2]
    run = lambda: call(*c, out=torch.full_like(q, 5.0))
    clean = run()
    assert pool.cache.error() == binding.EDGE0_OK
    for limit in (1, 500, 1000, 2000, 4000, 8000, 16000) * 3:
        binding.set_wait_limit(limit)
        try:
            got = run()
        finally:
            binding.set_wait_limit()
        lost = torch.isnan(got).all(2)
        assert torch.equal(got[~lost], clean[~lost]), limit
        error = pool.cache.error()          # (a wait may run out that no row lacks anything for)
        assert error == binding.EDGE0_ETIMEOUT if lost.any() else error in (binding.EDGE0_OK, binding.EDGE0_ETIMEOUT), limit
        assert torch.equal(run(), clean) and pool.cache.error() == binding.EDGE0_OK, limit


@pytest.mark.parametrize("bits,D", [(4, 128), (8, 256), (4, 64)])
@pytest.mark.parametrize("chain", [False, True])
def test_blocks_of_few_and_of_many_rows_in_turn(bits, D, chain):
    """Blocks of up to 64 rows and of more alternate within a share, next to sequences without rows, without a context,
    with all rows in one tile."""
    rng = np.random.default_rng(5)
    counts = [int(c) for c in rng.choice([0, 1, 15, 16, 17, 32, 33, 40, 64], 90)]
    lens = [int(n) for n in rng.choice([0, 3, 60, 64, 250, 700, 1500], 90)]
    args = case(bits, D, 4, 4, 16, lens, counts, chain=chain)
    check(call(*args), *args)


@pytest.mark.parametrize("bits,D", [(4, 128), (8, 256)])
def test_threads_and_streams(bits, D):
    cases = [case(bits, D, 2, 4, 32, [200 + 900 * i, 4000, 30], [5, 20 + i, 33], seed=i) for i in range(4)]
    ready = [(c[0].cache, c[1], i32(c[2]), i32(c[3]), i32(c[4]), i32(c[5])) for c in cases]
    want = [binding.attn_tree(*r) for r in ready]
    torch.cuda.synchronize()
    got = [[] for _ in ready]

    def work(i):
        s = torch.cuda.Stream()
        for j in range(12):
            got[i].append(binding.attn_tree(*ready[i], stream=s if j % 2 else None))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        assert all(torch.equal(x, want[i]) for x in got[i])
    check(want[0], *cases[0])


def test_refusals():
    pool, q, table, lens, cu, mask = case(4, 128, 2, 4, 16, [30, 20], [5, 6])
    t, n, c, m = i32(table), i32(lens), i32(cu), i32(mask)
    f = lambda **kw: binding.attn_tree(pool.cache, **{**dict(q=q, table=t, lens=n, cu_rows=c, mask=m), **kw})
    for kw in (dict(q=q[:, :, :64]), dict(q=q[:, :7]), dict(q=q.float()), dict(table=t[0]), dict(table=t.long()), dict(lens=n[:1]),
               dict(cu_rows=c[:2]), dict(mask=m[:5]), dict(mask=m.long()), dict(mask=m[:, :0]), dict(mask=m[:, 0]), dict(scale=-1.0),
               dict(scale=float("inf")), dict(out=q[:3]), dict(out=q[:1].expand(11, 8, 128)),
               dict(workspace=torch.empty(64, dtype=torch.uint8, device=DEV)), dict(lens=n.cpu())):
        with pytest.raises(binding.Edge0Error) as e:
            f(**kw)
        assert e.value.code == binding.EDGE0_EINVAL, kw.keys()
    with pytest.raises(binding.Edge0Error) as e:
        f(q=rows(11, 130, 128))
    assert e.value.code == binding.EDGE0_EUNSUPPORTED
    assert f(q=q[:0], mask=m[:0]).shape == (0, 8, 128)


def over_cache(q, k, v, seen):
    """What attention over a cache gives that kv_read returns k and v of, in 64 bits, and how far a result may be off:
    attend's bound, with the parts of a group's values at most three times the largest of them (|s z + b| is the middle
    of a range that the values span), and what is not known of the cache: K and V as read are off by half an fp16 step,
    2^-11 of themselves and 2^-25.  Scores are off by d at most then, normalised weights by a factor of e^(2 d)."""
    q, k, v = q.double(), k.double(), v.double()
    scale = q.shape[2] ** -0.5
    most = lambda x: 3 * x.abs().unflatten(2, (-1, 64)).amax(3).repeat_interleave(64, 2)
    o, bound = flash_ref.attend(q, k, v, seen, scale, most(k), most(v), 2 * v.abs())
    wide = lambda x: x.repeat_interleave(q.shape[1] // k.shape[1], 1)
    # (p |v| as attention over |v|)
    pv = flash_ref.attend(q, k, v.abs(), seen, scale)[0]
    d = scale * torch.einsum("nhd,mhd->hnm", q.abs(), wide(2.0 ** -11 * k.abs() + 2.0 ** -25)).amax(2).T[:, :, None]
    f = torch.exp(2 * d)
    return o, bound + (f - 1) * pv + f * (2.0 ** -11 * pv + 2.0 ** -25)


@pytest.mark.parametrize("bits,D", [(4, 128), (8, 64), (8, 256)])
def test_a_prompt_and_drafted_tokens_through_the_block(bits, D):
    """As a program runs them: positions, the prompt's attention and cache, a tree drafted behind it, the accepted
    path drawn together, the next token, and a continuation on copied pages."""
    H, G, page, W, B = 2, 4, 16, 30, 3
    cache = binding.KVCache(2 * B * W, page, H, D, bits, device=DEV)
    plan = binding.RopePlan(D, base=500000.0, device=DEV)
    table = i32(np.random.default_rng(0).permutation(2 * B * W)[:B * W].reshape(B, W))
    counts, drafts = [200, 1, 333], [9, 12, 5]
    cu, cd = i32(np.concatenate([[0], np.cumsum(counts)])), i32(np.concatenate([[0], np.cumsum(drafts)]))
    zero, lens = i32([0] * B), i32(counts)
    T, N = sum(counts), sum(drafts)
    q, k, v = rows(T, H * G, D), rows(T, H, D), rows(T, H, D)
    q, k = binding.rope(plan, q, k, zero, cu)
    o = binding.attn_prompt(q, k, v, cu)
    binding.kv_append(cache, k, v, table, zero, cu)
    # the prompt's rows over the cache, and over what is read back of it
    kr, vr = binding.kv_read(cache, table, zero, cu, T)
    o_read, o_tree = binding.attn_prompt(q, kr, vr, cu), binding.attn_tree(cache, q, table, zero, cu)
    for b in range(B):
        r = slice(sum(counts[:b]), sum(counts[:b + 1]))
        seen = flash_ref.causal(counts[b], counts[b], DEV)
        for got, (want, bound) in ((o_read, flash_ref.attend(q[r].double(), kr[r].double(), vr[r].double(), seen, D ** -0.5)),
                                   (o_tree, over_cache(q[r], kr[r], vr[r], seen))):
            assert flash_ref.close(got[r], want, bound)
    # a tree: positions go by depth, places by row
    mask = tree_words(drafts, 1, np.random.default_rng(3))
    depth = np.array([bin(m).count("1") - 1 for m in mask[:, 0]]) + np.repeat(counts, drafts)
    qd, kd, vd = rows(N, H * G, D), rows(N, H, D), rows(N, H, D)
    qd, kd = binding.rope(plan, qd, kd, i32(depth))
    binding.kv_append(cache, kd, vd, table, lens, cd)
    od = binding.attn_tree(cache, qd, table, lens, cd, i32(mask))
    # the path to each sequence's last drafted token is accepted
    paths = [[j for j in range(x) if int(mask[sum(drafts[:b]) + x - 1, 0]) >> j & 1] for b, x in enumerate(drafts)]
    src = [counts[b] + j for b in range(B) for j in paths[b]]
    ca = i32(np.concatenate([[0], np.cumsum([len(p) for p in paths])]))
    binding.kv_compact(cache, table, lens, i32(src), ca)
    longer = i32([c + len(p) for c, p in zip(counts, paths)])
    # the last accepted token's row, decoded over what was kept, is the tree's row
    last = torch.tensor([sum(drafts[:b + 1]) - 1 for b in range(B)], device=DEV)
    dec = binding.attn_decode(cache, qd[last].contiguous(), table, longer)
    for b in range(B):
        n = int(longer[b])
        kr, vr = binding.kv_read(cache, table[b:b + 1], zero[:1], i32([0, n]), n)
        want, bound = over_cache(qd[last[b:b + 1]], kr, vr, torch.ones(1, n, dtype=torch.bool, device=DEV))
        assert flash_ref.close(dec[b:b + 1], want, bound) and flash_ref.close(od[last[b:b + 1]], want, bound)
    # a continuation on pages of its own
    used = torch.arange(W, device=DEV)[None, :] * page < longer[:, None]
    other = i32(np.random.default_rng(0).permutation(2 * B * W)[B * W:].reshape(B, W))
    binding.kv_copy_pages(cache, torch.where(used, table, -1), torch.where(used, other, -1))
    binding.kv_append(cache, kd[:B], vd[:B], table, longer)
    assert torch.equal(binding.attn_decode(cache, qd[last].contiguous(), other, longer), dec)
    assert o.isfinite().all() and cache.error() == binding.EDGE0_OK
