"""Projection, KV-cache and attention calls on the GPU against their plain 64-bit
forms (block_ref), at the sizes, masks and layouts where they can go wrong."""
import math
import threading

import numpy as np
import pytest
import torch

import block_ref as ref
from int4_routed_expert_prerouter_gb300 import binding, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else torch.tensor(a)
    return (t if dtype is None else t.to(dtype)).to(DEV)


def i32(a):
    return dev(np.asarray(a, np.int32))


# ------------------------------------------------------------ projection ----
def q4_bound(W_parts, x, y, n_in):
    """Half an fp16 step of the result (2^-24 where subnormal) plus fp32 sums: at most
    n_in / 16 matrix steps, n_in / 64 group sums and 16 joins, 2^-23 each, of terms that add up
    to |s q| |x| + |b| |x|."""
    mag = np.abs(x) @ W_parts.T
    return 2.0 ** -11 * np.abs(y) + 2.0 ** -24 + (n_in / 16 + n_in / 64 + 16) * 2.0 ** -23 * mag


def q4_case(n_out, n_in, seed=0):
    q, s, b = inputs.int4_stack(seed, 0, 1, 1, n_out, n_in)
    qn, sn, bn = q[0].numpy(), s[0].numpy(), b[0].numpy()
    zero = np.zeros_like(bn)
    parts = ref.dequant_q4(qn, np.abs(sn), zero) + np.repeat(np.abs(bn.astype(np.float64)), 64, -1)
    return tuple(t.to(DEV) for t in (q, s, b)), ref.dequant_q4(qn, sn, bn), parts


@pytest.mark.parametrize("B,n_in,n_out", [(1, 64, 1), (1, 128, 17), (1, 2048, 512), (2, 192, 16), (3, 1536, 100), (7, 320, 33),
                                          (8, 2048, 48), (9, 512, 47), (16, 640, 257), (17, 1536, 64), (33, 256, 130),
                                          (64, 1536, 96), (100, 448, 65), (255, 128, 31), (256, 2048, 144), (1, 16448, 19),
                                          (5, 8192, 40), (40, 4160, 129), (1, 131072, 5), (16, 65536, 3)])
def test_q4_linear(B, n_in, n_out):
    trip, W, parts = q4_case(n_out, n_in, seed=B)
    rng = np.random.default_rng(B + n_in)
    x = rng.standard_normal((B, n_in)).astype(np.float16)
    y = binding.q4_linear(binding.pack_q4_rows(trip), n_out, dev(x))
    want = x.astype(np.float64) @ W.T
    err = np.abs(y.cpu().numpy().astype(np.float64) - want)
    assert (err <= q4_bound(parts, x.astype(np.float64), want, n_in)).all(), err.max()


@pytest.mark.parametrize("B", [1, 5, 12, 70])
def test_q4_linear_slices_leave_the_rest(B):
    n_in, n_out = 512, 90
    trip, W, parts = q4_case(n_out, n_in)
    wide = torch.randn(B, n_in + 72, device=DEV).half()
    x = wide[:, 64:64 + n_in]
    out = torch.full((B, n_out + 11), 7.0, dtype=torch.float16, device=DEV)
    y = binding.q4_linear(binding.pack_q4_rows(trip), n_out, x, y=out[:, 3:3 + n_out])
    xn = x.cpu().numpy().astype(np.float64)
    want = xn @ W.T
    assert (np.abs(y.cpu().numpy() - want) <= q4_bound(parts, xn, want, n_in)).all()
    assert (out[:, :3] == 7).all() and (out[:, 3 + n_out:] == 7).all()


def test_q4_linear_special_values():
    n_in, n_out = 256, 32
    trip, W, _ = q4_case(n_out, n_in)
    packed = binding.pack_q4_rows(trip)
    x = torch.randn(9, n_in, device=DEV).half()
    clean = binding.q4_linear(packed, n_out, x)
    x[4, 100] = float("nan")
    got = binding.q4_linear(packed, n_out, x)
    rows = [i for i in range(9) if i != 4]
    assert torch.isnan(got[4]).all() and torch.equal(got[rows], clean[rows])     # one token's NaN stays its own
    assert not binding.q4_linear(packed, n_out, torch.zeros_like(x)).any()
    # results above fp16's range become infinities, as the rounding of the exact sum does
    trip = (torch.full((1, 16, 8), -1, dtype=torch.int32, device=DEV), torch.full((1, 16, 1), 100.0, dtype=torch.float16, device=DEV),
            torch.zeros(1, 16, 1, dtype=torch.float16, device=DEV))
    y = binding.q4_linear(binding.pack_q4_rows(trip), 16, torch.full((1, 64), 1.0, dtype=torch.float16, device=DEV))
    assert torch.isinf(y).all()


def test_q4_linear_agrees_with_the_shared_expert_layout_and_lora():
    # y = W x + (alpha / r) B A x, the pages' projection, from the two calls a program makes
    n_in, n_out, r, B = 256, 80, 4, 6
    trip, W, parts = q4_case(n_out, n_in)
    A = (torch.randn(r, n_in, device=DEV) * 0.05).half()
    Bm = (torch.randn(n_out, r, device=DEV) * 0.05).half()
    x = torch.randn(B, n_in, device=DEV).half()
    y = binding.q4_linear(binding.pack_q4_rows(trip), n_out, x)
    At = A.t().contiguous()
    d = binding.LoraDesc(r, n_in, n_out, 8.0, binding._ptr(binding.pack_f16(A)), binding._ptr(At), binding._ptr(Bm))
    binding.lora_delta(d, x, y)
    xn = x.cpu().numpy().astype(np.float64)
    delta = 2.0 * (xn @ A.cpu().numpy().astype(np.float64).T) @ Bm.cpu().numpy().astype(np.float64).T
    want = xn @ W.T + delta
    # two fp16 roundings: of W x, and of the sum
    bound = q4_bound(parts, xn, want - delta, n_in) + 2.0 ** -11 * np.abs(want) + 1e-5
    assert (np.abs(y.cpu().numpy() - want) <= bound * 1.01).all()


# ----------------------------------------------------------------- cache ----
KV_SHAPES = [(4, 64, 1, 16), (4, 128, 2, 48), (4, 256, 3, 16), (8, 64, 5, 32), (8, 128, 1, 64), (8, 256, 2, 16)]


def adversarial(rng, T, H, D):
    """Rows with ties, constants, tiny and huge ranges, zeros and denormals among them."""
    x = rng.standard_normal((T, H, D)).astype(np.float16)
    flat = x.reshape(-1, 64)
    n = flat.shape[0]
    for i in range(n):
        kind = i % 9
        if kind == 1:
            flat[i] = np.float16(rng.standard_normal())
        elif kind == 2:
            flat[i] = (rng.integers(0, 31, 64) * 0.5).astype(np.float16)          # half steps: ties
            flat[i, :2] = 0, 15
        elif kind == 3:
            flat[i] = (rng.integers(-2, 3, 64) * 2.0 ** -24).astype(np.float16)   # subnormal steps
        elif kind == 4:
            flat[i] = (rng.standard_normal(64) * 2.0 ** -20).astype(np.float16)
        elif kind == 5:
            flat[i] = (rng.uniform(-1, 1, 64) * 65504).astype(np.float16)
        elif kind == 6:
            flat[i] = (rng.integers(0, 511, 64) * 0.25 - 60).astype(np.float16)
            flat[i, :2] = -60, -60 + 127.5
        elif kind == 7:
            flat[i] = (1000 + rng.standard_normal(64)).astype(np.float16)
        elif kind == 8:
            flat[i] = np.clip(rng.standard_normal(64) * np.exp(4 * rng.standard_normal(64)), -6e4, 6e4).astype(np.float16)
    return x


@pytest.mark.parametrize("bits,D,H,page", KV_SHAPES)
def test_kv_append_writes_the_defined_bytes(bits, D, H, page):
    rng = np.random.default_rng(bits * D + H)
    counts, start = [0, 1, page + 3, 5, 33], [4, page - 1, 7, -1, 0]
    cu = np.concatenate([[0], np.cumsum(counts)])
    T = int(cu[-1]) + 2                                   # two rows behind the last sequence
    W, n_pages = 4, 24
    table = rng.permutation(n_pages)[:20].reshape(5, W)
    k, v = adversarial(rng, T, H, D), adversarial(rng, T, H, D)
    before = rng.integers(0, 256, (n_pages, binding.lib().edge0_kv_page_bytes(bits, H, D, page)), dtype=np.uint8)
    cache = binding.KVCache(n_pages, page, H, D, bits, pages=dev(before))
    binding.kv_append(cache, dev(k), dev(v), i32(table), i32(start), i32(cu))
    # the same through the definition: codes of every slot that a row names
    want = before.copy()
    img = {}
    for b in range(5):
        for i in range(counts[b]):
            pos = start[b] + i
            if start[b] >= 0:
                img[(table[b, pos // page], pos % page)] = int(cu[b]) + i
    for (pg, tok), r in img.items():
        both = np.stack([k[r], v[r]])[None, :, None]      # [1, 2, 1 token, H, D]
        q, s, bb = ref.quantise(both, bits)
        full = lambda a: np.repeat(a, page, 2)
        one = ref.page_image(full(q), full(s), full(bb), bits)
        mask = np.zeros_like(q)
        mask = ref.page_image(np.zeros((1, 2, page, H, D), np.uint8), np.zeros((1, 2, page, H, D // 64), np.float16),
                              np.zeros((1, 2, page, H, D // 64), np.float16), 8 if bits == 8 else 4)
        codes1 = np.zeros((1, 2, page, H, D), np.uint8)
        codes1[:, :, tok] = 15 if bits == 4 else 255
        ones = np.zeros((1, 2, page, H, D // 64), np.float16)
        ones[:, :, tok] = np.frombuffer(b"\xff\xff", np.float16)[0]
        mask = ref.page_image(codes1, ones, ones, bits)[0] == 255
        want[pg][mask] = one[0][mask]
    got = cache.pages.cpu().numpy()
    assert np.array_equal(got, want)
    assert cache.error() == binding.EDGE0_OK


@pytest.mark.parametrize("bits,D,H,page", KV_SHAPES)
def test_kv_read_returns_the_values(bits, D, H, page):
    rng = np.random.default_rng(D + H)
    c = ref.Cache(12, page, H, D, bits, rng)
    cache = binding.KVCache(12, page, H, D, bits, pages=dev(c.image))
    counts, start = [1, 0, 2 * page, 17], [page - 1, 0, 3, -5]
    cu = np.concatenate([[0], np.cumsum(counts)])
    T = int(cu[-1]) + 3
    table = rng.permutation(12).reshape(4, 3)
    k0 = torch.full((T, H, D), 5.0, dtype=torch.float16, device=DEV)
    k, v = binding.kv_read(cache, i32(table), i32(start), i32(cu), T, k=k0, v=k0.clone())
    exact = ref.values(c.codes, c.s, c.b).astype(np.float16)              # one rounding of s q + b
    for which, got in enumerate((k.cpu().numpy(), v.cpu().numpy())):
        want = np.full((T, H, D), 5.0, np.float16)
        for b in range(4):
            for i in range(counts[b]):
                pos = start[b] + i
                if start[b] >= 0:
                    want[cu[b] + i] = exact[table[b, pos // page], which, pos % page]
        assert np.array_equal(got, want)


def test_kv_round_trip_error_and_poisoned_groups():
    rng = np.random.default_rng(3)
    H, D, page, T = 2, 128, 16, 40
    k = (rng.standard_normal((T, H, D)) * 3).astype(np.float16)
    v = k[::-1].copy()
    v[5, 1, 70], v[6, 0, 3] = np.nan, -np.inf
    for bits in (4, 8):
        cache = binding.KVCache(3, page, H, D, bits, device=DEV)
        table, start, cu = i32([[2, 0, 1]]), i32([0]), i32([0, T])
        binding.kv_append(cache, dev(k), dev(v), table, start, cu)
        gk, gv = (t.cpu().numpy().astype(np.float64) for t in binding.kv_read(cache, table, start, cu, T))
        g = k.astype(np.float64).reshape(T, H, 2, 64)
        # half a step, the clamp's at most 2^-11 of the range, and the result's rounding
        step = (g.max(-1) - g.min(-1)) / (2 ** bits - 1)
        lim = step * 0.5 * (1 + 2.0 ** -10) + (g.max(-1) - g.min(-1)) * 2.0 ** -11
        lim = lim[..., None] + 2.0 ** -11 * np.abs(gk).reshape(g.shape)
        assert (np.abs(gk.reshape(g.shape) - g) <= lim).all()
        bad = np.isnan(gv.reshape(T, H, 2, 64))
        want = np.zeros_like(bad)
        want[5, 1, 1] = want[6, 0, 0] = True
        assert np.array_equal(bad, want)


def test_kv_widest_ranges_stay_finite():
    H, D, page, T = 1, 64, 16, 64
    rng = np.random.default_rng(8)
    x = (rng.uniform(-1, 1, (T, H, D)) * 65504).astype(np.float16)
    x[:, :, 0], x[:, :, 1] = -65504, 65504
    x[1::2] = np.abs(x[1::2])
    for bits in (4, 8):
        cache = binding.KVCache(4, page, H, D, bits, device=DEV)
        table, start, cu = i32([[0, 1, 2, 3]]), i32([0]), i32([0, T])
        binding.kv_append(cache, dev(x), dev(x), table, start, cu)
        k, v = binding.kv_read(cache, table, start, cu, T)
        q, s, b = ref.quantise(x, bits)
        want = ref.values(q, s, b).astype(np.float16)
        assert torch.isfinite(k).all() and np.array_equal(k.cpu().numpy(), want) and torch.equal(k, v)


def test_kv_and_attention_calls_without_rows():
    cache = binding.KVCache(2, 16, 1, 64, 4, device=DEV)
    none = torch.empty(0, 1, 64, dtype=torch.float16, device=DEV)
    binding.kv_append(cache, none, none, i32([[0]]), i32([0]), i32([0, 0]))
    k, v = binding.kv_read(cache, i32([[0]]), i32([0]), i32([0, 0]), 0)
    assert k.shape == v.shape == (0, 1, 64) and not cache.pages.any()
    o = binding.attn_decode(cache, torch.empty(0, 2, 64, dtype=torch.float16, device=DEV), i32(np.zeros((0, 1))), i32(np.zeros(0)))
    assert o.shape == (0, 2, 64)
    y = binding.q4_linear(torch.zeros(576, dtype=torch.uint8, device=DEV), 16, torch.empty(0, 64, dtype=torch.float16, device=DEV))
    assert y.shape == (0, 16)
    assert cache.error() == 0


def test_kv_slices_of_a_fused_projection_and_one_row_per_sequence():
    H, D, page, B = 2, 64, 32, 6
    wide = torch.randn(B, 4 * H * D + 8, device=DEV).half()
    k, v = wide[:, 2 * H * D:3 * H * D].unflatten(1, (H, D)), wide[:, 3 * H * D:4 * H * D].unflatten(1, (H, D))
    cache, twin = (binding.KVCache(B, page, H, D, 8, device=DEV) for _ in range(2))
    table, start = i32(np.arange(B)[:, None]), i32([0, 31, 5, -1, 16, 15])
    binding.kv_append(cache, k, v, table, start)
    binding.kv_append(twin, k.contiguous(), v.contiguous(), table, start, i32(np.arange(B + 1)))
    assert torch.equal(cache.pages, twin.pages) and cache.pages.any()
    ks, _ = binding.kv_read(cache, table, start, k=torch.zeros_like(k).contiguous(), v=torch.zeros(B, H, D, device=DEV).half())
    assert not ks[3].any() and ks[0].any()


def test_kv_bad_pages_and_positions_are_recorded_and_left_alone():
    H, D, page = 1, 64, 16
    for table, start in (([[0, 9]], [10]), ([[0, -1]], [10]), ([[0, 1]], [30]), ([[7, 1]], [0])):
        cache = binding.KVCache(7, page, H, D, 4, device=DEV)
        k = torch.randn(8, H, D, device=DEV).half()
        binding.kv_append(cache, k, k, i32(table), i32(start), i32([0, 8]))
        assert cache.error() == binding.EDGE0_EINVAL and cache.error() == binding.EDGE0_OK
        got = torch.full((8, H, D), 3.0, dtype=torch.float16, device=DEV)
        binding.kv_read(cache, i32(table), i32(start), i32([0, 8]), 8, k=got, v=got.clone())
        assert cache.error() == binding.EDGE0_EINVAL
        n_ok = {(0, 9): 6, (0, -1): 6, (0, 1): 2, (7, 1): 0}[tuple(table[0])]
        assert (got[n_ok:] == 3).all() and not (got[:n_ok] == 3).all() if n_ok else (got == 3).all()
        assert not cache.pages[2:].any()


def test_kv_offsets_beyond_32_bits():
    H, D, page, bits = 8, 256, 64, 8
    per = binding.lib().edge0_kv_page_bytes(bits, H, D, page)
    n = (1 << 32) // per + 40
    pages = torch.empty(n, per, dtype=torch.uint8, device=DEV)
    pages[-1].zero_(), pages[0].zero_()
    cache = binding.KVCache(n, page, H, D, bits, pages=pages)
    k, v = torch.randn(2, 70, H, D, device=DEV).half()
    table, start, cu = i32([[n - 1, n - 2]]), i32([0]), i32([0, 70])
    binding.kv_append(cache, k, v, table, start, cu)
    gk, gv = binding.kv_read(cache, table, start, cu, 70)
    small = binding.KVCache(2, page, H, D, bits, device=DEV)
    binding.kv_append(small, k, v, i32([[1, 0]]), start, cu)
    sk, sv = binding.kv_read(small, i32([[1, 0]]), start, cu, 70)
    assert torch.equal(gk, sk) and torch.equal(gv, sv) and not pages[0].any()
    q = torch.randn(1, 16, D, device=DEV).half()
    o = binding.attn_decode(cache, q, table, i32([70]))
    assert torch.equal(o, binding.attn_decode(small, q, i32([[1, 0]]), i32([70])))
    assert torch.equal(binding.attn_decode(cache, q, table, i32([0]), i32([n - 1, n - 2]), 70),
                       binding.attn_decode(small, q, i32([[1, 0]]), i32([0]), i32([1, 0]), 70))


# ------------------------------------------------------------- attention ----
def run_attention(bits, D, H, G, page, lens, P, seed=0, k_offset=0.0, v_scale=1.0, scale=None, junk=True, pad=()):
    """Runs one call on a shuffled pool and checks every row; returns what a twin needs."""
    rng = np.random.default_rng(seed + bits * D + H + G)
    B = len(lens)
    W = max(1, max(-(-n // page) for n in lens)) + 1
    n_pre = -(-P // page)
    need = [-(-max(n, 0) // page) for n in lens]
    n_pages = sum(need) + n_pre + 2
    c = ref.Cache(n_pages, page, H, D, bits, rng, k_offset, v_scale)
    order = rng.permutation(n_pages)
    table = np.full((B, W), -1, np.int32)
    image = c.image.copy()
    at = 0

    def fill(pages, n):
        # bytes of tokens that are not there: NaN scales, any codes
        if junk and n % page and len(pages):
            whole = image[pages[-1]].reshape(H, page // 16, -1)
            mask = ref.page_image(*[np.concatenate([np.zeros((1, 2, n % page, H, d)), np.ones((1, 2, page - n % page, H, d)) * f], 2).astype(t)
                                    for d, f, t in ((D, 255 if bits == 8 else 15, np.uint8), (D // 64, np.nan, np.float16),
                                                    (D // 64, np.nan, np.float16))], bits).reshape(whole.shape)
            whole[mask != 0] = 255
            image[pages[-1]] = whole.reshape(-1)

    lists = []
    for b in range(B):
        mine = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = mine
        fill(mine, max(lens[b], 0))
        lists.append(mine)
    pre = order[at:at + n_pre]
    fill(pre, P)
    cache = binding.KVCache(n_pages, page, H, D, bits, pages=dev(image))
    wide = rng.standard_normal((B, H * G * D + 16)).astype(np.float16)
    q = dev(wide)[:, 8:8 + H * G * D].unflatten(1, (H * G, D))
    real = list(lens)
    for b in pad:
        real[b] = -1 - b
    out = torch.full((B, H * G + 1, D), 9.0, dtype=torch.float16, device=DEV)
    args = (cache, q, i32(table), i32(real), i32(pre) if P else None, P, scale)
    got = binding.attn_decode(*args, out=out[:, :H * G])
    assert cache.error() == binding.EDGE0_OK
    sc = D ** -0.5 if scale is None else scale
    kp, vp, pp, zp = c.tokens(pre, P)
    g = got.cpu().numpy().astype(np.float64)
    for b in range(B):
        if b in pad:
            assert (g[b] == 9).all()
            continue
        own = c.tokens(lists[b], lens[b]) if lens[b] else (kp[:0],) * 4
        k, v, parts, sz = (np.concatenate(x) for x in zip((kp, vp, pp, zp), own))
        want, bound = ref.attention(wide[b, 8:8 + H * G * D].astype(np.float64).reshape(H * G, D), k, v, parts, sz, sc)
        err = np.abs(g[b] - want)
        assert (err <= bound).all(), (b, lens[b], (err / bound).max())
    assert (out[:, H * G:] == 9).all()
    return args, got


LENS = [1, 0, 15, 16, 17, 31, 32, 33, 64, 100, 257, 2]


@pytest.mark.parametrize("bits,D", [(4, 64), (4, 128), (4, 256), (8, 64), (8, 128), (8, 256)])
@pytest.mark.parametrize("H,G,page,P", [(1, 1, 16, 0), (2, 4, 64, 47), (2, 3, 48, 0), (1, 8, 32, 333), (2, 5, 16, 1), (1, 16, 64, 64),
                                        (1, 20, 32, 100), (3, 2, 112, 16)])
def test_attention(bits, D, H, G, page, P):
    run_attention(bits, D, H, G, page, LENS, P)


@pytest.mark.parametrize("lens,P", [([1], 0), ([0], 1), ([0, 0, 0], 17), ([5], 0), ([3000], 0), ([1999], 1001), ([0, 2500, 1], 0),
                                    ([1] * 70, 300), ([40] * 33, 0), (list(range(0, 256)), 65)])
@pytest.mark.parametrize("bits", [4, 8])
def test_attention_lengths(bits, lens, P):
    run_attention(bits, 128, 2, 4, 64, lens, P, seed=len(lens))


@pytest.mark.parametrize("bits,D,P", [(4, 128, 0), (8, 64, 40), (8, 256, 0), (4, 256, 130)])
def test_attention_one_long_sequence_in_a_large_batch(bits, D, P):
    # its parts are many, the other sequences' rows have none, one or two
    lens = [int(n) for n in np.random.default_rng(D).integers(0, 40, 129)]
    lens[77], lens[5] = 16001, 700
    run_attention(bits, D, 1, 8, 64, lens, P, seed=3, pad=(0, 128))


def test_attention_many_query_heads():
    run_attention(4, 64, 1, 64, 16, [33, 0, 7], 50)
    run_attention(8, 128, 2, 33, 32, [64, 1], 130)


def test_attention_empty_and_padding_rows():
    _, got = run_attention(4, 128, 2, 4, 32, [0, 5, 0, 40], 0, pad=(3,))
    assert not got[0].any() and not got[2].any()
    run_attention(8, 64, 2, 4, 32, [0, 5, 0, 40], 20, pad=(0, 1))
    run_attention(8, 64, 2, 4, 32, [7, 5], 0, pad=(0, 1))


@pytest.mark.parametrize("kw", [dict(k_offset=30.0), dict(v_scale=2.0 ** -12), dict(v_scale=3000.0), dict(scale=4.0), dict(scale=1e-6),
                                dict(scale=0.0883)])
@pytest.mark.parametrize("bits", [4, 8])
def test_attention_ranges(bits, kw):
    run_attention(bits, 128, 2, 8, 64, [0, 1, 40, 513], 200, **kw)


@pytest.mark.parametrize("bits,D,B", [(4, 128, 1), (8, 64, 2), (4, 64, 40), (8, 128, 9), (4, 256, 9)])
def test_attention_constant_groups(bits, D, B):
    """Constant groups (s = 0) of every kind among the tokens: zeros, one value, tiny and large."""
    rng = np.random.default_rng(B)
    H, G, page, n, P = 1, 4, 16, 75, 90
    x = rng.standard_normal((12, 2, page, H, D))
    for i, c in enumerate((0.0, -0.0, 1.5, -1.5, 2.0 ** -24, -3e-5, 9.0)):
        x[:, :, i::11, :, :64] = c
        x[i, :, :, :, D - 64:] = c
    codes, s, b = ref.quantise(x.astype(np.float16), bits)
    assert (s == 0).any()
    val = ref.values(codes, s, b)
    cache = binding.KVCache(12, page, H, D, bits, pages=dev(ref.page_image(codes, s, b, bits)))
    table = np.stack([rng.permutation(12)[:5] for _ in range(B)])
    pre = rng.permutation(12)[:6]
    q = rng.standard_normal((B, H * G, D)).astype(np.float16)
    got = binding.attn_decode(cache, dev(q), i32(table), i32([n] * B), i32(pre), P).cpu().numpy().astype(np.float64)
    z = 2.0 ** (bits - 1)
    sw, bw = (np.repeat(a[:, 1].astype(np.float64), 64, -1) for a in (s, b))
    flat = lambda a, pages, m: a[pages].reshape(-1, H, D)[:m]
    # a constant group's value b is |b| times (0 - z) + (z +- 1): its part that meets a code is z |b|
    parts = np.where(sw == 0, (2 * z + 1) * np.abs(bw), np.abs(sw * (codes[:, 1].astype(np.float64) - z)) + np.abs(sw * z + bw))
    big = np.where(sw == 0, np.abs(bw), sw) * z
    for i in range(B):
        k, v, pp, zz = (np.concatenate([flat(a, pre, P), flat(a, table[i], n)]) for a in (val[:, 0], val[:, 1], parts, big))
        want, bound = ref.attention(q[i].astype(np.float64), k, v, pp, zz, D ** -0.5)
        assert (np.abs(got[i] - want) <= bound).all()


def test_attention_captured_without_a_call_before():
    """A process whose first attention, cache and projection calls are inside a capture."""
    import subprocess
    import sys
    code = """
import torch
from int4_routed_expert_prerouter_gb300 import binding as b
dev = "cuda:0"
cache = b.KVCache(40, 16, 2, 128, 4, device=dev)
k = torch.randn(96, 2, 128, device=dev).half()
i = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)
table, start, cu = i([[*range(6)]]), i([0]), i([0, 96])
q = torch.randn(24, 8, 128, device=dev).half()
own, lens, pre = i([[6 + j % 30] for j in range(24)]), i([j % 17 for j in range(24)]), i([*range(6)])
w = torch.zeros(48 * 9 * 16, dtype=torch.uint8, device=dev)[:576 * 4].contiguous()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    b.kv_append(cache, k, k, table, start, cu)
    o = b.attn_decode(cache, q, own, lens, pre, 90)
    y = b.q4_linear(w, 16, q.view(48, 512)[:3, :256].contiguous())
g.replay()
torch.cuda.synchronize()
first = o.clone()
g.replay()
e = b.attn_decode(cache, q, own, lens, pre, 90)
torch.cuda.synchronize()
assert torch.equal(first, o) and torch.equal(e, o) and o.isfinite().all() and o.any() and cache.error() == 0
print("captured")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_attention_scores_that_grow_along_the_context():
    # the running maximum rises by far more than one step, late and in every part
    rng = np.random.default_rng(5)
    H, D, page, n, bits = 1, 128, 64, 1500, 8
    x = rng.standard_normal((24, 2, page, H, D)) * 0.5
    u = rng.standard_normal(D)
    ramp = np.arange(24 * page).reshape(24, page) / 40.0
    x[:, 0] += (ramp[..., None, None] * u / np.sqrt(D))
    codes, s, b = ref.quantise(x.astype(np.float16), bits)
    val = ref.values(codes, s, b)
    cache = binding.KVCache(24, page, H, D, bits, pages=dev(ref.page_image(codes, s, b, bits)))
    q = (np.stack([u, -u, 3 * u, 0 * u]) ).astype(np.float16)
    got = binding.attn_decode(cache, dev(q[None]), i32(np.arange(24)[None]), i32([n])).cpu().numpy()[0]
    z = 128.0
    sw, bw = (np.repeat(a[:, 1].astype(np.float64), 64, -1) for a in (s, b))
    flat = lambda a: a.reshape(-1, H, D)[:n]
    parts = np.abs(sw * (codes[:, 1].astype(np.float64) - z)) + np.abs(sw * z + bw)
    want, bound = ref.attention(q.astype(np.float64), flat(val[:, 0]), flat(val[:, 1]), flat(parts), flat(sw * z), D ** -0.5)
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("bits,D,B", [(4, 128, 1), (8, 64, 2), (4, 64, 20), (8, 128, 9), (4, 256, 9)])
def test_attention_scores_of_any_magnitude(bits, D, B):
    """Scores up to 10^16, each far from the next: the largest one's token alone, whose weight
    is exactly 1: the result's rounding, 2^-11 of it, and fp32 sums of its two parts.  The
    weight times s is exact in fp16 while that is normal; below, half a subnormal step of units
    of 2^-7 2^e, 2^e at most twice the largest s: 2^-25 2^-7 2 max(s), times |q - z| <= z."""
    rng = np.random.default_rng(D)
    H, G, page, n, P = 1, 4, 16, 150, 90
    for size, scale in ((1.0, 1e6), (200.0, 1e6), (200.0, 1.0)):
        x = rng.standard_normal((16, 2, page, H, D))
        x[:, 0] = rng.permutation(np.arange(1, 257)).reshape(16, page, 1, 1) * size * np.where(np.arange(D) % 2, 1.0, 0.5)
        x[:, 1] *= 2.0 ** rng.integers(-12, 12, (16, page, 1, 1))
        codes, s, b = ref.quantise(x.astype(np.float16), bits)
        val = ref.values(codes, s, b)
        cache = binding.KVCache(16, page, H, D, bits, pages=dev(ref.page_image(codes, s, b, bits)))
        table = np.stack([rng.permutation(10) for _ in range(B)])
        pre = np.arange(10, 16)
        u = np.where(np.arange(D) % 2, 1.0, 0.5) * size
        q = (np.stack([u, -u, u / 2, -u / 2])[None] * 2.0 ** -rng.integers(0, 3, (B, 1, 1))).astype(np.float16)
        got = binding.attn_decode(cache, dev(q), i32(table), i32([n] * B), i32(pre), P, scale).cpu().numpy().astype(np.float64)
        z = 2.0 ** (bits - 1)
        sw, bw = (np.repeat(a[:, 1].astype(np.float64), 64, -1) for a in (s, b))
        parts = np.abs(sw * (codes[:, 1].astype(np.float64) - z)) + np.abs(sw * z + bw)
        step = 2.0 ** -32 * 2 * s[:, 1].astype(np.float64).max() * z
        flat = lambda a, pages, m: a[pages].reshape(-1, D)[:m]
        for i in range(B):
            k, v, pp = (np.concatenate([flat(a, pre, P), flat(a, table[i], n)]) for a in (val[:, 0], val[:, 1], parts))
            sc = scale * q[i].astype(np.float64) @ k.T
            top = np.sort(sc, 1)
            assert (top[:, -1] - top[:, -2] > 100).all()
            at = sc.argmax(1)
            assert (np.abs(got[i] - v[at]) <= 2.0 ** -11 * np.abs(v[at]) + 2.0 ** -24 + 2.0 ** -20 * pp[at] + step).all()


@pytest.mark.parametrize("bits,D,B", [(4, 128, 1), (8, 64, 2), (4, 64, 20), (8, 128, 9), (4, 256, 9)])
def test_attention_one_token_of_large_values(bits, D, B):
    """Values that differ by a few fp16 steps (b far above s) beside a token whose values span the
    type's range and whose weight is next to nothing."""
    rng = np.random.default_rng(D + bits)
    H, G, page, n, P = 1, 4, 16, 75, 90
    x = rng.standard_normal((12, 2, page, H, D))
    u = rng.standard_normal(D)
    x[:, 1] = 1.0 + 2.0 ** -10 * rng.integers(0, 3, x[:, 1].shape)
    x[::2, 1, :, :, :64] *= -1000.0
    for page_no, tok in ((0, 3), (7, 9)):
        x[page_no, 0, tok] = -3.0 * u
        x[page_no, 1, tok] = rng.uniform(-1, 1, (H, D)) * 30000
        x[page_no, 1, tok, :, ::64] = 30000
    codes, s, b = ref.quantise(x.astype(np.float16), bits)
    val = ref.values(codes, s, b)
    cache = binding.KVCache(12, page, H, D, bits, pages=dev(ref.page_image(codes, s, b, bits)))
    q = np.stack([np.stack([u, 1.1 * u, 0.9 * u, u])] * B).astype(np.float16)
    z = 2.0 ** (bits - 1)
    sw, bw = (np.repeat(a[:, 1].astype(np.float64), 64, -1) for a in (s, b))
    flat_s = sw == 0
    parts = np.where(flat_s, (2 * z + 1) * np.abs(bw), np.abs(sw * (codes[:, 1].astype(np.float64) - z)) + np.abs(sw * z + bw))
    big = np.where(flat_s, np.abs(bw), sw) * z
    flat = lambda a, pages, m: a[pages].reshape(-1, H, D)[:m]
    for P in (0, 90):
        table = np.stack([rng.permutation(6) for _ in range(B)])
        pre = 6 + rng.permutation(6)
        got = binding.attn_decode(cache, dev(q), i32(table), i32([n] * B), i32(pre), P).cpu().numpy().astype(np.float64)
        for i in range(B):
            k, v, pp, zz = (np.concatenate([flat(a, pre, P), flat(a, table[i], n)]) for a in (val[:, 0], val[:, 1], parts, big))
            # near-constant groups: z s is far below |b|, so V's parts are V's own size
            want, bound = ref.attention(q[i].astype(np.float64), k, v, pp, zz, D ** -0.5)
            err = np.abs(got[i] - want)
            assert (err <= bound).all(), (P, i, (err / bound).max())


def test_attention_nan_reaches_only_its_own_rows():
    H, G, D, page = 2, 4, 128, 16
    args, clean = run_attention(4, D, H, G, page, [20, 33, 16], 10)
    cache, q, table, lens, pre, P, scale = args
    q = q.clone()
    q[1, 2, 5] = float("nan")
    got = binding.attn_decode(cache, q, table, lens, pre, P)
    same = torch.ones(3, H * G, dtype=torch.bool, device=DEV)
    same[1, 2] = False
    assert torch.isnan(got[1, 2]).all() and torch.equal(got[same], clean[same])
    # a poisoned group of one token's V, head 1: that group of that sequence's heads
    strip = cache.pages[table[2, 0].long()].view(H, -1)
    half = strip.shape[1] // 2
    strip[1, half + 16 * 64 + 3 * 8 + 4:half + 16 * 64 + 3 * 8 + 8] = 255
    got = binding.attn_decode(cache, args[1], table, lens, pre, P)
    nan = torch.isnan(got)
    want = torch.zeros_like(nan)
    want[2, G:, 64:] = True
    assert torch.equal(nan, want)
    assert torch.equal(got[~want], clean[~want])


def test_attention_bad_pages_and_lengths_are_recorded():
    H, D, page = 1, 64, 16
    cache = binding.KVCache(4, page, H, D, 4, device=DEV)
    q = torch.randn(2, 2, D, device=DEV).half()
    for table, lens, pre, P in (([[0, 4], [1, 2]], [20, 20], None, 0), ([[0, -7], [1, 2]], [20, 3], None, 0),
                                ([[0, 1], [1, 2]], [33, 3], None, 0), ([[0, 1], [1, 2]], [3, 3], [2, 9], 17)):
        o = binding.attn_decode(cache, q, i32(table), i32(lens), None if pre is None else i32(pre), P)
        assert torch.isfinite(o).all() and cache.error() == binding.EDGE0_EINVAL
    # entries that no token reaches are not looked at
    binding.attn_decode(cache, q, i32([[0, 99], [-5, 99]]), i32([16, 0]))
    assert cache.error() == binding.EDGE0_OK


def test_attention_repeats_bit_by_bit_and_needs_no_clean_workspace():
    args, a = run_attention(4, 128, 2, 4, 64, [700, 0, 33, 1200], 500)
    nb = binding.attn_workspace_bytes(args[0], 4, 8)
    for fill in (0, 255):
        ws = torch.full((nb,), fill, dtype=torch.uint8, device=DEV)
        for _ in range(3):
            assert torch.equal(binding.attn_decode(*args, workspace=ws), a)


# ------------------------------------------- streams, graphs, used together ----
def test_calls_on_another_stream():
    side = torch.cuda.Stream(DEV)
    args, a = run_attention(8, 128, 2, 4, 64, [300, 1], 90)
    trip, _, _ = q4_case(100, 256)
    packed = binding.pack_q4_rows(trip)
    x = torch.randn(3, 256, device=DEV).half()
    y = binding.q4_linear(packed, 100, x)
    side.wait_stream(torch.cuda.current_stream())
    b = binding.attn_decode(*args, stream=side)
    z = binding.q4_linear(packed, 100, x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b) and torch.equal(y, z)


def block_step(h, w, cache, table, lens, pre, P, H, G, D):
    """One token's attention half of a block: projections, cache, attention, output."""
    qkv = binding.q4_linear(w["qkv"], (H * G + 2 * H) * D, h)
    k = qkv[:, H * G * D:(H * G + H) * D].unflatten(1, (H, D))
    v = qkv[:, (H * G + H) * D:].unflatten(1, (H, D))
    binding.kv_append(cache, k, v, table, lens)
    lens += 1
    o = binding.attn_decode(cache, qkv[:, :H * G * D].unflatten(1, (H * G, D)), table, lens, pre, P)
    return h + binding.q4_linear(w["o"], h.shape[1], o.flatten(1))


@pytest.mark.parametrize("bits", [4, 8])
def test_decode_steps_of_a_block_eager_and_captured(bits):
    """Prompt written and read back, then decode steps of a batch behind it: against the plain
    forms step by step, and the captured step's replays against the eager ones."""
    H, G, D, page, d, B, P, steps = 2, 4, 64, 16, 256, 5, 37, 20
    rng = np.random.default_rng(bits)
    qkv, Wqkv, pqkv = q4_case((H * G + 2 * H) * D, d, seed=1)
    oo, Wo, po = q4_case(d, H * G * D, seed=2)
    w = dict(qkv=binding.pack_q4_rows(qkv), o=binding.pack_q4_rows(oo))
    n_pages = 4 * B + 3
    prompt = rng.standard_normal((P, d)).astype(np.float16)
    pre = i32([1, 0, 2])
    table = i32(3 + rng.permutation(4 * B).reshape(B, 4))
    hs = dev(rng.standard_normal((steps, B, d)).astype(np.float16))

    def fresh():
        cache = binding.KVCache(n_pages, page, H, D, bits, device=DEV)
        rows = binding.q4_linear(w["qkv"], (H * G + 2 * H) * D, dev(prompt))
        kv = rows[:, H * G * D:].unflatten(1, (2, H, D))
        binding.kv_append(cache, kv[:, 0], kv[:, 1], pre[None], i32([0]), i32([0, P]))
        return cache, i32(np.zeros(B))

    cache, lens = fresh()
    eager = [block_step(hs[t], w, cache, table, lens, pre, P, H, G, D).clone() for t in range(steps)]
    assert cache.error() == 0
    # step by step against the plain forms, fed with what the pages hold
    got_k, got_v = binding.kv_read(cache, table, i32(np.zeros(B)), i32(np.arange(B + 1) * steps), B * steps)
    # (the steps' own calls again: another number of rows adds its fp32 sums up in another order, and a sum
    # next to a border of fp16 may then round to the other side)
    rows = torch.stack([binding.q4_linear(w["qkv"], (H * G + 2 * H) * D, hs[t]) for t in range(steps)]).cpu().numpy()
    for t in (0, 1, steps - 1):
        want = hs[t].cpu().numpy().astype(np.float64) @ Wqkv.T
        b1 = q4_bound(pqkv, hs[t].cpu().numpy().astype(np.float64), want, d)
        assert (np.abs(rows[t] - want) <= b1).all()
    kk = rows[:, :, H * G * D:].reshape(steps, B, 2, H, D)
    q_, s_, b_ = ref.quantise(np.ascontiguousarray(kk), bits)
    v16 = ref.values(q_, s_, b_).astype(np.float16)
    assert np.array_equal(got_k.view(B, steps, H, D).cpu().numpy(), v16[:, :, 0].transpose(1, 0, 2, 3))
    assert np.array_equal(got_v.view(B, steps, H, D).cpu().numpy(), v16[:, :, 1].transpose(1, 0, 2, 3))
    # captured: one graph of the step replayed, lengths advancing on the device
    cache2, lens2 = fresh()
    h_in = hs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    pages0, lens0 = cache2.pages.clone(), lens2.clone()
    with torch.cuda.graph(graph):
        h_out = block_step(h_in, w, cache2, table, lens2, pre, P, H, G, D)
    cache2.pages.copy_(pages0)
    lens2.copy_(lens0)
    for t in range(steps):
        h_in.copy_(hs[t])
        graph.replay()
        assert torch.equal(h_out, eager[t]), t
    assert torch.equal(cache2.pages, cache.pages) and cache2.error() == 0


def test_two_captured_graphs_with_their_own_workspaces_overlap():
    a_args, a = run_attention(4, 128, 2, 4, 64, [600, 33], 300)
    b_args, b = run_attention(8, 64, 2, 4, 32, [90, 0, 500], 64)
    graphs, outs = [], []
    for args in (a_args, b_args):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(binding.attn_decode(*args))
        graphs.append(g)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        for s, g in zip((s1, s2), graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], a) and torch.equal(outs[1], b)


def test_kept_workspaces_are_not_shared_across_streams_and_graphs():
    """Calls without a workspace: eager ones on two streams and replays of a graph captured on one
    of them, all under way together, and one of another size in between."""
    a, _ = run_attention(4, 128, 2, 4, 64, [700, 0, 33, 1200], 500)
    b, _ = run_attention(8, 64, 2, 8, 32, [3000, 15, 900], 0, seed=4)
    args = (a[0],) + a[1:]
    want = binding.attn_decode(*args)
    q1 = a[1][:1].contiguous()
    small = binding.attn_decode(a[0], q1, a[2][:1].contiguous(), a[3][:1].contiguous(), a[4], a[5])
    other = binding.attn_decode(*b)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [[], [], []]
    with torch.cuda.stream(one):
        binding.attn_decode(*args)
    one.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=one):
        captured = binding.attn_decode(*args)
    for _ in range(20):
        with torch.cuda.stream(one):
            outs[0].append(binding.attn_decode(*args))
            outs[1].append(binding.attn_decode(a[0], q1, a[2][:1].contiguous(), a[3][:1].contiguous(), a[4], a[5]))
        with torch.cuda.stream(two):
            g.replay()
            outs[2].append(captured.clone())
            outs[0].append(binding.attn_decode(*args))
        assert torch.equal(binding.attn_decode(*b), other)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs[0] + outs[2])
    assert all(torch.equal(o, small) for o in outs[1])


def test_calls_of_several_threads_on_one_stream():
    # without workspaces of their own: the threads' launches share a stream and what the cache keeps for it
    cases = [run_attention(4, 128, 2, 4, 64, [700, 0, 33, 1200], 500), run_attention(4, 128, 2, 4, 64, [40] * 33, 30, seed=1)]
    shared = cases[0][0][0]
    (_, q1, t1, l1, p1, P1, s1), want1 = cases[0]
    q2 = q1[:2].contiguous() * 0.5
    want2 = binding.attn_decode(shared, q2, t1[:2].contiguous(), l1[:2].contiguous(), p1, P1, s1)
    torch.cuda.synchronize()
    outs = [[] for _ in range(6)]

    def work(i):
        for _ in range(60):
            if i % 2:
                outs[i].append(binding.attn_decode(shared, q2, t1[:2].contiguous(), l1[:2].contiguous(), p1, P1, s1))
            else:
                outs[i].append(binding.attn_decode(shared, q1, t1, l1, p1, P1, s1))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i, got in enumerate(outs):
        assert len(got) == 60 and all(torch.equal(o, want2 if i % 2 else want1) for o in got)


def test_calls_right_behind_their_producers_and_consumers():
    """Every kernel may begin before its predecessor has ended: chains in which each call reads what
    the one before wrote and overwrites what the one before read, eager and captured, with copies,
    fills, events from another stream and kernels of other kinds between them."""
    rng = np.random.default_rng(9)
    H, G, D, page, B = 2, 4, 128, 64, 40
    trip, _, _ = q4_case(2 * H * D, 512, seed=2)
    packed = binding.pack_q4_rows(trip)
    cache = binding.KVCache(B + 4, page, H, D, 4, device=DEV)
    table, pre = i32(np.arange(B)[:, None]), i32([B, B + 1, B + 2])
    old = torch.randn(192, H, D, device=DEV).half()
    binding.kv_append(cache, old, old, pre[None].contiguous(), i32([0]), i32([0, 192]))
    clean = cache.pages.clone()
    xs = [dev(rng.standard_normal((B, 512)).astype(np.float16)) for _ in range(6)]
    big = torch.zeros(1 << 22, device=DEV)
    other = torch.cuda.Stream()

    def buffers():
        return dict(x=torch.empty(B, 512, device=DEV).half(), kv=torch.empty(B, 2 * H * D, device=DEV).half(),
                    k=torch.empty(B, H, D, device=DEV).half(), v=torch.empty(B, H, D, device=DEV).half(),
                    o=torch.zeros(B, G * H, D, device=DEV).half(), pos=torch.zeros(B, dtype=torch.int32, device=DEV),
                    lens=torch.zeros(B, dtype=torch.int32, device=DEV),
                    ws=torch.empty(binding.attn_workspace_bytes(cache, B, G * H), dtype=torch.uint8, device=DEV))

    def chain(b, wait, n_prefix):
        got = []
        step = torch.cuda.current_stream().synchronize if wait else lambda: None
        cache.pages.copy_(clean)
        b["pos"].zero_()
        b["lens"].fill_(1)
        for x in xs:
            b["x"].copy_(x)
            step()
            binding.q4_linear(packed, 2 * H * D, b["x"], y=b["kv"])
            step()
            k, v = b["kv"][:, :H * D].unflatten(1, (H, D)), b["kv"][:, H * D:].unflatten(1, (H, D))
            binding.kv_append(cache, k, v, table, b["pos"])
            step()
            binding.kv_read(cache, table, b["pos"], k=b["k"], v=b["v"])
            step()
            q = torch.cat([b["k"], b["v"]] * 2, 1)
            step()
            binding.attn_decode(cache, q, table, b["lens"], pre, n_prefix, out=b["o"], workspace=b["ws"])
            step()
            ev = torch.cuda.Event()
            ev.record()
            with torch.cuda.stream(other):
                other.wait_event(ev)
                got.append(b["o"].clone())
                big.add_(1)
                back = torch.cuda.Event()
                back.record()
            torch.cuda.current_stream().wait_event(back)
            binding.attn_decode(cache, b["o"], table, b["lens"], pre, n_prefix, out=b["o"].new_empty(b["o"].shape), workspace=b["ws"])
            binding.q4_linear(packed, 2 * H * D, b["x"], y=b["kv"])       # overwritten while the last call may still run
            got.append(b["kv"].clone())
            b["pos"] += 1
            b["lens"] += 1
            step()
        return got

    for n_prefix in (0, 5, 190):
        b = buffers()
        want = [t.clone() for t in chain(b, True, n_prefix)]
        torch.cuda.synchronize()
        for _ in range(5):
            for a, w in zip(chain(b, False, n_prefix), want):
                torch.cuda.synchronize()
                assert torch.equal(a, w)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = chain(b, False, n_prefix)
        for _ in range(5):
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, w) for a, w in zip(outs, want))


def test_binding_refuses_what_does_not_fit():
    E = binding.Edge0Error
    cache = binding.KVCache(4, 16, 2, 64, 4, device=DEV)
    k = torch.zeros(3, 2, 64, dtype=torch.float16, device=DEV)
    table, start = i32([[0], [1], [2]]), i32([0, 0, 0])
    bad = [lambda: binding.kv_append(cache, k.float(), k, table, start), lambda: binding.kv_append(cache, k[:2], k, table, start),
           lambda: binding.kv_append(cache, k, k, table.long(), start), lambda: binding.kv_append(cache, k, k, table, start[:2]),
           lambda: binding.kv_append(cache, k.transpose(1, 2), k, table, start),
           lambda: binding.kv_append(cache, k[:, :1], k[:, :1], table, start),
           lambda: binding.kv_append(cache, k.cpu(), k, table, start),
           lambda: binding.kv_read(cache, table, start, None, 4),
           lambda: binding.kv_read(cache, table, start, i32([0, 1, 2])),
           lambda: binding.attn_decode(cache, k[:, :1], table, start),          # one query head for two K/V heads
           lambda: binding.attn_decode(cache, k, table, start, None, 3),
           lambda: binding.attn_decode(cache, k, table, start, i32([0]), 17),
           lambda: binding.attn_decode(cache, k, table[:2], start),
           lambda: binding.attn_decode(cache, k, table, start, scale=-1.0),
           lambda: binding.attn_decode(cache, k, table, start, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV)),
           lambda: binding.KVCache(4, 17, 2, 64, 4, device=DEV), lambda: binding.KVCache(4, 16, 2, 64, 6, device=DEV),
           lambda: binding.KVCache(4, 16, 2, 64, 4, pages=torch.zeros(5, dtype=torch.uint8, device=DEV)),
           lambda: binding.q4_linear(torch.zeros(100, dtype=torch.uint8, device=DEV), 16, k.view(3, 128)),
           lambda: binding.q4_linear(torch.zeros(1152, dtype=torch.uint8, device=DEV), 16, k.view(3, 128)[:, ::2])]
    for i, f in enumerate(bad):
        with pytest.raises(E):
            f()
            raise AssertionError(i)
