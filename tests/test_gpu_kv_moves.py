"""Rows and pages moved inside the cache, byte for byte against a plain walk over the rows."""
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


def i32(a):
    return torch.tensor(np.asarray(a, np.int32), device=DEV)


def row_bytes_of(bits, H, D, page, page_id, token):
    """Byte numbers of a token's row in the pool, [H, 2, codes + pairs] in an order that does not go by its place."""
    R, G = D * bits // 8, D // 64
    half = 16 * (R + 4 * G)
    strip, r = divmod(token, 16)
    codes = np.concatenate([r * R + 16 * (c ^ ref.turn(R, r)) + np.arange(16) for c in range(R // 16)])
    inner = np.concatenate([codes, 16 * R + r * 4 * G + np.arange(4 * G)])
    base = page_id * H * (page // 16) * 2 * half + (np.arange(H) * (page // 16) + strip) * 2 * half
    return base[:, None, None] + np.arange(2)[:, None] * half + inner


def compacted(pages, bits, H, D, page, table, start, src, cu):
    out = pages.copy()
    flat, new = pages.reshape(-1), out.reshape(-1)
    for b in range(len(start)):
        if start[b] < 0:
            continue
        for r in range(cu[b], cu[b + 1]):
            dst = start[b] + r - cu[b]
            if src[r] < dst:
                continue
            at = [row_bytes_of(bits, H, D, page, table[b, p // page], p % page) for p in (src[r], dst)]
            new[at[1]] = flat[at[0]]
    return out


@pytest.mark.parametrize("bits,D,H,page", [(4, 64, 1, 16), (4, 128, 3, 48), (4, 256, 2, 64), (8, 64, 5, 32), (8, 128, 2, 16), (8, 256, 1, 128)])
@pytest.mark.parametrize("kept", [[6], [0, 1, 5, 0, 16, 3], [700, 0, 300], [1] * 40])
def test_compact(bits, D, H, page, kept):
    rng = np.random.default_rng(D + len(kept))
    B, room = len(kept), 3 * max(kept) + 40
    W = -(-room // page)
    pages = torch.randint(0, 256, (B * W, int(binding.lib().edge0_kv_page_bytes(bits, H, D, page))), dtype=torch.uint8, device=DEV)
    cache = binding.KVCache(B * W, page, H, D, bits, pages=pages)
    table = rng.permutation(B * W).reshape(B, W)
    start = rng.integers(0, 20, B)
    if B > 2:
        start[1] = -1                                   # padding
    cu, src = np.concatenate([[0], np.cumsum(kept)]), []
    for b in range(B):
        own = np.sort(rng.choice(room - 20, kept[b], replace=False))      # overlapping places, some rows where they are
        own[:kept[b] // 4] = np.arange(kept[b] // 4)
        src += list(np.maximum(own, np.arange(kept[b])) + max(start[b], 0))
    before = pages.cpu().numpy()
    want = compacted(before, bits, H, D, page, table, start, src, cu)
    binding.kv_compact(cache, i32(table), i32(start), i32(src), i32(cu))
    assert cache.error() == binding.EDGE0_OK
    assert np.array_equal(pages.cpu().numpy(), want)


def test_compact_of_one_row_each_and_of_repeated_sources():
    bits, D, H, page, B = 4, 128, 2, 32, 5
    pages = torch.randint(0, 256, (10, int(binding.lib().edge0_kv_page_bytes(bits, H, D, page))), dtype=torch.uint8, device=DEV)
    cache = binding.KVCache(10, page, H, D, bits, pages=pages)
    table = np.arange(10).reshape(5, 2)
    before = pages.cpu().numpy()
    binding.kv_compact(cache, i32(table), i32([3, 0, 31, 7, -1]), i32([9, 0, 63, 40, 50]))
    want = compacted(before, bits, H, D, page, table, [3, 0, 31, 7, -1], [9, 0, 63, 40, 50], range(6))
    assert np.array_equal(pages.cpu().numpy(), want)
    # the same source several times, sources out of order: every row as it was before the call
    src = [60, 20, 20, 59, 4, 60]
    before = pages.cpu().numpy()
    binding.kv_compact(cache, i32(table[:1]), i32([0]), i32(src), i32([0, 6]))
    assert np.array_equal(pages.cpu().numpy(), compacted(before, bits, H, D, page, table[:1], [0], src, [0, 6]))
    assert cache.error() == binding.EDGE0_OK


def test_compact_of_the_last_rows_that_an_int_counts():
    """Rows up to 2^31 - 1: a chunk behind the last one is none."""
    bits, D, H, page, n, T = 4, 64, 1, 16, 300, 2 ** 31 - 1
    pages = torch.randint(0, 256, (40, int(binding.lib().edge0_kv_page_bytes(bits, H, D, page))), dtype=torch.uint8, device=DEV)
    cache = binding.KVCache(40, page, H, D, bits, pages=pages)
    table, before = np.random.default_rng(0).permutation(40)[None], pages.cpu().numpy()
    src = torch.empty(T, dtype=torch.int32, device=DEV)
    src[-n:] = torch.arange(2 * n, device=DEV, dtype=torch.int32)[1::2]
    binding.kv_compact(cache, i32(table), i32([0]), src, i32([T - n, T]))
    want = compacted(before, bits, H, D, page, table, [0], range(1, 2 * n, 2), [0, n])
    assert np.array_equal(pages.cpu().numpy(), want) and cache.error() == binding.EDGE0_OK


def test_compact_reports_what_it_cannot_move():
    bits, D, H, page = 8, 64, 2, 16
    pages = torch.randint(0, 256, (6, int(binding.lib().edge0_kv_page_bytes(bits, H, D, page))), dtype=torch.uint8, device=DEV)
    cache = binding.KVCache(6, page, H, D, bits, pages=pages)
    table = np.array([[0, 1, 2], [3, 77, -5]])
    for start, src, cu in (([5], [4], None), ([5], [48], None), ([47, 0], [47, 49], [0, 2, 2]), ([0, 3], [16], [0, 0, 1]),
                           ([0, 3], [40], [0, 0, 1]), ([0], [2 ** 31 - 1], None), ([0, 17], [17, 20], [0, 0, 2])):
        before = pages.clone()
        binding.kv_compact(cache, i32(table[:len(start)]), i32(start), i32(src), None if cu is None else i32(cu))
        assert cache.error() == binding.EDGE0_EINVAL and torch.equal(pages, before)
    # the others of the same call move
    before = pages.cpu().numpy()
    binding.kv_compact(cache, i32(table), i32([0, 2]), i32([9, 8, 12, 17, 5]), i32([0, 3, 5]))
    want = compacted(before, bits, H, D, page, table, [0, 3], [9, 8, 12, 5], [0, 3, 4])
    assert cache.error() == binding.EDGE0_EINVAL
    assert np.array_equal(pages.cpu().numpy(), want)


@pytest.mark.parametrize("bits,D,H,page", [(4, 64, 1, 16), (4, 128, 8, 64), (8, 256, 3, 128), (8, 64, 64, 4096)])
@pytest.mark.parametrize("n", [1, 7, 300])
def test_copy_pages(bits, D, H, page, n):
    nbytes = int(binding.lib().edge0_kv_page_bytes(bits, H, D, page))
    n = min(n, max(2, (1 << 31) // nbytes))
    total = 2 * n + 3
    pages = torch.randint(0, 256, (total, nbytes), dtype=torch.uint8, device=DEV)
    cache = binding.KVCache(total, page, H, D, bits, pages=pages)
    rng = np.random.default_rng(n)
    order = rng.permutation(total)
    dst, src = order[:n].copy(), rng.choice(order[n:], n)            # one page may be copied to several places
    want = pages.clone()
    want[dst] = pages[src]
    more = n > 2
    if more:
        src[1], dst[2] = -1, -7                                        # entries that ask for nothing
        want[dst[1]] = pages[dst[1]]
        want[order[2]] = pages[order[2]]
    binding.kv_copy_pages(cache, i32(src), i32(dst))
    assert torch.equal(pages, want) and cache.error() == binding.EDGE0_OK
    bad = i32([total, 0]), i32([0, total])
    binding.kv_copy_pages(cache, *bad)
    assert torch.equal(pages, want) and cache.error() == binding.EDGE0_EINVAL


def test_moves_in_a_graph():
    bits, D, H, page = 4, 128, 2, 16
    pages = torch.randint(0, 256, (8, int(binding.lib().edge0_kv_page_bytes(bits, H, D, page))), dtype=torch.uint8, device=DEV)
    cache = binding.KVCache(8, page, H, D, bits, pages=pages)
    table, start, src, cu = i32([[0, 1], [2, 3]]), i32([0, 0]), i32([0, 0, 0, 0]), i32([0, 0, 0])
    a, b = i32([-1, -1]), i32([-1, -1])
    before = pages.clone()
    g = torch.cuda.CUDAGraph()
    binding.kv_compact(cache, table, start, src, cu)
    binding.kv_copy_pages(cache, a, b)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        binding.kv_compact(cache, table, start, src, cu)
        binding.kv_copy_pages(cache, a, b)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(pages, before)
    start.copy_(i32([4, 30]))
    src.copy_(i32([9, 20, 31, 31]))
    cu.copy_(i32([0, 2, 4]))
    a.copy_(i32([0, 3]))
    b.copy_(i32([6, 7]))
    g.replay()
    torch.cuda.synchronize()
    want = compacted(before.cpu().numpy(), bits, H, D, page, np.array([[0, 1], [2, 3]]), [4, 30], [9, 20, 31, 31], [0, 2, 4])
    want[6], want[7] = want[0], want[3]
    assert np.array_equal(pages.cpu().numpy(), want)


def test_refusals():
    cache = binding.KVCache(4, 16, 2, 64, 4, device=DEV)
    table, one = i32([[0, 1], [2, 3]]), i32([1, 1])
    for f in (lambda: binding.kv_compact(cache, table, one, i32([1, 2, 3])), lambda: binding.kv_compact(cache, table, one, one.long()),
              lambda: binding.kv_compact(cache, table.cpu(), one, one), lambda: binding.kv_copy_pages(cache, one, i32([1])),
              lambda: binding.kv_copy_pages(cache, one.long(), one), lambda: binding.kv_copy_pages(cache, one[::2], one)):
        with pytest.raises(binding.Edge0Error) as e:
            f()
        assert e.value.code == binding.EDGE0_EINVAL
    binding.kv_copy_pages(cache, one[:0], one[:0])
