"""Attention of packed prompts on the GPU against its definition in 64 bits."""
import threading

import numpy as np
import pytest
import torch

import flash_ref
from int4_routed_expert_prerouter_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def i32(a):
    return torch.tensor(np.asarray(a, np.int32), device=DEV)


def rows(T, *shape, gen=None):
    return torch.randn(T, *shape, device=DEV, generator=gen).half()


def check(got, q, k, v, cu, ck, scale=None, seqs=None):
    """Rows of all sequences against the definition, each within its bound."""
    D = q.shape[2]
    for b in range(len(cu) - 1) if seqs is None else seqs:
        r, kr = slice(cu[b], cu[b + 1]), slice(ck[b], ck[b + 1])
        n, m = cu[b + 1] - cu[b], ck[b + 1] - ck[b]
        o, bound = flash_ref.attend(q[r].double(), k[kr].double(), v[kr].double(), flash_ref.causal(n, m, DEV), scale or D ** -0.5)
        err = (got[r].double() - o).abs()
        assert (err <= bound).all(), (b, n, m, (err - bound).max().item(), err.max().item())


def cut(counts, lead=0):
    return [int(x) for x in np.concatenate([[0], np.cumsum(counts)]) + lead]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,H", [(1, 1), (4, 4), (8, 2), (5, 1), (6, 2), (16, 2), (64, 1)])
@pytest.mark.parametrize("counts", [[1], [127], [128, 129], [0, 300, 1, 0, 17], [33] * 9])
def test_heads_and_lengths(D, Hq, H, counts):
    cu = cut(counts)
    q, k, v = rows(cu[-1], Hq, D), rows(cu[-1], H, D), rows(cu[-1], H, D)
    got = binding.attn_prompt(q, k, v, i32(cu))
    check(got, q, k, v, cu, cu)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("counts", [[2500], [1025, 2, 1500], [640, 641, 642, 643, 1, 900]])
def test_long_prompts(D, counts):
    cu = cut(counts)
    q, k, v = rows(cu[-1], 6, D), rows(cu[-1], 2, D), rows(cu[-1], 2, D)
    check(binding.attn_prompt(q, k, v, i32(cu)), q, k, v, cu, cu)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,m", [([1], [5000]), ([70], [9000]), ([300, 1, 0, 40], [2000, 1, 700, 3000]), ([50, 200, 3], [20, 0, 3]),
                                 ([513], [12345]), ([1, 1, 1], [128, 129, 4097]), ([2000], [100])])
def test_rows_behind_more_keys_or_fewer(D, n, m):
    """The next part of a prompt behind keys read back; with fewer keys than rows the first rows see none: zeros."""
    cu, ck = cut(n), cut(m)
    q, k, v = rows(cu[-1], 8, D), rows(ck[-1], 2, D), rows(ck[-1], 2, D)
    check(binding.attn_prompt(q, k, v, i32(cu), i32(ck)), q, k, v, cu, ck)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("counts", [[6000], [1, 4500, 130, 5000]])
def test_blocks_cut_at_any_length(D, counts):
    cu = cut(counts)
    q, k, v = rows(cu[-1], 2, D), rows(cu[-1], 2, D), rows(cu[-1], 2, D)
    check(binding.attn_prompt(q, k, v, i32(cu)), q, k, v, cu, cu)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinities_behind_a_row_in_blocks_that_are_cut(D):
    """Keys of the last tiles that only some rows see, in a block that several shares have."""
    n, m = 200, 7000
    q, k, v = rows(n, 4, D), rows(m, 1, D), rows(m, 1, D)
    for at, x in ((m - 150, float("inf")), (m - 90, float("nan")), (m - 1, float("-inf"))):
        v[at, 0, at % D] = x
    got = binding.attn_prompt(q, k, v, i32([0, n]), i32([0, m]))
    seen = flash_ref.causal(n, m, DEV)
    finite = torch.where(v.isfinite(), v, torch.zeros_like(v))
    o, bound = flash_ref.attend(q.double(), k.double(), finite.double(), seen, D ** -0.5)
    for at, x in ((m - 150, float("inf")), (m - 90, float("nan")), (m - 1, float("-inf"))):
        o[seen[:, at], :, at % D] = x
    inf = o.isinf()
    assert torch.equal(got.double()[inf], o[inf])
    assert flash_ref.close(got.masked_fill(inf, 0.0), o.masked_fill(inf, 0.0), bound)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [2, 30, 100])
@pytest.mark.parametrize("m", [256, 512, 2048, 8192])
def test_infinities_in_the_last_of_an_even_number_of_tiles(D, n, m):
    """Blocks of one row tile, whose two streams take the tiles in turn: the last one, which only some rows see in whole, is the second
    stream's, and its infinities are added by the first.  The same bits on every run."""
    H = 24
    q, k, v = rows(n, H, D), rows(m, H, D), rows(m, H, D)
    at = m - n // 2
    v[at, :, 5], v[at, :, 9] = float("nan"), float("inf")
    seen = flash_ref.causal(n, m, DEV)
    finite = torch.where(v.isfinite(), v, torch.zeros_like(v))
    o, bound = flash_ref.attend(q.double(), k.double(), finite.double(), seen, D ** -0.5)
    o[seen[:, at], :, 5], o[seen[:, at], :, 9] = float("nan"), float("inf")
    inf, first = o.isinf(), None
    args = q, k, v, i32([0, n]), i32([0, m])
    for _ in range(60):
        got = binding.attn_prompt(*args)
        first = got if first is None else first
        assert torch.equal(got.view(torch.int16), first.view(torch.int16))
    assert torch.equal(got.isinf(), inf) and (got[inf] > 0).all()
    assert flash_ref.close(got.masked_fill(inf, 0.0), o.masked_fill(inf, 0.0), bound)


def test_without_any_key():
    q, k = rows(70, 4, 128), torch.empty(0, 2, 128, dtype=torch.float16, device=DEV)
    got = binding.attn_prompt(q, k, k, i32([0, 50, 70]), i32([0, 0, 0]))
    assert not got.any()
    got = binding.attn_prompt(q[:0], k, k, i32([0, 0]))
    assert got.shape == (0, 4, 128)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_slices_padding_rows_and_scale(D):
    """Rows cut from a fused projection into a slice; rows of no sequence stay, what lies between stays."""
    Hq, H, T = 4, 2, 800
    wide = rows(T, (Hq + 2 * H) * D + 24)
    q, k, v = (wide[:, a:b].unflatten(1, (-1, D)) for a, b in ((8, 8 + Hq * D), (8 + Hq * D, 8 + (Hq + H) * D), (8 + (Hq + H) * D, 8 + (Hq + 2 * H) * D)))
    room = torch.full((T, Hq * D + 16), 7.0, dtype=torch.float16, device=DEV)
    out = room[:, 8:8 + Hq * D].unflatten(1, (Hq, D))
    cu = [5, 5, 400, 401, 790]
    got = binding.attn_prompt(q, k, v, i32(cu), scale=0.3, out=out)
    assert got is out
    check(got, q, k, v, cu, cu, scale=0.3)
    assert (room[:, :8] == 7).all() and (room[:, 8 + Hq * D:] == 7).all() and (room[:5] == 7).all() and (room[790:] == 7).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_scale,k_offset", [(1.0, 30.0), (300.0, 0.0), (1e-6, 0.0), (40.0, 5.0), (1.0, -1000.0)])
def test_scores_of_any_magnitude(D, q_scale, k_offset):
    cu = cut([700, 260])
    q, k, v = (rows(960, 4, D).float() * q_scale).half(), (rows(960, 2, D).float() + k_offset).half(), rows(960, 2, D)
    check(binding.attn_prompt(q, k, v, i32(cu)), q, k, v, cu, cu)


def equal_scores(T, D, q_size, k_size, q_heads, k_heads, gen):
    """q and k of one dim each that is not zero, so that every score is one product of two fp16, exact in fp32: signs of either kind,
    magnitudes of a few classes."""
    power = lambda n, h, size: torch.where(torch.rand(n, h, generator=gen) < 0.3, -1.0, 1.0) * size * 0.5 ** torch.randint(0, 3, (n, h), generator=gen)
    q, k = torch.zeros(T, q_heads, D), torch.zeros(T, k_heads, D)
    q[..., 3], k[..., 3] = power(T, q_heads, q_size), power(T, k_heads, k_size)
    return q.half().to(DEV), k.half().to(DEV)


def means(q, k, v, seen):
    """What scores far apart but for equal ones give, the mean of the v of a row's largest ones, and how far an fp16 result may be
    off: its rounding, each weight's (the weights are the same number, so the sum's too) and fp32 sums."""
    G = q.shape[1] // k.shape[1]
    wide = lambda x: x.double().repeat_interleave(G, 1)
    s = torch.einsum("nhd,mhd->hnm", q.double(), wide(k)).masked_fill(~seen, -float("inf"))
    p = (s == s.amax(2, keepdim=True)).double()
    p /= p.sum(2, keepdim=True)
    o, a = (torch.einsum("hnm,mhd->nhd", p, x) for x in (wide(v), wide(v).abs()))
    return o, 2.0 ** -11 * o.abs() + 2.0 ** -25 + (2.0 ** -11 + (k.shape[0] / 16 + 64) * 2.0 ** -23) * a


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_size,k_size,scale", [(2001.0, 1111.0, 1.0), (3001.0, 16008.0, None), (50016.0, 40032.0, None),
                                                 (1.375, 1.125, 1e6), (60000.0, 50016.0, 1e6), (513.0, 1025.0, 3.0)])
@pytest.mark.parametrize("n,m", [(300, 300), (40, 3000), (700, 700)])
def test_scores_beyond_what_fp32_tells_apart(D, q_size, k_size, scale, n, m):
    """Exponents of 2^21 up to 2^50, whose fp32 steps are up to 2^26: the largest scores of a row weigh the same, all others nothing."""
    gen = torch.Generator().manual_seed(D + n)
    q, k = equal_scores(m, D, q_size, k_size, 4, 2, gen)
    q, v = q[:n].contiguous(), rows(m, 2, D)
    got = binding.attn_prompt(q, k, v, i32([0, n]), i32([0, m]), scale=scale)
    o, bound = means(q, k, v, flash_ref.causal(n, m, DEV))
    assert ((got.double() - o).abs() <= bound).all(), ((got.double() - o).abs() - bound).nan_to_num(99.0).max().item()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_size,k_size,scale", [(20000.0, 10000.0, None), (3000.0, 3000.0, None), (3000.0, 10.0, 1e4), (1.0, 1.0, 1e6)])
def test_rows_of_huge_scores_beside_ordinary_ones(D, q_size, k_size, scale):
    """Finite, within the bound, and nothing to the rows beside them."""
    n = 260
    q, k, v = rows(n, 4, D), (rows(n, 2, D).float() * k_size).clamp(-60000, 60000).half(), rows(n, 2, D)
    q = (q.float() / (k_size * (scale or D ** -0.5) * D ** 0.5)).half()
    args = k, v, i32([0, n])
    clean = binding.attn_prompt(q, *args, scale=scale)
    far = torch.rand(n, device=DEV) < 0.3
    huge = q.clone()
    huge[far] = (rows(int(far.sum()), 4, D).float() * q_size).clamp(-60000, 60000).half()
    got = binding.attn_prompt(huge, *args, scale=scale)
    assert torch.equal(got[~far], clean[~far])
    check(got, huge, k, v, [0, n], [0, n], scale=scale)
    # (the bound says little of them; they lie between the values that they are means of)
    seen = flash_ref.causal(n, n, DEV)
    for h in range(4):
        vv = v[:, h // 2].float()
        lo = torch.where(seen[:, :, None], vv[None], torch.inf).amin(1)
        hi = torch.where(seen[:, :, None], vv[None], -torch.inf).amax(1)
        assert ((got[:, h].float() >= lo - 0.01) & (got[:, h].float() <= hi + 0.01)).all()


def test_weights_far_below_the_largest():
    """A token of huge V and tiny weight beside small values: weights stay normal far below the largest."""
    n, D = 400, 128
    q, k, v = rows(n, 2, D), rows(n, 1, D), (rows(n, 1, D).float() * 1e-3).half()
    k[10] = k[10] * 0 - 0.7 * torch.sign(q[n - 1, 0])
    v[10] = 30000
    cu = [0, n]
    check(binding.attn_prompt(q, k, v, i32(cu)), q, k, v, cu, cu)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_what_a_row_does_not_see_has_no_influence(D, G, bad):
    """Infinities and NaN in later tokens, in other sequences and behind the last row."""
    H, counts = 2, [200, 130, 333]
    cu = cut(counts, 3)
    T = cu[-1] + 5
    q, k, v = rows(T, H * G, D), rows(T, H, D), rows(T, H, D)
    clean = binding.attn_prompt(q, k, v, i32(cu))
    for name, x in (("k", k), ("v", v)):
        for at in (0, 2, cu[0] + 150, cu[1] + 64, cu[2] - 1, cu[2] + 140, cu[2] + 300, T - 1):
            y = x.clone()
            y[at, 1, D // 2 + 1] = bad
            got = binding.attn_prompt(q, *((y, v) if name == "k" else (k, y)), i32(cu))
            hit = torch.zeros(T, H * G, dtype=torch.bool, device=DEV)
            for b in range(3):
                if cu[b] <= at < cu[b + 1]:
                    hit[at:cu[b + 1], G:] = True
            keep = ~hit
            keep[:cu[0]] = False
            keep[cu[-1]:] = False
            assert torch.equal(got[keep], clean[keep]), (name, at)
            if name == "v" and hit.any():
                dim = got[..., D // 2 + 1][hit]
                assert torch.isnan(dim).all() if bad != bad else ((dim == bad) | torch.isnan(dim)).all(), at
                rest = torch.arange(D, device=DEV) != D // 2 + 1
                assert torch.equal(got[hit][:, rest], clean[hit][:, rest]), at
            if name == "k" and bad != bad and hit.any():
                assert torch.isnan(got[hit]).all()


def test_the_same_bits_whatever_else_is_packed():
    """A sequence's rows do not depend on the numbers beside it, and a call gives the same bits each time."""
    D, counts = 128, [700, 90, 1500, 3]
    cu = cut(counts)
    q, k, v = rows(cu[-1], 8, D), rows(cu[-1], 2, D), rows(cu[-1], 2, D)
    a = binding.attn_prompt(q, k, v, i32(cu))
    for _ in range(3):
        assert torch.equal(binding.attn_prompt(q, k, v, i32(cu)), a)
    k2, v2, q2 = k.clone(), v.clone(), q.clone()
    for x in (q2, k2, v2):
        x[:cu[2]] = float("nan")
    assert torch.equal(binding.attn_prompt(q2, k2, v2, i32(cu))[cu[2]:], a[cu[2]:])


@pytest.mark.parametrize("D,Hq", [(64, 8), (128, 8), (256, 10)])
def test_rows_behind_2_31_elements(D, Hq):
    T, ld, H = 290, 1 << 23, 2
    wide = torch.empty(T, ld, dtype=torch.float16, device=DEV)
    at = np.cumsum([0, Hq * D, H * D, H * D, Hq * D])
    q, k, v, out = (wide[:, a:b].unflatten(1, (-1, D)) for a, b in zip(at, at[1:]))
    for x in (q, k, v):
        x.copy_(rows(*x.shape))
    v[200, 1, 3] = float("inf")
    cu = [0, 20, T]
    binding.attn_prompt(q, k, v, i32(cu), out=out)
    dense = [x.contiguous() for x in (q, k, v)]
    assert torch.equal(out, binding.attn_prompt(*dense, i32(cu)))
    dense[2][200, 1, 3] = 0
    check(out.contiguous().masked_fill(out.isinf(), 0.0)[:200], *dense, [0, 20, 200], [0, 20, 200])


def test_bounds_outside_the_rows_touch_nothing():
    D = 128
    q, k, v = rows(100, 2, D), rows(100, 1, D), rows(100, 1, D)
    guard = torch.full((300, 2, D), 9.0, dtype=torch.float16, device=DEV)
    out = guard[100:200]
    binding.attn_prompt(q, k, v, i32([-50, 40, 1000, 7, 2 ** 31 - 1]), out=out)
    torch.cuda.synchronize()
    assert (guard[:100] == 9).all() and (guard[200:] == 9).all()


def test_in_a_graph_lengths_are_read_at_replay():
    D = 128
    q, k, v = rows(3000, 4, D), rows(3000, 1, D), rows(3000, 1, D)
    cu = i32([0, 1000, 3000])
    g = torch.cuda.CUDAGraph()
    binding.attn_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        a = binding.attn_prompt(q, k, v, cu)
        b = binding.attn_prompt(a, k, v, cu)
    for now in ([0, 1000, 3000], [0, 1, 2999], [0, 0, 0], [0, 2700, 3000]):
        cu.copy_(i32(now))
        g.replay()
        torch.cuda.synchronize()
        want = binding.attn_prompt(q, k, v, cu)
        n = now[-1]
        assert torch.equal(a[:n], want[:n])
        assert torch.equal(b[:n], binding.attn_prompt(a, k, v, cu)[:n])


def test_threads_and_streams():
    D = 128
    cases = []
    for i in range(4):
        cu = cut([300 + 100 * i, 5000])
        q, k, v = rows(cu[-1], 4, D), rows(cu[-1], 1, D), rows(cu[-1], 1, D)
        cases.append((q, k, v, i32(cu)))
    want = [binding.attn_prompt(*c) for c in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]

    def work(i):
        s = torch.cuda.Stream()
        for j in range(12):
            got[i].append(binding.attn_prompt(*cases[i], stream=s if j % 2 else None))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(4):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,m", [([300, 5], [300, 5]), ([60, 7], [9000, 70])])
def test_without_waiting(D, n, m):
    """Waits that run out give NaN and leave the next call as it would have been."""
    cu, ck = cut(n, 2), cut(m)
    q, k, v = rows(cu[-1] + 3, 8, D), rows(ck[-1], 2, D), rows(ck[-1], 2, D)
    clean = binding.attn_prompt(q, k, v, i32(cu), i32(ck), out=torch.full_like(q, 5.0))
    for _ in range(3):
        binding.set_wait_limit(0)
        try:
            got = binding.attn_prompt(q, k, v, i32(cu), i32(ck), out=torch.full_like(q, 5.0))
        finally:
            binding.set_wait_limit()
        assert torch.isnan(got[cu[0]:cu[-1]]).all() and (got[:2] == 5).all() and (got[cu[-1]:] == 5).all()
        assert torch.equal(binding.attn_prompt(q, k, v, i32(cu), i32(ck), out=torch.full_like(q, 5.0)), clean)


@pytest.mark.parametrize("D,G", [(64, 4), (128, 4), (256, 4), (128, 5), (128, 1)])
@pytest.mark.parametrize("n,m", [([300, 5], [300, 5]), ([60, 7], [9000, 70]), ([1, 130, 64], [100, 700, 64])])
def test_waits_that_run_out_on_the_way(D, G, n, m):
    """Limits shorter than the call: rows that lack something are NaN, the others as they should be, and so is the next call."""
    cu, ck = cut(n, 2), cut(m)
    q, k, v = rows(cu[-1] + 3, 2 * G, D), rows(ck[-1], 2, D), rows(ck[-1], 2, D)
    call = lambda: binding.attn_prompt(q, k, v, i32(cu), i32(ck), out=torch.full_like(q, 5.0))
    clean = call()
    for limit in (1, 500, 1000, 2000, 4000, 8000, 16000) * 3:
        binding.set_wait_limit(limit)
        try:
            got = call()
        finally:
            binding.set_wait_limit()
        lost = torch.isnan(got).all(2)
        assert torch.equal(got[~lost], clean[~lost]) and not lost[:2].any() and not lost[cu[-1]:].any(), limit
        assert torch.equal(call(), clean), limit


def test_refusals():
    q, k, cu = rows(10, 4, 128), rows(10, 2, 128), i32([0, 10])
    bad = [lambda: binding.attn_prompt(q, k, k[:5], cu), lambda: binding.attn_prompt(q, k[:5], k[:5], cu),
           lambda: binding.attn_prompt(q, rows(10, 3, 128), rows(10, 3, 128), cu), lambda: binding.attn_prompt(q, k, k, cu.long()),
           lambda: binding.attn_prompt(q, k, k, cu[:1]), lambda: binding.attn_prompt(q, k, k, cu, i32([0, 1, 2])),
           lambda: binding.attn_prompt(q.float(), k, k, cu), lambda: binding.attn_prompt(q, k, k, cu, scale=0.0),
           lambda: binding.attn_prompt(q, k, k, cu, scale=float("nan")), lambda: binding.attn_prompt(q, k, k, cu, out=q[:5]),
           lambda: binding.attn_prompt(q, k.transpose(0, 1), k.transpose(0, 1), cu), lambda: binding.attn_prompt(q, k, k, cu.cpu()),
           lambda: binding.attn_prompt(q, k, k, cu, out=q[:1].expand(10, 4, 128)),
           lambda: binding.attn_prompt(q, k[:1].expand(10, 2, 128), k, cu),
           lambda: binding.attn_prompt(q, k, k, cu, workspace=torch.empty(100, dtype=torch.uint8, device=DEV))]
    for i, f in enumerate(bad):
        with pytest.raises(binding.Edge0Error) as e:
            f()
        assert e.value.code == binding.EDGE0_EINVAL, i
    for f in (lambda: binding.attn_prompt(rows(10, 2, 96), rows(10, 1, 96), rows(10, 1, 96), cu),
              lambda: binding.attn_prompt(rows(10, 65, 64), rows(10, 1, 64), rows(10, 1, 64), cu)):
        with pytest.raises(binding.Edge0Error) as e:
            f()
        assert e.value.code == binding.EDGE0_EUNSUPPORTED
