"""Rotary positions on the GPU against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from int4_routed_expert_prerouter_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def i32(a):
    return torch.tensor(np.asarray(a, np.int32), device=DEV)


def turned(x, pos, plan, backward=False):
    """x [T, H, D] float64 at positions pos [T], and how far an fp16 result may be off: half its step, and
    fp32 cosines and sines (2^-22 each), magnitude, products and sum (2^-24 each) of both terms."""
    rot, half = plan.rot_dim, plan.layout == 0
    ang = np.asarray(pos, np.float64)[:, None] * plan.radians * (-1 if backward else 1)
    c, s = (plan.magnitude * f(ang)[:, None, :] for f in (np.cos, np.sin))
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if half else (x[..., 0:rot:2], x[..., 1:rot:2])
    y, parts = x.copy(), np.zeros_like(x)
    u, v = a * c - b * s, a * s + b * c
    big = plan.magnitude * (np.abs(a) + np.abs(b))
    for dst, (p, q) in ((y, (u, v)), (parts, (big, big))):
        if half:
            dst[..., :rot // 2], dst[..., rot // 2:rot] = p, q
        else:
            dst[..., 0:rot:2], dst[..., 1:rot:2] = p, q
    return y, np.where(parts > 0, 2.0 ** -11 * np.abs(y) + 2.0 ** -25 + 2.0 ** -20 * parts, 0.0)


def check(got, x, pos, plan, rows=slice(None), backward=False):
    want, bound = turned(x.double().cpu().numpy()[rows], np.asarray(pos)[rows], plan, backward)
    err = np.abs(got.double().cpu().numpy()[rows] - want)
    assert (err <= bound).all(), (err - bound).max()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 64), (256, 64), (64, 58), (128, 2), (8, 8), (512, 512), (24, 12), (72, 40)])
def test_layouts_and_parts_of_the_head(layout, D, rot):
    plan = binding.RopePlan(D, rot, base=500000.0, layout=layout, device=DEV)
    T = 37
    q, k = torch.randn(T, 5, D, device=DEV).half(), torch.randn(T, 2, D, device=DEV).half()
    pos = np.random.default_rng(D + rot).integers(0, 200000, T)
    pos[:3] = 0, 1, 2 ** 31 - 1
    qo, ko = binding.rope(plan, q, k, i32(pos))
    check(qo, q, pos, plan)
    check(ko, k, pos, plan)
    # forth and back: the transpose of a rotation is its inverse (two roundings, each half a step of a value
    # of at most |a| + |b|)
    back, _ = binding.rope(plan, qo, None, i32(pos), backward=True)
    check(back, qo, pos, plan, backward=True)
    assert (back.float() - q.float()).abs().max() <= 4 * 2.0 ** -11 * 2 * q.float().abs().max()


@pytest.mark.parametrize("scaling,extra", [("linear", {}), ("base", {}), ("ramp", dict(trained_len=4096.0, low=1.0, high=32.0)),
                                           ("bands", dict(trained_len=4096.0, low=1.0, high=4.0))])
def test_scalings(scaling, extra):
    plan = binding.RopePlan(128, 96, base=10000.0, layout="half", scaling=scaling, factor=8.0, device=DEV, **extra)
    q = torch.randn(50, 3, 128, device=DEV).half()
    pos = np.arange(50) * 2711
    qo, none = binding.rope(plan, q, None, i32(pos))
    assert none is None
    check(qo, q, pos, plan)


def test_own_frequencies():
    rad = np.linspace(0, np.pi, 32)
    plan = binding.RopePlan(64, radians=rad, magnitude=0.5, device=DEV)
    q = torch.randn(9, 1, 64, device=DEV).half()
    pos = np.arange(9) * 100001
    check(binding.rope(plan, q, None, i32(pos))[0], q, pos, plan)


@pytest.mark.parametrize("counts", [[5], [0, 3, 0, 1, 17, 0], [1] * 64, [3000, 1, 500], [0, 0], [1300] * 7])
@pytest.mark.parametrize("layout,rot", [("half", 128), ("interleaved", 32), ("half", 100)])
def test_packed_sequences_padding_and_slices(counts, layout, rot):
    """Rows cut from a fused projection, written into slices; padding sequences and rows of none stay."""
    plan = binding.RopePlan(128, rot, layout=layout, device=DEV)
    B, lead, tail = len(counts), 2, 3
    cu = np.concatenate([[0], np.cumsum(counts)]) + lead
    T = int(cu[-1]) + tail
    start = np.random.default_rng(B).integers(0, 100000, B)
    if B > 2:
        start[2] = -1
    wide = torch.randn(T, 8 * 128 + 8, device=DEV).half()
    q, k = wide[:, 8:8 + 4 * 128].unflatten(1, (4, 128)), wide[:, 8 + 6 * 128:].unflatten(1, (2, 128))
    room = torch.full((T, 7 * 128), 3.0, dtype=torch.float16, device=DEV)
    qo, ko = room[:, :512].unflatten(1, (4, 128)), room[:, 640:].unflatten(1, (2, 128))
    got = binding.rope(plan, q, k, i32(start), i32(cu), q_out=qo, k_out=ko)
    assert got[0] is qo and got[1] is ko
    pos, rows = np.zeros(T), np.zeros(T, bool)
    for b in range(B):
        if start[b] >= 0:
            rows[cu[b]:cu[b + 1]] = True
            pos[cu[b]:cu[b + 1]] = start[b] + np.arange(counts[b])
    check(qo, q, pos, plan, rows)
    check(ko, k, pos, plan, rows)
    assert (room[:, 512:640] == 3).all() and (room[torch.from_numpy(~rows).to(DEV)] == 3).all()
    # in place
    want = wide.clone()
    want[:, 8:520].unflatten(1, (4, 128))[torch.from_numpy(rows).to(DEV)] = qo[torch.from_numpy(rows).to(DEV)]
    binding.rope(plan, q, None, i32(start), i32(cu), q_out=q)
    assert torch.equal(wide, want)


def test_special_values_stay_in_their_pair():
    plan = binding.RopePlan(64, device=DEV)
    q = torch.randn(4, 2, 64, device=DEV).half()
    clean = binding.rope(plan, q, None, i32([3, 4, 5, 6]))[0]
    q[1, 0, 7] = float("nan")
    q[2, 1, 40] = float("inf")
    got = binding.rope(plan, q, None, i32([3, 4, 5, 6]))[0]
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[1, 0, [7, 39]] = True
    hit[2, 1, [8, 40]] = True
    assert torch.equal(got[~hit], clean[~hit]) and not torch.isfinite(got[hit]).any()


def test_the_last_rows_that_an_int_counts():
    """2^31 - 1 rows, in place; those of no sequence stay."""
    T, n = 2 ** 31 - 1, 37
    plan = binding.RopePlan(8, device=DEV)
    q = torch.empty(T, 1, 8, dtype=torch.float16, device=DEV)
    q[-2 * n:] = torch.randn(2 * n, 1, 8, device=DEV).half()
    before = q[-2 * n:].clone()
    binding.rope(plan, q, None, i32([1000]), i32([T - n, T]), q_out=q)
    assert torch.equal(q[-2 * n:-n], before[:n])
    check(q[-n:], before[n:], 1000 + np.arange(n), plan)


def test_in_a_graph_and_on_another_stream():
    plan = binding.RopePlan(128, device=DEV)
    q, k = torch.randn(33, 4, 128, device=DEV).half(), torch.randn(33, 1, 128, device=DEV).half()
    pos = i32(np.arange(33))
    want = binding.rope(plan, q, k, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.rope(plan, q, k, pos, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = binding.rope(plan, q, k, pos)
    pos += 1000
    want = binding.rope(plan, q, k, pos)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_refusals():
    plan = binding.RopePlan(128, device=DEV)
    q, pos = torch.zeros(3, 2, 128, device=DEV, dtype=torch.float16), i32([1, 2, 3])
    for a in ((q[:, :, :64], None, pos), (q, q[:2], pos), (q, None, pos[:2]), (q.float(), None, pos), (q, None, pos.long()),
              (q.transpose(1, 2).contiguous().transpose(1, 2), None, pos), (q.cpu(), None, pos)):
        with pytest.raises(binding.Edge0Error) as e:
            binding.rope(plan, *a)
        assert e.value.code == binding.EDGE0_EINVAL
    with pytest.raises(binding.Edge0Error):
        binding.rope(plan, q, None, pos, q_out=q[:1].expand(3, 2, 128))
    for kw in (dict(rot_dim=3), dict(rot_dim=130), dict(layout="both"), dict(scaling="more"), dict(radians=[4.0] * 64), dict(radians=[0.1]),
               dict(magnitude=0.0), dict(base=0.5)):
        with pytest.raises(binding.Edge0Error) as e:
            binding.RopePlan(128, device=DEV, **kw)
        assert e.value.code == binding.EDGE0_EINVAL
    assert binding.rope(plan, q[:0], None, pos[:0])[0].shape == (0, 2, 128)
