"""Rotary positions and moves inside the cache without a GPU: frequencies against their
formulas in exact arithmetic, and what the calls refuse before anything is launched."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from int4_routed_expert_prerouter_gb300 import binding, build
from test_block_ops_refusals import handed, on_gpu  # noqa: F401 (a fixture)

EINVAL, EUNSUP = binding.EDGE0_EINVAL, binding.EDGE0_EUNSUPPORTED
A = C.c_void_p(1 << 20)          # an aligned address that is never read
ODD = C.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def turns(lib, rot, scaling="plain", base=10000.0, factor=1.0, trained=0.0, low=0.0, high=0.0):
    t, rad, m = np.empty(max(1, rot // 2), np.uint64), np.empty(max(1, rot // 2)), C.c_float()
    spec = binding.RopeSpec(rot, binding._ROPE_SCALINGS.get(scaling, scaling), base, factor, trained, low, high)
    code = lib.edge0_rope_turns(C.byref(spec), t.ctypes.data, rad.ctypes.data, C.byref(m))
    return code, t, rad, m.value


@pytest.mark.parametrize("rot", [2, 16, 58, 128, 512])
def test_turns_are_the_radians_as_64_bit_fractions(lib, rot):
    code, t, rad, m = turns(lib, rot, base=500000.0)
    assert code == 0 and m == 1.0
    want = 500000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    assert np.allclose(rad, want, rtol=2.0 ** -50, atol=0)
    # 2^64 / (2 pi) is good to 2^-52 of itself here
    assert all(abs(int(a) - w / (2 * math.pi) * 2.0 ** 64) <= 2.0 ** -50 * int(a) + 1 for a, w in zip(t, rad))


def test_scalings(lib):
    r, base, factor, trained = 128, 500000.0, 16.0, 8192.0
    plain = turns(lib, r, base=base)[2]
    assert np.allclose(turns(lib, r, "linear", base, factor)[2], plain / factor, rtol=1e-15)
    f = turns(lib, r, "base", base, factor)[2]
    # the fastest pair stays, the slowest is slowed down by the factor
    assert f[0] == 1.0 and math.isclose(f[-1], plain[-1] / factor, rel_tol=1e-13)
    code, _, f, m = turns(lib, r, "ramp", base, factor, trained, 1.0, 32.0)
    assert math.isclose(m, 0.1 * math.log(16.0) + 1, rel_tol=1e-7)
    spins = trained * plain / (2 * math.pi)
    ratio = f / plain
    assert (ratio[spins >= 33] == 1).all() and np.allclose(ratio[spins <= 0.99], 1 / factor)
    assert (np.diff(ratio) <= 1e-15).all() and ((ratio < 1) & (ratio > 1 / factor)).sum() > 5
    f = turns(lib, r, "bands", base, factor, trained, 1.0, 4.0)[2]
    keep = np.clip((spins - 1) / 3, 0, 1)
    assert np.allclose(f, plain * keep + plain / factor * (1 - keep), rtol=1e-14)
    # a factor of one changes nothing
    for kind in ("linear", "base", "ramp", "bands"):
        assert np.allclose(turns(lib, r, kind, base, 1.0, trained, 1.0, 4.0)[2], plain, rtol=1e-14)


def test_frequency_refusals(lib):
    nan, inf = float("nan"), float("inf")
    for a in (dict(rot=0), dict(rot=-2), dict(rot=7), dict(rot=8, base=1.0), dict(rot=8, base=nan), dict(rot=8, base=inf),
              dict(rot=8, scaling=9), dict(rot=8, scaling=-1), dict(rot=8, scaling="linear", factor=0.5),
              dict(rot=8, scaling="linear", factor=nan), dict(rot=2, scaling="base", factor=2.0),
              dict(rot=8, scaling="ramp", factor=2.0, trained=0.0, low=1.0, high=4.0),
              dict(rot=8, scaling="ramp", factor=2.0, trained=100.0, low=4.0, high=4.0),
              dict(rot=8, scaling="bands", factor=2.0, trained=100.0, low=0.0, high=4.0)):
        assert turns(lib, **a)[0] == EINVAL, a
    assert turns(lib, 514)[0] == EUNSUP
    spec, m = binding.RopeSpec(8, 0, 10000.0, 1.0, 0, 0, 0), C.c_float()
    assert lib.edge0_rope_turns(None, A, None, C.byref(m)) == EINVAL
    assert lib.edge0_rope_turns(C.byref(spec), None, None, C.byref(m)) == EINVAL


def test_rope_refusals(lib):
    def call(t=A, D=128, rot=128, layout=0, m=1.0, q=A, ldq=512, nq=4, qo=A, ldqo=512, k=A, ldk=256, nk=2, ko=A, ldko=256, T=3,
             st=A, cu=A, B=2):
        return lib.edge0_rope(t, D, rot, layout, m, 0, q, ldq, nq, qo, ldqo, k, ldk, nk, ko, ldko, T, st, cu, B, None)

    inf = float("inf")
    for kw in (dict(t=None), dict(t=C.c_void_p((1 << 20) + 4)), dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(st=None),
               dict(st=ODD), dict(cu=ODD), dict(T=-1), dict(B=0), dict(B=257), dict(cu=None), dict(layout=2), dict(rot=0), dict(rot=3),
               dict(rot=130), dict(D=0, rot=0), dict(m=0.0), dict(m=-1.0), dict(m=inf), dict(m=float("nan")), dict(nq=0), dict(nk=-1),
               dict(q=ODD), dict(qo=ODD), dict(k=ODD), dict(ko=ODD), dict(ldq=504), dict(ldq=516), dict(ldqo=504), dict(ldk=248),
               dict(ldko=260), dict(ldqo=520), dict(ldko=264)):
        assert call(**kw) == EINVAL, kw
    assert call(D=132, rot=16) == EUNSUP and call(D=520, rot=16) == EUNSUP and call(nq=4097, ldq=1 << 20, ldqo=1 << 20) == EUNSUP
    assert call(T=0) == 0 and call(T=0, nk=0, k=None, ko=None) == 0


def test_move_refusals(lib):
    ok = binding.KvCacheDesc(4, 2, 128, 64, 8, A)

    def compact(c=ok, tb=A, B=2, W=3, st=A, src=A, cu=A, T=4):
        return lib.edge0_kv_compact(C.byref(c) if c else None, tb, B, W, st, src, cu, T, None, None)

    for kw in (dict(c=None), dict(c=binding.KvCacheDesc(4, 2, 128, 64, 0, A)), dict(tb=None), dict(st=None), dict(src=None), dict(B=0),
               dict(B=257), dict(W=0), dict(T=-1), dict(cu=None), dict(tb=ODD), dict(st=ODD), dict(src=ODD), dict(cu=ODD)):
        assert compact(**kw) == EINVAL, kw
    assert compact(c=binding.KvCacheDesc(5, 2, 128, 64, 8, A)) == EUNSUP
    assert compact(T=0) == 0 and compact(T=0, src=None) == 0

    def copy(c=ok, src=A, dst=A, n=3):
        return lib.edge0_kv_copy_pages(C.byref(c) if c else None, src, dst, n, None, None)

    for kw in (dict(c=None), dict(src=None), dict(dst=None), dict(n=-1), dict(src=ODD), dict(dst=ODD)):
        assert copy(**kw) == EINVAL, kw
    assert copy(n=0, src=None, dst=None) == 0
    assert copy(c=binding.KvCacheDesc(4, 2, 96, 64, 8, A)) == EUNSUP


def test_own_frequencies_as_the_first_call_of_a_process(handed, monkeypatch):  # noqa: F811
    """A plan of the caller's frequencies needs nothing of the library, so the call itself has to load it."""
    recorder = binding._lib
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "lib", lambda: recorder)
    monkeypatch.setattr(torch.Tensor, "to", lambda t, *a, **kw: on_gpu(t))
    plan = binding.RopePlan(64, radians=np.linspace(0, np.pi, 32))
    q = on_gpu(torch.zeros(3, 2, 64, dtype=torch.float16))
    binding._rope(plan, q, None, on_gpu(torch.zeros(3, dtype=torch.int32)), None, q, None, False, None)
    assert [name for name, _ in handed] == ["edge0_rope"]
