"""Projection, KV-cache and attention calls without a GPU: sizes, refusals on the
host (nothing is launched), the reference forms' own definitions."""
import ctypes as C

import numpy as np
import pytest

import block_ref as ref
from int4_routed_expert_prerouter_gb300 import binding, build

EINVAL, EUNSUP = binding.EDGE0_EINVAL, binding.EDGE0_EUNSUPPORTED
A = C.c_void_p(1 << 20)          # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def desc(bits=4, H=2, D=128, page=64, n=8, pages=A):
    return binding.KvCacheDesc(bits, H, D, page, n, pages)


def test_page_bytes(lib):
    # per token and head: K and V codes plus one (s, b) pair per 64 dims each
    assert lib.edge0_kv_page_bytes(4, 1, 128, 16) == 16 * 2 * (64 + 8)
    assert lib.edge0_kv_page_bytes(8, 3, 256, 48) == 3 * 48 * 2 * (256 + 16)
    assert lib.edge0_kv_page_bytes(4, 64, 64, 4096) == 64 * 4096 * 2 * (32 + 4)
    for bad in ((5, 1, 128, 16), (16, 1, 128, 16), (4, 0, 128, 16), (4, 65, 128, 16), (4, 1, 96, 16), (4, 1, 512, 16),
                (4, 1, 128, 0), (4, 1, 128, 24), (4, 1, 128, 4112), (4, 1, 128, -16)):
        assert lib.edge0_kv_page_bytes(*bad) == 0, bad


def test_q4_linear_refusals(lib):
    f = lib.edge0_q4_linear
    good = dict(w=A, out=48, n=128, x=A, ldx=128, B=2, y=A, ldy=48)

    def call(**kw):
        a = {**good, **kw}
        return f(a["w"], a["out"], a["n"], a["x"], a["ldx"], a["B"], a["y"], a["ldy"], None)

    for kw in (dict(w=None), dict(x=None), dict(y=None), dict(out=0), dict(n=0), dict(n=100), dict(B=0), dict(B=257),
               dict(ldx=120), dict(ldx=132), dict(ldy=47), dict(x=C.c_void_p((1 << 20) + 8)),
               dict(w=C.c_void_p((1 << 20) + 8)), dict(y=C.c_void_p((1 << 20) + 1))):
        assert call(**kw) == EINVAL, kw
    most = 1 << 28
    assert call(out=most + 1, ldy=most + 1) == EUNSUP and call(n=most + 64, ldx=most + 64) == EUNSUP


def test_cache_refusals(lib):
    ap, rd = lib.edge0_kv_append, lib.edge0_kv_read
    ok = desc()

    def append(c=ok, k=A, ldk=256, v=A, ldv=256, T=2, tb=A, B=2, W=3, st=A, cu=A):
        return ap(C.byref(c) if c else None, k, ldk, v, ldv, T, tb, B, W, st, cu, None, None)

    def read(c=ok, T=2, tb=A, B=2, W=3, st=A, cu=A, k=A, v=A):
        return rd(C.byref(c) if c else None, tb, B, W, st, cu, T, k, v, None, None)

    odd = C.c_void_p((1 << 20) + 2)
    for kw in (dict(c=None), dict(c=desc(pages=None)), dict(c=desc(pages=odd)), dict(c=desc(n=0)), dict(c=desc(H=0)),
               dict(k=None), dict(v=None), dict(tb=None), dict(st=None), dict(B=0), dict(B=257), dict(W=0), dict(T=-1),
               dict(cu=None, T=3), dict(tb=odd), dict(cu=odd)):
        assert append(**kw) == EINVAL, kw
        if "T" not in kw or kw["T"] < 0 or "cu" in kw:
            assert read(**kw) == EINVAL, kw
    for kw in (dict(k=odd), dict(v=odd), dict(ldk=248), dict(ldv=260)):
        assert append(**kw) == EINVAL, kw
    assert read(k=odd) == EINVAL and read(v=odd) == EINVAL
    for c in (desc(bits=5), desc(D=96), desc(page=40), desc(H=65)):
        assert append(c=c) == EUNSUP and read(c=c) == EUNSUP
    assert append(T=0) == 0 and read(T=0) == 0          # nothing to do


def test_attention_refusals(lib):
    f = lib.edge0_attn_decode
    ok = desc()
    big = 1 << 40

    def call(c=ok, q=A, ldq=1024, B=2, Hq=8, tb=A, W=3, lens=A, prefix=A, P=5, scale=0.1, out=A, ldo=1024, ws=A,
             nb=big):
        return f(C.byref(c) if c else None, q, ldq, B, Hq, tb, W, lens, prefix, P, scale, out, ldo, None, ws, nb, None)

    odd = C.c_void_p((1 << 20) + 8)
    inf = float("inf")
    for kw in (dict(c=None), dict(q=None), dict(tb=None), dict(lens=None), dict(out=None), dict(ws=None), dict(B=0),
               dict(B=257), dict(Hq=0), dict(Hq=7), dict(W=0), dict(P=-1), dict(prefix=None), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=inf), dict(scale=float("nan")), dict(ldq=1016), dict(ldq=1028),
               dict(ldo=1016), dict(ldo=1028), dict(q=odd), dict(out=odd), dict(ws=odd), dict(nb=0)):
        assert call(**kw) == EINVAL, kw
    assert call(Hq=2 * 65, ldq=1 << 15, ldo=1 << 15) == EUNSUP
    assert call(c=desc(bits=3)) == EUNSUP
    assert call(P=(1 << 30) + 1) == EUNSUP
    ws = lib.edge0_attn_workspace_bytes
    assert ws(C.byref(ok), 2, 8) > 0
    assert ws(C.byref(ok), 0, 8) == ws(C.byref(ok), 257, 8) == ws(C.byref(ok), 2, 7) == ws(C.byref(ok), 2, 130) == 0


def test_reference_quantiser():
    # whole-step data: 0..15 and 0..255 in steps of a power of two are exact
    for bits in (4, 8):
        x = (np.arange(64) % (2 ** bits) * 0.125 - 3.0).astype(np.float16)
        x[63] = (2 ** bits - 1) * 0.125 - 3.0
        q, s, b = ref.quantise(x, bits)
        assert s[0] == 0.125 and b[0] == -3.0
        assert np.array_equal(ref.values(q, s, b), x.astype(np.float64))
    # constant groups, and ties go to the even code
    q, s, b = ref.quantise(np.full(64, 7.5, np.float16), 4)
    assert s[0] == 0 and not q.any() and b[0] == 7.5
    x = np.zeros(64, np.float16)
    x[1], x[2], x[3] = 15.0, 2.5, 3.5
    q, s, b = ref.quantise(x, 4)
    assert s[0] == 1 and q[2] == 2 and q[3] == 4
    # the widest range: no finite value comes back as infinity
    for bits in (4, 8):
        x = np.linspace(-65504, 65504, 64).astype(np.float16)
        q, s, b = ref.quantise(x, bits)
        assert np.isfinite(ref.values(q, s, b).astype(np.float16)).all()
        x[:] = np.linspace(60000, 65504, 64)
        q, s, b = ref.quantise(x, bits)
        assert np.isfinite(ref.values(q, s, b).astype(np.float16)).all()
    # a non-finite value marks its group only
    x = np.ones(128, np.float16)
    x[70] = np.inf
    q, s, b = ref.quantise(x, 8)
    assert s[0] == 0 and np.isnan(s[1]) and np.isnan(b[1])


def test_page_image_places_every_byte_once():
    rng = np.random.default_rng(0)
    for bits, D, H, page in ((4, 64, 1, 16), (4, 128, 2, 48), (8, 128, 1, 16), (8, 256, 2, 32), (8, 64, 1, 16), (4, 256, 1, 16)):
        R = D * bits // 8
        for r in range(16):
            assert sorted(c ^ ref.turn(R, r) for c in range(R // 16)) == list(range(R // 16))
        # eight consecutive rows' piece c: eight different 16-byte banks of a 128-byte line
        for r0 in (0, 8):
            for c in range(R // 16):
                assert len({(r * R // 16 + (c ^ ref.turn(R, r))) % 8 for r in range(r0, r0 + 8)}) == 8
        c = ref.Cache(2, page, H, D, bits, rng)
        assert c.image.shape == (2, H * page * 2 * (R + D // 16))


def test_reference_attention_by_hand():
    # two tokens with equal scores average; one token returns its value
    k = np.zeros((2, 1, 64))
    v = np.stack([np.full((1, 64), 1.0), np.full((1, 64), 3.0)])
    o, _ = ref.attention(np.ones((2, 64)), k, v, np.abs(v), np.abs(v), 0.125)
    assert np.allclose(o, 2.0)
    o, _ = ref.attention(np.ones((2, 64)), k[:1], v[:1], np.abs(v[:1]), v[:1], 0.125)
    assert np.allclose(o, 1.0)
    o, _ = ref.attention(np.ones((2, 64)), k[:0], v[:0], v[:0], v[:0], 0.125)
    assert not o.any()
