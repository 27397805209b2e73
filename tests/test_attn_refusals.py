"""Attention of prompts and of drafted tokens without a GPU: what the calls refuse before anything is
launched, and counts that the binding has to refuse."""
import ctypes as C

import pytest
import torch

from int4_routed_expert_prerouter_gb300 import binding, build
from test_block_ops_refusals import cache, handed, meta, on_gpu  # noqa: F401 (a fixture)

EINVAL, EUNSUP = binding.EDGE0_EINVAL, binding.EDGE0_EUNSUPPORTED
A = C.c_void_p(1 << 20)          # an aligned address that is never read
ODD2, ODD8 = C.c_void_p((1 << 20) + 2), C.c_void_p((1 << 20) + 8)
INF, NAN, BIG = float("inf"), float("nan"), 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def test_prompt_refusals(lib):
    def call(q=A, ldq=1024, T=9, Hq=8, k=A, ldk=256, v=A, ldv=256, Tk=9, H=2, D=128, cu=A, ck=None, B=2, scale=0.1, out=A, ldo=1024,
             ws=A, nb=BIG):
        return lib.edge0_attn_prompt(q, ldq, T, Hq, k, ldk, v, ldv, Tk, H, D, cu, ck, B, scale, out, ldo, ws, nb, None)

    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(cu=None), dict(out=None), dict(ws=None), dict(B=0), dict(B=257),
               dict(T=-1), dict(Tk=-1), dict(Hq=0), dict(H=0), dict(Hq=7), dict(scale=0.0), dict(scale=-1.0), dict(scale=INF),
               dict(scale=NAN), dict(ldq=1016), dict(ldq=1028), dict(ldk=248), dict(ldk=260), dict(ldv=248), dict(ldv=260),
               dict(ldo=1016), dict(ldo=1028), dict(q=ODD8), dict(k=ODD8), dict(v=ODD8), dict(out=ODD8), dict(ws=ODD8),
               dict(cu=ODD2), dict(ck=ODD2), dict(Tk=10), dict(nb=0),
               dict(nb=lib.edge0_attn_prompt_workspace_bytes(128) - 1)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(D=96), dict(D=512), dict(Hq=130, ldq=130 * 128, ldo=130 * 128), dict(T=1 << 30, Tk=1 << 30)):
        assert call(**kw) == EUNSUP, kw
    assert call(T=0, ck=A) == 0 and call(T=0, Tk=0) == 0             # nothing to do
    assert lib.edge0_attn_prompt_workspace_bytes(96) == 0


def test_tree_refusals(lib):
    ok = binding.KvCacheDesc(4, 2, 128, 64, 8, A)

    def call(c=ok, q=A, ldq=1024, T=9, Hq=8, tb=A, B=2, W=3, lens=A, cu=A, mask=A, words=1, scale=0.1, out=A, ldo=1024, ws=A, nb=BIG):
        return lib.edge0_attn_tree(C.byref(c) if c else None, q, ldq, T, Hq, tb, B, W, lens, cu, mask, words, scale, out, ldo, None,
                                   ws, nb, None)

    for kw in (dict(c=None), dict(c=binding.KvCacheDesc(4, 2, 128, 64, 0, A)), dict(q=None), dict(tb=None), dict(lens=None), dict(cu=None),
               dict(out=None), dict(ws=None), dict(B=0), dict(B=257), dict(W=0), dict(T=-1), dict(Hq=0), dict(Hq=7), dict(words=0),
               dict(words=-1), dict(mask=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=INF), dict(scale=NAN), dict(ldq=1016),
               dict(ldq=1028), dict(ldo=1016), dict(ldo=1028), dict(q=ODD8), dict(out=ODD8), dict(ws=ODD8), dict(tb=ODD2),
               dict(lens=ODD2), dict(cu=ODD2), dict(mask=ODD2), dict(nb=0),
               dict(nb=lib.edge0_attn_tree_workspace_bytes(C.byref(ok)) - 1)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(c=binding.KvCacheDesc(5, 2, 128, 64, 8, A)), dict(c=binding.KvCacheDesc(4, 2, 96, 64, 8, A)),
               dict(Hq=130, ldq=130 * 128, ldo=130 * 128), dict(T=1 << 30), dict(words=(1 << 20) + 1)):
        assert call(**kw) == EUNSUP, kw
    assert call(T=0) == 0 and call(T=0, mask=None, words=0) == 0     # nothing to do
    assert lib.edge0_attn_tree_workspace_bytes(C.byref(binding.KvCacheDesc(5, 2, 128, 64, 8, A))) == 0


def test_counts_that_do_not_fit_an_int_are_refused(handed):  # noqa: F811
    """2^32 + n would arrive as n."""
    big, i32 = 1 << 32, torch.int32
    q, k = on_gpu(torch.zeros(1, 4, 64, dtype=torch.float16)), on_gpu(torch.zeros(1, 2, 64, dtype=torch.float16))
    tall = lambda h: on_gpu(torch.empty(big + 1, h, 64, dtype=torch.float16, device="meta"))
    one, lens, cu = on_gpu(torch.zeros(1, 1, dtype=i32)), on_gpu(torch.zeros(1, dtype=i32)), on_gpu(torch.zeros(2, dtype=i32))
    calls = [lambda: binding._attn_prompt(tall(4), k, k, cu, cu, None, None, None, 0, None),
             lambda: binding._attn_prompt(q, tall(2), tall(2), cu, cu, None, None, None, 0, None),
             lambda: binding._attn_prompt(q, k, k, meta(big + 2, dtype=i32), None, None, None, None, 0, None),
             lambda: binding._attn_tree(cache(), tall(4), one, lens, cu, None, None, None, None, None),
             lambda: binding._attn_tree(cache(), q, meta(1, big + 1, dtype=i32), lens, cu, None, None, None, None, None),
             lambda: binding._attn_tree(cache(), q, meta(big + 1, 1, dtype=i32), meta(big + 1, dtype=i32), meta(big + 2, dtype=i32), None,
                                        None, None, None, None),
             lambda: binding._attn_tree(cache(), q, one, lens, cu, meta(1, big + 1, dtype=i32), None, None, None, None)]
    for i, call in enumerate(calls):
        with pytest.raises(binding.Edge0Error) as e:
            call()
        assert e.value.code == EUNSUP, i
    assert not handed
