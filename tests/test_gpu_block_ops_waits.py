"""Waits inside the projection and attention kernels that run out: with a limit of zero every wait
is given up, which has to end the launch, be seen by the caller and leave the next call as it
would have been."""
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


@pytest.fixture
def no_waiting():
    """Calls the function it is given with waits that run out at once; the limit is put back whatever happens."""
    def run(f):
        binding.set_wait_limit(0)
        try:
            return f()
        finally:
            binding.set_wait_limit()
            torch.cuda.synchronize()
    yield run
    binding.set_wait_limit()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, np.int32))).to(DEV)


def filled(bits, D, H, page, n_pages, seed):
    """A cache of random tokens: one chunk of pages with what they hold, repeated."""
    c = ref.Cache(8, page, H, D, bits, np.random.default_rng(seed))
    image = torch.from_numpy(c.image).to(DEV)
    return binding.KVCache(n_pages, page, H, D, bits, pages=image.repeat(-(-n_pages // 8), 1)[:n_pages].contiguous())


@pytest.mark.parametrize("B,n_in,n_out", [(1, 2048, 20000), (7, 2048, 5120), (16, 1536, 9000), (64, 1536, 6144), (200, 2048, 2000)])
def test_projection_without_waiting(no_waiting, B, n_in, n_out):
    q, s, b = (t.to(DEV) for t in inputs.int4_stack(B, 0, 1, 1, n_out, n_in))
    packed = binding.pack_q4_rows((q, s, b))
    x = torch.randn(B, n_in, device=DEV).half()
    clean = binding.q4_linear(packed, n_out, x)
    for _ in range(3):
        assert torch.isnan(no_waiting(lambda: binding.q4_linear(packed, n_out, x))).all()
        assert torch.equal(binding.q4_linear(packed, n_out, x), clean)


@pytest.mark.parametrize("bits,D,G", [(4, 128, 4), (8, 128, 8), (4, 256, 8), (8, 64, 16), (4, 128, 16), (8, 256, 2)])
def test_own_contexts_without_waiting(no_waiting, bits, D, G):
    H, page, B = 2, 64, 6
    cache = filled(bits, D, H, page, 40 * B, D + G)
    table, lens = i32(np.random.default_rng(1).permutation(40 * B).reshape(B, 40)), i32([2500, 1, 0, 700, 2048, 33])
    q = torch.randn(B, H * G, D, device=DEV).half()
    clean = binding.attn_decode(cache, q, table, lens)
    for _ in range(3):
        no_waiting(lambda: binding.attn_decode(cache, q, table, lens))
        assert cache.error() == binding.EDGE0_ETIMEOUT
        assert torch.equal(binding.attn_decode(cache, q, table, lens), clean) and cache.error() == binding.EDGE0_OK


@pytest.mark.parametrize("bits,D,B,G", [(4, 128, 5, 4), (8, 128, 70, 4), (4, 256, 9, 8), (8, 256, 20, 16), (4, 64, 33, 4), (8, 64, 17, 16)])
@pytest.mark.parametrize("P", [30, 700, 2051])
def test_prefix_on_the_tensor_cores_without_waiting(no_waiting, bits, D, B, G, P):
    H, page = 2, 64
    cache = filled(bits, D, H, page, 40, D + G)
    table, lens, pre = i32(np.zeros((B, 1))), i32(np.zeros(B)), i32(np.random.default_rng(1).permutation(40))
    q = torch.randn(B, H * G, D, device=DEV).half()
    clean = binding.attn_decode(cache, q, table, lens, pre, P)
    for _ in range(3):
        no_waiting(lambda: binding.attn_decode(cache, q, table, lens, pre, P))
        assert cache.error() == binding.EDGE0_ETIMEOUT
        assert torch.equal(binding.attn_decode(cache, q, table, lens, pre, P), clean) and cache.error() == binding.EDGE0_OK


@pytest.mark.parametrize("bits,D,B,G,P", [(4, 128, 6, 4, 0), (8, 256, 3, 2, 0), (8, 64, 6, 16, 0), (4, 128, 2, 4, 300), (8, 64, 3, 8, 200),
                                          (4, 128, 33, 4, 700), (8, 64, 40, 8, 1500), (4, 256, 20, 8, 300)])
def test_rows_that_lack_tokens_are_nan(no_waiting, bits, D, B, G, P):
    """Not what an earlier call left in the workspace, nor a softmax over fewer tokens; rows without
    any token and padding rows as ever."""
    H, page = 2, 64
    cache = filled(bits, D, H, page, 40, D + G)
    rng = np.random.default_rng(2)
    table, pre = i32(rng.integers(0, 40, (B, 12))), i32(rng.permutation(40))
    n = rng.integers(1, 12 * page, B)
    n[0], n[1] = 0, -1
    lens = i32(n)
    q, other = torch.randn(2, B, H * G, D, device=DEV).half()
    ws = torch.empty(binding.attn_workspace_bytes(cache, B, H * G), dtype=torch.uint8, device=DEV)
    clean = binding.attn_decode(cache, q, table, lens, pre, P, workspace=ws, out=torch.full_like(q, 5.0))
    for _ in range(2):
        got = no_waiting(lambda: binding.attn_decode(cache, other, table, lens, pre, P, workspace=ws, out=torch.full_like(q, 5.0)))
        assert torch.isnan(got[2:]).all() and (got[1] == 5).all()
        assert torch.isnan(got[0]).all() if P else not got[0].any()
        assert cache.error() == binding.EDGE0_ETIMEOUT
        assert torch.equal(binding.attn_decode(cache, q, table, lens, pre, P, workspace=ws, out=torch.full_like(q, 5.0)), clean)
