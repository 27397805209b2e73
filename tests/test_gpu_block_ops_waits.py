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
