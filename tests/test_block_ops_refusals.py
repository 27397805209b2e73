"""Outputs and counts that the projection, cache and attention calls have to refuse before anything
is launched: what the binding hands to the C calls, checked without a GPU."""
import ctypes as C

import pytest
import torch

from int4_routed_expert_prerouter_gb300 import binding, build

A = C.c_void_p(1 << 20)          # an aligned address that is never read


class OnGpu(torch.Tensor):
    """A host tensor that says it lies on a GPU: enough for the binding's checks."""
    is_cuda = True

    def get_device(self):
        return 0


def on_gpu(t):
    return t.as_subclass(OnGpu)


@pytest.fixture
def handed(monkeypatch):
    """Records the arguments of each C call instead of making it."""
    build.build()
    real, calls = binding.lib(), []

    class Recorder:
        edge0_status_string = real.edge0_status_string

        def __getattr__(self, name):
            def call(*args):
                calls.append((name, args))
                return 0
            return call

    monkeypatch.setattr(binding, "_lib", Recorder())
    monkeypatch.setattr(binding, "_raw_stream", lambda index, stream: 0)
    return calls


@pytest.mark.parametrize("B,n_out", [(2, 16), (8, 48), (3, 1)])
def test_projection_outputs_that_overlap_are_refused(handed, B, n_out):
    real = C.CDLL(build.LIB)
    packed = on_gpu(torch.zeros((n_out + 15) // 16 * 576, dtype=torch.uint8))
    x = on_gpu(torch.zeros(B, 64, dtype=torch.float16))
    real.edge0_q4_linear.argtypes = [C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_longlong, C.c_int, C.c_void_p, C.c_longlong,
                                     C.c_void_p]
    storage = torch.zeros(B * n_out, dtype=torch.float16)
    expanded = storage[:n_out].view(1, n_out).expand(B, n_out)
    short = storage.as_strided((B, n_out), (n_out - 1, 1))
    for y in (expanded, short):
        handed.clear()
        binding._q4_linear(packed, n_out, x, on_gpu(y), 0, None)
        (_, args), = handed
        ldy = args[7]
        assert ldy == y.stride(0)
        assert real.edge0_q4_linear(A, n_out, 64, A, 64, B, A, ldy, None) == binding.EDGE0_EINVAL
    # rows side by side, and a single row whatever its stride says
    binding._q4_linear(packed, n_out, x, on_gpu(storage.view(B, n_out)), 0, None)
    assert handed[-1][1][7] == n_out
    binding._q4_linear(packed, n_out, x[:1], on_gpu(storage.as_strided((1, n_out), (0, 1))), 0, None)
    assert handed[-1][1][7] >= n_out


def meta(*shape, dtype):
    """A tensor of any size without memory."""
    return on_gpu(torch.empty(*shape, dtype=dtype, device="meta"))


def cache(page=4096):
    c = binding.KVCache.__new__(binding.KVCache)
    c.n_pages, c.page_tokens, c.n_kv_heads, c.head_dim, c.bits = 8, page, 2, 64, 4
    c._index, c._desc, c._status, c.device = 0, None, 0, torch.device("cpu")
    return c


def test_counts_that_do_not_fit_an_int_are_refused(handed):
    """2^32 + n would arrive as n."""
    big = 1 << 32
    i32 = torch.int32
    q = on_gpu(torch.zeros(1, 4, 64, dtype=torch.float16))
    one, lens = on_gpu(torch.zeros(1, 1, dtype=i32)), on_gpu(torch.zeros(1, dtype=i32))
    k = on_gpu(torch.zeros(1, 2, 64, dtype=torch.float16))
    tall = on_gpu(torch.zeros(1, 2, 64, dtype=torch.float16).expand(big + 1, 2, 64))
    cu = on_gpu(torch.zeros(2, dtype=i32))
    calls = [lambda: binding._attn_decode(cache(), q, one, lens, meta(big // 4096 + 1, dtype=i32), big + 5, None, q.clone(), k, None),
             lambda: binding._attn_decode(cache(), q, one, lens, meta((1 << 30) // 4096 + 1, dtype=i32), (1 << 30) + 1, None, q.clone(), k, None),
             lambda: binding._attn_decode(cache(), q, meta(1, big + 1, dtype=i32), lens, None, 0, None, q.clone(), k, None),
             lambda: binding._kv_append(cache(), k, k, meta(1, big + 1, dtype=i32), lens, None, None),
             lambda: binding._kv_append(cache(), tall, tall, one, lens, cu, None),
             lambda: binding._kv_append(cache(), k, k, meta(big + 1, 1, dtype=i32), meta(big + 1, dtype=i32), meta(big + 2, dtype=i32), None),
             lambda: binding._kv_read(cache(), one, lens, cu, big + 1, k, k, None),
             lambda: binding._q4_linear(meta((big + 16) // 16 * 576, dtype=torch.uint8), big + 16, meta(1, 64, dtype=torch.float16), None, 0, None),
             lambda: binding._q4_linear(meta((1 << 28) // 64 * 576 + 576, dtype=torch.uint8), 16, meta(1, (1 << 28) + 64, dtype=torch.float16), None, 0, None)]
    for i, call in enumerate(calls):
        with pytest.raises(binding.Edge0Error) as e:
            call()
        assert e.value.code == binding.EDGE0_EUNSUPPORTED, i
    assert not handed
