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
    binding.lib()
    calls = []

    class Recorder:
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
