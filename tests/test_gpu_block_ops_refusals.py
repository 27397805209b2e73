"""Calls of the projection, cache and attention operators that are refused on a GPU machine as well:
nothing is launched, and memory beside the buffers stays as it was."""
import pytest
import torch

from int4_routed_expert_prerouter_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("B", [2, 8, 40])
def test_projection_outputs_that_overlap_are_refused(B):
    n_out = 48
    packed = torch.zeros(3 * 576, dtype=torch.uint8, device=DEV)
    x = torch.zeros(B, 64, dtype=torch.float16, device=DEV)
    memory = torch.full((4 * B * n_out,), 7.0, dtype=torch.float16, device=DEV)
    for y in (memory[:n_out].view(1, n_out).expand(B, n_out), memory.as_strided((B, n_out), (n_out - 1, 1))):
        with pytest.raises(binding.Edge0Error) as e:
            binding.q4_linear(packed, n_out, x, y=y)
        assert e.value.code == binding.EDGE0_EINVAL
    torch.cuda.synchronize()
    assert (memory == 7).all()
