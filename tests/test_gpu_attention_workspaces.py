"""Workspaces that attention calls without one keep: one per device and stream for all caches."""
import threading

import pytest
import torch

from int4_routed_expert_prerouter_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def layers(n, B, H=2, G=4, D=128, page=64, W=3):
    """Caches of a model's layers, filled, with a call's arguments for each."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(n + B)
    table = torch.arange(B * W, device=DEV, dtype=torch.int32).view(B, W)
    lens = (torch.arange(B, device=DEV) * 37 % (W * page) + 1).int()
    cu = (torch.arange(B + 1, device=DEV) * W * page).int()
    out = []
    for _ in range(n):
        c = binding.KVCache(B * W, page, H, D, 4, device=DEV)
        k, v = torch.randn(2, B * W * page, H, D, generator=gen, device=DEV).half()
        binding.kv_append(c, k, v, table, torch.zeros(B, dtype=torch.int32, device=DEV), cu)
        q = torch.randn(B, H * G, D, generator=gen, device=DEV).half()
        out.append((c, q, table, lens, table[0].contiguous(), 100))
    return out


def test_many_caches_on_one_stream_keep_one_workspace():
    binding.release_workspaces()
    calls = layers(40, 12)
    ws = torch.empty(binding.attn_workspace_bytes(calls[0][0], 12, 8), dtype=torch.uint8, device=DEV)
    want = [binding.attn_decode(*a, workspace=ws) for a in calls]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    got = [binding.attn_decode(*a) for a in calls]
    kept = torch.cuda.memory_allocated() - before - sum(g.numel() * 2 for g in got)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ws.numel() <= kept <= ws.numel() + (1 << 20)
    # a larger batch takes the smaller one's place, and all of it is given back on demand
    big = layers(2, 60)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    got = [binding.attn_decode(*a) for a in big + calls[:3]]
    need = binding.attn_workspace_bytes(big[0][0], 60, 8)
    grown = torch.cuda.memory_allocated() - before - sum(g.numel() * 2 for g in got)
    assert abs(grown - (need - ws.numel())) <= 1 << 20
    assert all(torch.equal(a, b) for a, b in zip(got[2:], want))
    held = torch.cuda.memory_allocated()
    binding.release_workspaces()
    assert held - torch.cuda.memory_allocated() >= need
    assert torch.equal(binding.attn_decode(*calls[5]), want[5])


def test_release_beside_calls_under_way_on_two_streams():
    calls = layers(6, 20)
    want = [binding.attn_decode(*a) for a in calls]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(120):
        with torch.cuda.stream(streams[i % 2]):
            got.append(binding.attn_decode(*calls[i % 6]))
            junk = torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)      # takes what was given back
            del junk
        if i % 7 == 0:
            binding.release_workspaces()
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 6]) for i, g in enumerate(got))


def test_threads_with_caches_of_their_own_on_one_stream():
    calls = layers(6, 16)
    want = [binding.attn_decode(*a) for a in calls]
    torch.cuda.synchronize()
    outs = [[] for _ in calls]

    def work(i):
        for _ in range(60):
            outs[i].append(binding.attn_decode(*calls[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i, got in enumerate(outs):
        assert len(got) == 60 and all(torch.equal(o, want[i]) for o in got)
