"""What a rank of the KV-group sharding hands its model with a call: its own slices of the gate and of the rows that the
8-bit cache takes (no GPU, no process group: gather=False)."""
import types

import pytest
import torch

from sparse_long_context_sgqa_b200 import sharding as Sh
from sparse_long_context_sgqa_b200.binding import Params

S, N, G, HG, D, H, DI = 2, 3, 4, 16, 6, 8, 4


def layer(world, rank, **model):
    calls = []
    m = types.SimpleNamespace(kp=torch.zeros(S, 16, DI), c=torch.zeros(S, 16, DI), forward=lambda *a, **kw: calls.append(kw), **model)
    return Sh.GroupShardedSGQA(Params(num_kv_groups=G, topk=2), world, rank, lambda p: m), m, calls


def queries():
    return torch.randn(S, N, G * HG, D), torch.randn(S, N, G, H, DI), torch.randn(S, N, G, H)


@pytest.mark.parametrize("world,rank", [(1, 0), (2, 1), (4, 2)])
def test_gate_of_the_ranks_heads(world, rank):
    sh, _, calls = layer(world, rank)
    gate = torch.randn(S, N, G * HG)
    per = G * HG // world
    own = gate[:, :, rank * per:(rank + 1) * per]
    for given in (gate, own.contiguous()):  # all heads' logits, or the rank's own
        sh.forward(0, *queries(), gather=False, gate=given)
        assert torch.equal(calls[-1]["gate"], own) and calls[-1]["gate"].is_contiguous()
    with pytest.raises(ValueError, match="gate"):
        sh.forward(0, *queries(), gather=False, gate=gate[:, :, 1:])
    sh.forward(0, *queries(), gather=False, gate=None, stream="side")
    assert calls[-1] == dict(gate=None, stream="side")


@pytest.mark.parametrize("world,rank", [(1, 0), (2, 1), (4, 3)])
def test_rows_of_the_8bit_cache(world, rank):
    sh, m, calls = layer(world, rank, kv_dtype="e4m3")
    kp, c, k, v = torch.randn(S, 9, DI), torch.randn(S, 9, DI), torch.randn(S, N, G, D), torch.randn(S, N, G, D)
    sh.load_cache(kp, c)
    assert torch.equal(m.kp[:, :9], kp) and torch.equal(m.c[:, :9], c) and not m.kp[:, 9:].any()
    per = G // world
    sh.forward(0, *queries(), gather=False, k=k, v=v)
    for name, t in (("k", k), ("v", v)):
        assert torch.equal(calls[-1][name], t[:, :, rank * per:(rank + 1) * per]) and calls[-1][name].is_contiguous()
    # the rows come with the calls: there is no BF16 cache to load
    with pytest.raises(ValueError, match="8-bit"):
        sh.load_cache(kp, c, k, v)


def test_bf16_caches_are_loaded_whole():
    sh, m, _ = layer(2, 1, kv_dtype="bf16", k=torch.zeros(S, 16, 2, D), v=torch.zeros(S, 16, 2, D))
    kp, c, k, v = torch.randn(S, 9, DI), torch.randn(S, 9, DI), torch.randn(S, 9, G, D), torch.randn(S, 9, G, D)
    with pytest.raises(ValueError, match="k and v"):
        sh.load_cache(kp, c)
    sh.load_cache(kp, c, k, v)
    assert torch.equal(m.k[:, :9], k[:, :, 2:]) and torch.equal(m.v[:, :9], v[:, :, 2:])
