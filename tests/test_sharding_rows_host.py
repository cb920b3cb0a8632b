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
