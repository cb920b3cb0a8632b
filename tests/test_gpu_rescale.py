"""Prefill attention whose running maximum keeps growing along the selection: every tile rescales the accumulated output,
which must hold the previous tile's product by then.  Keys grow with their block, so that later blocks outweigh all
earlier ones by large factors; results are compared with FP64 attention over the same selection."""
import math

import numpy as np
import pytest
import torch

from sparse_long_context_sgqa_b200.binding import Params

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [8, 2])
def test_growing_scores_rescale_every_tile(cuda_device, block):
    from sparse_long_context_sgqa_b200 import binding as Bd
    g = torch.Generator()
    g.manual_seed(3)
    G, D, H, nq, q0, k = 2, 192, 16, 256, 4096, 256
    n = q0 + nq
    q = torch.randn((1, nq, G * H, D), generator=g)
    q[..., 0] = 8.0
    K = torch.randn((1, n, G, D), generator=g) * 0.3
    V = torch.randn((1, n, G, D), generator=g)
    # the first coordinate climbs by about 7 powers of two of weight per 64 selected tokens
    K[..., 0] = (torch.arange(n).float() / 64 * 7 * math.log(2) * math.sqrt(D) / 8 * (k * block / q0))[None, :, None]
    q, K, V = q.to(torch.bfloat16), K.to(torch.bfloat16), V.to(torch.bfloat16)
    sel = torch.stack([torch.stack([torch.randperm(q0 // block, generator=g)[:k].sort().values for _ in range(G)])
                       for _ in range(nq)])[None].int()
    cnt = torch.full((1, nq, G), k, dtype=torch.int32)
    dev = cuda_device
    p = Params(num_kv_groups=G, block_size=block, topk=k)
    ws = Bd.alloc_workspace(p, 1, nq, n, dev)
    a = [x.to(dev) for x in (q, K, V, sel, cnt)]
    outs = []
    for _ in range(12):
        out = torch.zeros_like(a[0])
        Bd.sgqa_sparse_attn(p, 1, q0, nq, a[0], n, n, a[1], a[2], a[3], a[4], out, ws)
        Bd.sgqa_check()
        outs.append(out)
    # exact: FP64 over each query's tokens, in one masked product
    t = torch.arange(q0, n, device=dev)
    ref = torch.empty((nq, G * H, D), dtype=torch.float64, device=dev)
    for gg in range(G):
        mask = torch.zeros((nq, n // block), dtype=torch.bool, device=dev).scatter_(1, a[3][0, :, gg].long(), True)
        mask[torch.arange(nq, device=dev), t // block] = True
        seen = mask.repeat_interleave(block, 1) & (torch.arange(n, device=dev) <= t[:, None])
        s = torch.einsum("qhd,td->qht", a[0][0, :, gg * H:(gg + 1) * H].double(), a[1][0, :, gg].double()) / math.sqrt(D)
        w = torch.softmax(s.masked_fill(~seen[:, None], -math.inf), -1)
        ref[:, gg * H:(gg + 1) * H] = torch.einsum("qht,td->qhd", w, a[2][0, :, gg].double())
    for out in outs:
        assert float((out[0].double() - ref).abs().max()) <= 2e-2
    assert all(np.array_equal(o.cpu().view(torch.int16).numpy(), outs[0].cpu().view(torch.int16).numpy()) for o in outs)
