"""Host side of the 8-bit cache, of eviction and of what they share with the other calls, at their edges (no GPU)."""
import copy
import dataclasses
import pickle

import pytest

from sparse_long_context_sgqa_b200 import api
from sparse_long_context_sgqa_b200 import binding as Bd
from sparse_long_context_sgqa_b200.binding import Params


@pytest.mark.parametrize("size", [Bd.sgqa_workspace_size, Bd.sgqa_workspace_size_q8])
@pytest.mark.parametrize("S,G", [(1, 1), (2, 2), (1, 4), (16, 4), (5, 3)])
def test_a_workspace_serves_calls_of_fewer_queries(size, S, G):
    # a model's workspace is made for its chunk and serves every shorter call; few queries are split further than many
    p = Params(num_kv_groups=G, topk=9)
    for ctx in (512, 40_000, 300_000):
        sizes = [size(p, S, n, ctx) for n in (1, 2, 7, 16, 31, 32, 33, 40, 64, 200, 512)]
        assert sizes == sorted(sizes), ctx


def test_reset_clears_the_weights_on_the_calls_stream(monkeypatch):
    # the calls before it may still be adding weights on that stream
    class On:
        def __init__(self, st):
            self.st = st

        def __enter__(self):
            cur.append(self.st)

        def __exit__(self, *a):
            cur.pop()

    cur, seen = [], []
    m = api.SparseGQA(Params(num_kv_groups=1), 1, 64, 8, "cpu", kv_dtype="e4m3", track_weights=True)
    m.acc = type("Acc", (), {"zero_": lambda self: seen.append(list(cur))})()
    monkeypatch.setattr(api.torch.cuda, "stream", On)
    m.reset(stream="side")
    m.reset()
    assert seen == [["side"], []]


def test_params_hold_their_fields_only():
    # what a call keeps beside them is not one of them: copies by field, also after a call
    p = Params(num_kv_groups=2, topk=7)
    Bd.sgqa_workspace_size(p, 1, 1, 64)
    assert Params(**vars(p)) == p and list(vars(p)) == [f.name for f in dataclasses.fields(Params)]
    for q in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p)), dataclasses.replace(p, topk=9)):
        assert q.c().num_kv_groups == 2 and q.c().topk == q.topk
        q.topk = 11
        assert q.c().topk == 11 and p.c().topk == 7
