"""Host side of the 8-bit cache, of eviction and of what they share with the other calls, at their edges (no GPU)."""
import copy
import dataclasses
import pickle

import pytest
import torch

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


@pytest.mark.parametrize("lo_scale,exact_from,off", [(16.0, 2.0 ** -13.8, 2.0 ** -21.8), (1.0, 2.0 ** -9.8, 2.0 ** -17.8)])
def test_two_e4m3_values_carry_a_query_value(lo_scale, exact_from, off):
    # every BF16 value under the scale that brings its row's largest into (224, 448], split as the kernels split it: few
    # queries with the second value scaled by 16, many without.  Bounds as sgqa.h states them, for the least favourable
    # largest value, 225 (the first BF16 value above 224).
    x = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16).double()
    x = x[x <= 448]
    code = lambda t: t.float().to(torch.float8_e4m3fn).double()  # noqa: E731
    hi = code(x)
    wrong = (hi + code((x - hi) * lo_scale) / lo_scale - x).abs()
    assert not wrong[x >= 225 * exact_from].any()
    assert wrong.max() <= 225 * off
    assert wrong.max() >= 0.98 * 225 * off and wrong[x < 225 * exact_from].any()  # the bounds are tight


def _tokens(m, monkeypatch):
    """m.forward and m.evict without a GPU: forward(position, tokens)."""
    monkeypatch.setattr(Bd, "sgqa_forward_q8", lambda *a, **kw: None)
    monkeypatch.setattr(Bd, "sgqa_evict", lambda *a, **kw: None)

    def forward(pos, n):
        x = torch.zeros((1, n, 1, 192), dtype=torch.bfloat16)
        m.forward(pos, x, None, None, None, None, None, k=x, v=x)
    return forward


def test_tokens_taken_back_need_the_rows_of_their_block(monkeypatch):
    # `tail` holds the rows of the block that the last call ended in: a call that begins inside another one would quantise
    # that block from rows of a different block
    m = api.SparseGQA(Params(num_kv_groups=1), 1, 256, 8, "cpu", kv_dtype="e4m3", track_weights=True)
    forward = _tokens(m, monkeypatch)
    forward(13, 3)                       # a cache filled by hand: nothing is known of tail
    assert m.length == 16
    forward(16, 7)                       # drafts, of which three stay
    forward(19, 7)                       # 19 .. 25: into the next block
    for pos in (20, 23, 27, 29):         # in the block before, and behind the cache's end
        with pytest.raises(ValueError, match="tail"):
            forward(pos, 1)
        assert m.length == 26
    with pytest.raises(ValueError, match="tail"):
        m.evict(21, 1)
    forward(25, 1)                       # inside the block that tail holds
    forward(16, 9)                       # a whole block again, from its first row
    assert m.evict(24, 2) == 16          # (whole blocks need no rows)
    forward(16, 3)
    assert m.evict(19, 1) == 11
    forward(11, 1)
    m.length = None                      # filled outside these calls
    forward(21, 1)
    m.reset()
    assert m.length is None


def test_a_call_that_failed_leaves_the_length_unknown(monkeypatch):
    m = api.SparseGQA(Params(num_kv_groups=1), 1, 256, 8, "cpu", kv_dtype="e4m3")
    forward = _tokens(m, monkeypatch)
    forward(0, 5)

    def fails(*a, **kw):
        raise Bd.SgqaError(2, "")
    monkeypatch.setattr(Bd, "sgqa_forward_q8", fails)
    with pytest.raises(Bd.SgqaError):
        forward(5, 1)
    assert m.length is None


def test_bf16_caches_take_tokens_back_anywhere(monkeypatch):
    monkeypatch.setattr(Bd, "sgqa_forward", lambda *a, **kw: None)
    m = api.SparseGQA(Params(num_kv_groups=1), 1, 256, 8, "cpu")
    x = torch.zeros((1, 7, 16, 192), dtype=torch.bfloat16)
    for pos in (19, 21, 3, 40):
        m.forward(pos, x, None, None, None, None, None)
