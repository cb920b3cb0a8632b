"""Host side of the 8-bit cache and the eviction (no GPU): the reference arithmetic of the tests, refused calls, and the
calls SparseGQA makes of the library."""
import ctypes

import numpy as np
import pytest
import torch

from sparse_long_context_sgqa_b200 import api
from sparse_long_context_sgqa_b200 import binding as Bd
from sparse_long_context_sgqa_b200.binding import Params
from tests import _kv8_ref as R

PTR = 1 << 20  # an aligned address that no refused call follows


def test_reference_codes_match_torch_on_every_bf16_value():
    x = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16).to(torch.float32)
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    assert np.array_equal(R.e4m3_codes(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (225.0, 1.0), (0.0, 2.0 ** -100),
                                        (2.0 ** -120, 2.0 ** -100), (1.0, 2.0 ** -8), (3.0e38, 2.0 ** 120)])
def test_reference_scale(amax, scale):
    assert R.scale_of(amax) == scale


def _append(p=Params(), S=1, cap=64, pos0=0, n=8, k=PTR, v=PTR, tail=PTR, kv8=PTR, sc=PTR):
    return Bd._lib.sgqa_kv_append_q8(ctypes.byref(p.c()), S, cap, pos0, n, k, v, tail, kv8, sc, None)


@pytest.mark.parametrize("kw,code", [
    (dict(p=Params(block_size=4)), 2), (dict(p=Params(head_dim=128)), 2), (dict(S=0), 1), (dict(cap=60), 1),
    (dict(pos0=60), 1), (dict(pos0=-1), 1), (dict(n=-1), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(kv8=PTR + 8), 1),
    (dict(sc=None), 1), (dict(sc=PTR + 4), 1), (dict(n=7, tail=None), 1), (dict(pos0=3, n=5, tail=None), 1),
    (dict(k=PTR + 2), 1), (dict(pos0=1, n=1, tail=PTR + 8), 1), (dict(cap=1 << 31), 2)])
def test_append_refusals(kw, code):
    assert _append(**kw) == code
    assert Bd._lib.sgqa_last_error()


def test_append_of_nothing_is_accepted():
    assert _append(n=0, k=None, v=None, tail=None, kv8=None, sc=None) == 0


def _attn(p=Params(), S=1, q0=0, nq=1, q=PTR, cap=64, clen=64, kv8=PTR, sc=PTR, sel=PTR, cnt=PTR, gate=None, acc=None,
          out=PTR, ws=None, wsn=0):
    return Bd._lib.sgqa_sparse_attn_q8(ctypes.byref(p.c()), S, q0, nq, q, cap, clen, kv8, sc, sel, cnt, gate, acc, out,
                                       ws, wsn, None)


@pytest.mark.parametrize("kw,code", [
    (dict(p=Params(block_size=1)), 2), (dict(cap=68, clen=64), 1), (dict(clen=65), 1), (dict(q0=64), 1),
    (dict(q0=60, nq=4, clen=62), 1), (dict(q=None), 1), (dict(kv8=None), 1), (dict(kv8=PTR + 8), 1), (dict(sc=None), 1),
    (dict(sel=None), 1), (dict(cnt=None), 1), (dict(out=PTR + 8), 1), (dict(gate=PTR + 1), 1), (dict(acc=PTR + 4), 1)])
def test_attention_refusals(kw, code):
    assert _attn(**kw) == code


def test_attention_of_no_queries_is_accepted():
    assert _attn(nq=0, q=None) == 0


def test_forward_refuses_before_any_step():
    lib, p = Bd._lib, Params()
    args = [1, 0, 4, PTR, PTR, PTR, 64, PTR, PTR, PTR, PTR, PTR, PTR, PTR, None, PTR, PTR, PTR, None, None, PTR]
    # a missing tail, then a missing workspace
    bad = list(args)
    bad[11] = None
    assert lib.sgqa_forward_q8(ctypes.byref(p.c()), *bad, PTR, 1 << 40, None) == 1
    assert lib.sgqa_forward_q8(ctypes.byref(p.c()), *args, None, 0, None) == 3
    args[6] = 68
    assert lib.sgqa_forward_q8(ctypes.byref(p.c()), *args, PTR, 1 << 40, None) == 1


def _evict(p=Params(), S=1, cap=64, clen=64, keep=4, first=1, recent=1, acc=PTR, pos=None, known=0, evicted=0, acc_out=PTR,
           pos_out=PTR, arrays=(), ws=PTR, wsn=1 << 30):
    c = (Bd._CacheArray * max(1, len(arrays)))(*[Bd._CacheArray(*a) for a in arrays])
    return Bd._lib.sgqa_evict(ctypes.byref(p.c()), S, cap, clen, keep, first, recent, acc, pos, known, evicted, acc_out,
                              pos_out, c, len(arrays), ws, wsn, None)


@pytest.mark.parametrize("kw,code", [
    (dict(cap=60), 1), (dict(clen=65), 1), (dict(clen=-1), 1), (dict(keep=9), 1), (dict(keep=-1), 1), (dict(first=5), 1),
    (dict(recent=4), 1), (dict(first=-1), 1), (dict(recent=-1), 1), (dict(acc=None), 1), (dict(acc=PTR + 4), 1),
    (dict(acc_out=None), 1), (dict(pos_out=None), 1), (dict(known=2), 1), (dict(known=9, pos=PTR), 1),
    (dict(known=-1), 1), (dict(evicted=-1), 1), (dict(evicted=(1 << 31) - 8), 1), (dict(arrays=[(None, 16, 0)]), 1),
    (dict(arrays=[(PTR, 0, 0)]), 1), (dict(arrays=[(PTR, 16, 0)] * 9), 1), (dict(ws=None, wsn=0), 3),
    (dict(wsn=64), 3), (dict(ws=PTR + 64), 3), (dict(S=70000), 2)])
def test_evict_refusals(kw, code):
    assert _evict(**kw) == code


def test_evict_arrays_are_checked_by_the_binding():
    t = torch.zeros((1, 8, 4))
    with pytest.raises(ValueError):
        Bd.sgqa_evict(Params(), 1, 64, 64, 4, 0, 0, t, None, 0, 0, t, t, [t.transpose(1, 2)], None)
    with pytest.raises(ValueError):
        Bd.sgqa_evict(Params(), 1, 64, 64, 4, 0, 0, t, None, 0, 0, t, t, [torch.zeros(3, dtype=torch.uint8)], None)


def test_workspace_sizes():
    p = Params()
    assert Bd.sgqa_workspace_size_q8(p, 1, 8192, 131072) >= 8192 * 4 * 16384 * 4
    assert Bd.sgqa_workspace_size_q8(p, 2, 100, 512) >= Bd.sgqa_workspace_size_q8(p, 2, 1, 512)
    assert Bd.sgqa_evict_workspace_size(p, 2, 4096) > 2 * 512 * 8
    with pytest.raises(Bd.SgqaError):
        Bd.sgqa_workspace_size_q8(Params(block_size=1), 1, 8, 64)


def test_model_arguments():
    with pytest.raises(ValueError):
        api.SparseGQA(Params(), 1, 64, 8, "cpu", kv_dtype="int4")
    with pytest.raises(ValueError):
        api.SparseGQA(Params(), 1, 64, 8, "cpu", track_weights=True)
    with pytest.raises(ValueError):
        api.SparseGQA(Params(), 1, 60, 8, "cpu", kv_dtype="e4m3")
    with pytest.raises(ValueError):
        api.SparseGQA(Params(block_size=4), 1, 64, 8, "cpu", kv_dtype="e4m3")
    m = api.SparseGQA(Params(), 1, 64, 8, "cpu")
    q = torch.zeros((1, 1, 64, 192), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m.forward(0, q, None, None, None, None, None, k=q, v=q)
    with pytest.raises(ValueError):
        m.evict(64, 4)
    m = api.SparseGQA(Params(), 1, 64, 8, "cpu", kv_dtype="e4m3")
    with pytest.raises(ValueError):
        m.forward(0, q, None, None, None, None, None)
    with pytest.raises(ValueError):
        m.forward(0, q, None, None, None, None, None, cache_len=8, k=q, v=q)


def test_prefill_hands_every_chunk_its_own_rows(monkeypatch):
    calls = []

    def fake(p, S, q_pos0, nq, q, idx_q, idx_w, cap, kp, c, k, v, tail, kv8, kv_scale, merged, store, sel, cnt, out, ws,
             gate=None, acc=None, stream=None):
        assert k.is_contiguous() and v.is_contiguous() and k.shape[:2] == (S, nq)
        calls.append((q_pos0, k.clone(), v.clone(), acc))
        out.copy_(q)

    monkeypatch.setattr(api.Bd, "sgqa_forward_q8", fake)
    m = api.SparseGQA(Params(num_kv_groups=1, topk=4), 2, 64, 4, "cpu", kv_dtype="e4m3", track_weights=True)
    q = torch.randn(2, 10, 16, 3)
    k, v = torch.randn(2, 10, 1, 3), torch.randn(2, 10, 1, 3)
    out = torch.zeros_like(q)
    m.prefill(q, torch.zeros(2, 10, 1, 8, 64), torch.zeros(2, 10, 1, 8), out, q_pos0=5, k=k, v=v)
    assert [c[0] for c in calls] == [5, 9, 13]
    assert torch.equal(torch.cat([c[1] for c in calls], 1), k) and torch.equal(torch.cat([c[2] for c in calls], 1), v)
    assert all(c[3] is m.acc for c in calls) and torch.equal(out, q)


def test_evictions_are_counted_and_reset(monkeypatch):
    calls = []
    monkeypatch.setattr(api.Bd, "sgqa_evict", lambda p, S, cap, clen, keep, first, recent, acc, pos, known, evicted, *a,
                        **kw: calls.append((clen, keep, known, evicted, len(a[2]), len(kw["tail_arrays"]))))
    m = api.SparseGQA(Params(num_kv_groups=1), 1, 256, 8, "cpu", kv_dtype="e4m3", track_weights=True)
    assert m.evict(203, 20, 1, 2) == 163     # 25 complete blocks and 3 tokens
    assert m.evict(187, 20) == 163           # three more blocks came in
    assert calls == [(203, 20, 0, 0, 3, 2), (187, 20, 20, 5, 3, 2)]
    assert (m.evicted, m.pos_count) == (8, 20)
    m.acc.fill_(7)
    m.reset()
    assert (m.evicted, m.pos_count) == (0, 0) and not m.acc.any()


def test_reference_eviction_by_hand():
    # slots 0..5 with numbers 9 3 0 (known), then 3+7, 4+7, 5+7; protect number 0 and the last one (12)
    src, acc, num = R.evict(6, True, 4, 1, 1, [5, 1, 0, 5, 9, 2, 77], [9, 3, 0], 3, 7)
    # kept: 0 (protected, slot 2), 12 (protected, slot 5), weight 9 (slot 4), weight 5 with the smaller number 9 (slot 0)
    assert src == [0, 4, 2, 5, 6] and num == [9, 11, 0, 12]
    assert list(acc) == [5, 9, 0, 2, 77, 0, 0]


class _Tensor:
    """Looks like a CUDA tensor to the binding's checks."""
    def __init__(self, shape, dtype, device="cuda:1", contiguous=True, cuda=True):
        self.shape, self.dtype, self.device = shape, dtype, torch.device(device)
        self.is_cuda, self._c = cuda, contiguous

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self._c

    def data_ptr(self):
        return PTR

    def get_device(self):
        return self.device.index


def _append_tensors(**kw):
    t = dict(k=_Tensor((2, 3, 4, 192), torch.bfloat16), v=_Tensor((2, 3, 4, 192), torch.bfloat16),
             tail=_Tensor((2, 2, 8, 4, 192), torch.bfloat16), kv8=_Tensor((2, 8, 4, 2, 8, 192), torch.uint8),
             kv_scale=_Tensor((2, 8, 4, 2), torch.float32))
    t.update(kw)
    return t


@pytest.mark.parametrize("kw", [
    dict(k=_Tensor((2, 2, 4, 192), torch.bfloat16)), dict(v=_Tensor((2, 3, 4, 192), torch.float32)),
    dict(tail=_Tensor((2, 2, 8, 4, 192), torch.bfloat16, contiguous=False)),
    dict(kv8=_Tensor((2, 8, 4, 2, 8, 192), torch.uint8, cuda=False)), dict(kv_scale=_Tensor((2, 8, 4), torch.float32))])
def test_tensors_that_do_not_fit_are_refused(kw):
    with pytest.raises(ValueError):
        Bd.sgqa_kv_append_q8(Params(), 2, 64, 0, 3, **_append_tensors(**kw))


def test_calls_run_on_the_tensors_device(monkeypatch):
    class Guard:
        def __init__(self, dev):
            log.append(("enter", dev))

        def __enter__(self):
            pass

        def __exit__(self, *a):
            log.append("exit")

    class Stream:
        cuda_stream, device = 77, torch.device("cuda:1")

    log = []
    monkeypatch.setattr(Bd.torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(Bd.torch.cuda, "device", Guard)
    monkeypatch.setattr(Bd, "_raw_stream", lambda index: 76 + index)
    monkeypatch.setattr(Bd._lib, "sgqa_kv_append_q8", lambda *a: log.append(("call", a[-1])) or 0)
    Bd.sgqa_kv_append_q8(Params(), 2, 64, 0, 3, **_append_tensors())
    assert log == [("enter", 1), ("call", 77), "exit"]
    monkeypatch.setattr(Bd.torch.cuda, "current_device", lambda: 1)
    log.clear()
    Bd.sgqa_kv_append_q8(Params(), 2, 64, 0, 3, **_append_tensors())
    assert log == [("call", 77)]
    other = Stream()
    other.device = torch.device("cuda:0")
    with pytest.raises(ValueError):
        Bd.sgqa_kv_append_q8(Params(), 2, 64, 0, 3, stream=other, **_append_tensors())


@pytest.mark.parametrize("name", ["k", "v", "tail", "kv_scale"])
def test_tensors_of_a_call_share_a_device(monkeypatch, name):
    monkeypatch.setattr(Bd._lib, "sgqa_kv_append_q8", lambda *a: pytest.fail("called"))
    t = _append_tensors()
    t[name].device = torch.device("cuda:0")
    with pytest.raises(ValueError, match=name):
        Bd.sgqa_kv_append_q8(Params(), 2, 64, 0, 3, **t)


@pytest.mark.parametrize("which", ["arrays", "tail_arrays", "pos_out", "workspace"])
def test_evicted_arrays_share_a_device(monkeypatch, which):
    monkeypatch.setattr(Bd._lib, "sgqa_evict", lambda *a: pytest.fail("called"))
    t = {n: _Tensor((2, 8), torch.int32 if n.startswith("pos") else torch.int64) for n in ("acc", "pos", "acc_out", "pos_out")}
    one, tail, ws = _Tensor((2, 8, 16), torch.uint8), _Tensor((2, 64, 4), torch.uint8), _Tensor((4096,), torch.uint8)
    for x in (one, tail):
        x.nbytes = x.numel()
    {"arrays": one, "tail_arrays": tail, "pos_out": t["pos_out"], "workspace": ws}[which].device = torch.device("cuda:0")
    with pytest.raises(ValueError):
        Bd.sgqa_evict(Params(), 2, 64, 40, 2, 0, 0, t["acc"], t["pos"], 0, 0, t["acc_out"], t["pos_out"], [one], ws,
                      tail_arrays=[tail])


def test_evict_takes_the_tracked_weights_only(monkeypatch):
    # with others the tracked ones would keep the blocks' old slots, and a later eviction would go by them
    monkeypatch.setattr(Bd, "sgqa_evict", lambda *a, **kw: pytest.fail("called"))
    m = api.SparseGQA(Params(num_kv_groups=1), 1, 64, 8, "cpu", kv_dtype="e4m3", track_weights=True)
    with pytest.raises(ValueError):
        m.evict(64, 4, acc=torch.ones((1, 8), dtype=torch.int64))
    assert (m.evicted, m.pos_count) == (0, 0)


def test_evict_allocates_on_the_calls_stream(monkeypatch):
    class On:
        def __init__(self, st):
            self.st = st

        def __enter__(self):
            cur.append(self.st)

        def __exit__(self, *a):
            cur.pop()

    cur, seen = [], []
    monkeypatch.setattr(api.torch.cuda, "stream", On)
    monkeypatch.setattr(Bd, "alloc_evict_workspace", lambda *a: seen.append(list(cur)) or "ws")
    monkeypatch.setattr(Bd, "sgqa_evict", lambda *a, **kw: seen.append(kw["stream"]))
    m = api.SparseGQA(Params(num_kv_groups=1), 1, 64, 8, "cpu", kv_dtype="e4m3", track_weights=True)
    m.evict(64, 4, stream="side")
    assert seen == [["side"], "side"]


@pytest.mark.parametrize("missing", ["k", "v"])
def test_prefill_refuses_half_of_the_rows(monkeypatch, missing):
    monkeypatch.setattr(Bd, "sgqa_forward_q8", lambda *a, **kw: pytest.fail("called"))
    m = api.SparseGQA(Params(num_kv_groups=1, topk=4), 1, 64, 8, "cpu", kv_dtype="e4m3")
    q = torch.zeros((1, 4, 16, 192), dtype=torch.bfloat16)
    rows = {n: torch.zeros((1, 4, 1, 192), dtype=torch.bfloat16) for n in ("k", "v") if n != missing}
    with pytest.raises(ValueError, match="K/V rows"):
        m.prefill(q, torch.zeros((1, 4, 1, 8, 128)), torch.zeros((1, 4, 1, 8)), torch.empty_like(q), **rows)
