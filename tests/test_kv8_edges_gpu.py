"""The 8-bit cache's operators at their edges: wide contexts, scores that underflow, calls that gave up, lists out of order,
other scales, sinks.  Tolerances: tests/_kv8_ref.py and tests/test_kv8_gpu.py, unless a test derives its own.
"""
import ctypes
import math
import threading

import numpy as np
import pytest
import torch

from sparse_long_context_sgqa_b200.binding import Params
from tests import _kv8_ref as R
from tests import test_kv8_gpu as T

pytestmark = pytest.mark.gpu
D, HG, B = R.D, R.HG, R.B


@pytest.fixture(scope="module")
def Bd():
    from sparse_long_context_sgqa_b200 import binding
    return binding


# ------------------ wide id ranges
@pytest.mark.parametrize("weights", [False, True])
def test_union_of_a_context_too_wide_for_a_bitmap(Bd, cuda_device, weights):
    # 11.8 M tokens: a unit's union is planned by sorting.  Short lists, so that unions end inside a tile, and a workspace
    # of ones, which an earlier call may well leave there.
    H, nq, k, dev = 1_480_000, 40, 24, cuda_device
    q0, blocks, g = 8 * H + 3, H + 7, T.gen(11)
    used = torch.cat([torch.tensor([0, H - 1]), torch.randperm(H - 2, generator=g)[:58] + 1]).sort().values.unique()
    n = len(used)
    idx = torch.cat([used, torch.arange(H, blocks)])
    codes = (torch.randn((len(idx), 1, 2, B, D), generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    small_sc = torch.exp2(torch.randint(-9, -6, (len(idx), 1, 2), generator=g).float())
    kv8 = torch.empty((1, blocks, 1, 2, B, D), dtype=torch.uint8, device=dev)
    sc = torch.ones((1, blocks, 1, 2), device=dev)
    kv8[0, idx.to(dev)], sc[0, idx.to(dev)] = codes.to(dev), small_sc.to(dev)
    q = torch.randn((1, nq, HG, D), generator=g).to(torch.bfloat16)
    sel = torch.full((1, nq, 1, k), -1, dtype=torch.int32)
    cnt = torch.zeros((1, nq, 1), dtype=torch.int32)
    small_sel = sel.clone()
    for i in range(nq):
        c = int(torch.randint(0, 6, (1,), generator=g))
        pick = torch.randperm(n, generator=g)[:c].sort().values
        sel[0, i, 0, :c], small_sel[0, i, 0, :c], cnt[0, i, 0] = used[pick].int(), pick.int(), c
    p = Params(num_kv_groups=1, topk=k)
    ws = Bd.alloc_workspace_q8(p, 1, nq, q0 + nq, dev)
    ws.fill_(255)
    out = torch.zeros_like(q, device=dev)
    acc = torch.zeros((1, blocks), dtype=torch.int64, device=dev) if weights else None
    Bd.sgqa_sparse_attn_q8(p, 1, q0, nq, q.to(dev), 8 * blocks, q0 + nq, kv8, sc, sel.to(dev), cnt.to(dev), out, ws, acc=acc)
    Bd.sgqa_check()
    # the reference over the blocks that occur, renumbered in order
    ref, tol, wts = R.attention(q.double().numpy(), R.codes_to_values(codes)[None], small_sc.double().numpy()[None],
                                small_sel.numpy(), cnt.numpy(), 8 * n + 3)
    R.check_out(out, ref, tol)
    if weights:
        T.check_weights(acc[:, idx.to(dev)], 0, wts, 2 * nq)
        assert int(acc.sum()) == int(acc[:, idx.to(dev)].sum())


# ------------------ scores that underflow
@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -60])
def test_zero_heads_against_zero_keys(Bd, cuda_device, nq, size):
    # a head of zeros (or far below the others) at a current block of zero keys, as padding leaves them: the product of
    # both scales is below FP32's range, every score is 0, and the tokens behind the query stay out
    c = T.make_attn(2, 2, nq, 1002, 50, cuda_device)
    c["q"][:, :, 3:7] = size
    c["q"][:, :, 19] = -size
    first, last = 1002 // B, (1002 + nq - 1) // B
    c["kv8"][:, first:last + 1, :, 0] = 0
    c["sc"][:, first:last + 1, :, 0] = 2.0 ** -100
    ref, tol, weights = T.reference(c)
    acc = torch.zeros((2, c["cap"] // B), dtype=torch.int64, device=cuda_device)
    T.check_attn(c, T.run_attn(Bd, c, acc=acc), ref, tol)
    T.check_weights(acc, 0, weights, nq * 2 * 2)


# ------------------ calls that gave up
def gave_up(Bd, cuda_device, nq, limits):
    c = T.make_attn(2, 4, nq, 3000, 256, cuda_device)
    p = Params(num_kv_groups=4, topk=256)
    ws = Bd.alloc_workspace_q8(p, 2, nq, 3000 + nq, cuda_device)
    acc = torch.zeros((2, c["cap"] // B), dtype=torch.int64, device=cuda_device)
    T.run_attn(Bd, c, acc=acc, ws=ws)
    once, failed = acc.clone(), 0
    for ns in limits:
        ws.zero_()  # (stale sums and log-sums of 0 would count as large weights)
        before = acc.clone()
        try:
            Bd.sgqa_set_wait_limit_ns(ns)
            T.run_attn(Bd, c, acc=acc, ws=ws)
        except Bd.SgqaError as e:
            assert e.code == 5
            failed += 1
        finally:
            Bd.sgqa_set_wait_limit_ns(0)
        added = acc - before
        assert (added >= 0).all() and (added <= once).all(), (ns, int(added.min()), int((added - once).max()))
    assert failed >= 1
    before = acc.clone()
    T.run_attn(Bd, c, acc=acc, ws=ws)
    assert torch.equal(acc - before, once)


def test_few_queries_that_gave_up_add_no_weights_of_their_own(Bd, cuda_device):
    gave_up(Bd, cuda_device, 1, [1, 1, 500, 1000, 2000, 4000, 5000, 6000, 7000, 8000, 10000])


# ------------------ calls that gave up, many queries
def test_many_queries_that_gave_up_add_no_weights_of_their_own(Bd, cuda_device):
    gave_up(Bd, cuda_device, 64, [1, 1, 500, 1000, 2000, 4000, 5000, 6000, 7000, 8000, 10000])


# ------------------ a reference that moves in every tile
@pytest.mark.parametrize("nq", [1, 70])
def test_scores_that_grow_along_the_list(Bd, cuda_device, nq):
    # the first coordinate climbs by about 2^14 of weight per eight selected blocks: every tile's weights are computed twice
    c = T.make_attn(1, 2, nq, 6000, 200, cuda_device, sigma=0.3, spread=0)
    blocks = c["cap"] // B
    c["q"][..., 0] = 8.0
    c["kv8"][:, :, :, 0, :, 0] = torch.tensor(448.0).to(torch.float8_e4m3fn).view(torch.uint8).to(cuda_device)
    step = 14 * math.log(2) * math.sqrt(D) / (8 * 448) * 200 / (8 * 750)
    c["sc"][:, :, :, 0] = (1 + torch.arange(blocks, device=cuda_device))[None, :, None] * step
    ref, tol, weights = T.reference(c)
    outs = []
    for _ in range(6):
        acc = torch.zeros((1, blocks), dtype=torch.int64, device=cuda_device)
        outs.append((T.run_attn(Bd, c, acc=acc), acc))
    T.check_attn(c, outs[0][0], ref, tol)
    # Weights at scores of up to 480 (powers of two): a query value other than the row's largest, 8, is off by up to
    # 2^-17.8 of that (few queries: 2^-21.8), a score by that times its key; FP32 adds 2^-15 at magnitude 30, so 2^-11.
    # A weight takes a score's error and its row's sum the largest of them: twice.
    keys = (R.codes_to_values(c["kv8"])[0, :, :, 0, :, 1:] * c["sc"][0, :, :, 0].cpu().double().numpy()[:, :, None, None])
    far = 8 * 2.0 ** (-21.8 if nq <= 32 else -17.8) * np.abs(keys).sum(-1).max() / math.sqrt(D)
    rel = math.expm1(2 * (far + 2.0 ** -11 * math.log(2)))
    off = np.abs(outs[0][1].cpu().double().numpy() * R.UNIT - weights)
    assert rel < 0.1 and (off <= rel * weights + nq * 2 * 2 * R.UNIT).all()
    assert all(torch.equal(o.view(torch.int16), outs[0][0].view(torch.int16)) and torch.equal(a, outs[0][1]) for o, a in outs)


# ------------------ calls of several host threads
def test_threads_with_contexts_of_different_length(Bd, cuda_device):
    # the planner's shared memory goes by the context; one thread's calls must not take it from another's
    dev, g, nq, k = cuda_device, T.gen(4), 40, 8
    jobs = []
    for H in (300, 380_000):
        q0, blocks = 8 * H, H + 6
        kv8 = torch.zeros((1, blocks, 1, 2, B, D), dtype=torch.uint8, device=dev)
        kv8[:, :300] = torch.randint(0, 127, (1, 300, 1, 2, B, D), generator=g, dtype=torch.uint8).to(dev)
        sel = torch.stack([torch.randperm(300, generator=g)[:k].sort().values for _ in range(nq)]).view(1, nq, 1, k)
        p = Params(num_kv_groups=1, topk=k)
        jobs.append(dict(p=p, q0=q0, cap=8 * blocks, q=(torch.randn((1, nq, HG, D), generator=g) * 0.01).to(torch.bfloat16).to(dev),
                         kv8=kv8, sc=torch.full((1, blocks, 1, 2), 2.0 ** -8, device=dev), sel=sel.int().to(dev),
                         cnt=torch.full((1, nq, 1), k, dtype=torch.int32, device=dev),
                         out=torch.zeros((1, nq, HG, D), dtype=torch.bfloat16, device=dev),
                         ws=Bd.alloc_workspace_q8(p, 1, nq, q0 + nq, dev), stream=torch.cuda.Stream(device=dev)))

    def call(j):  # the library's call itself: host threads are inside it at once more often
        a = j.get("args")
        if a is None:
            ptr = {x: t.data_ptr() for x, t in j.items() if torch.is_tensor(t)}
            a = j["args"] = (ctypes.byref(j["p"].c()), 1, j["q0"], nq, ptr["q"], j["cap"], j["q0"] + nq, ptr["kv8"], ptr["sc"],
                             ptr["sel"], ptr["cnt"], None, None, ptr["out"], ptr["ws"], j["ws"].numel(), j["stream"].cuda_stream)
        Bd._ok(Bd._lib.sgqa_sparse_attn_q8(*a))

    want = []
    torch.cuda.synchronize()
    for j in jobs:
        call(j)
        torch.cuda.synchronize()
        want.append(j["out"].clone())
    errors = []

    def work(j):
        try:
            torch.cuda.set_device(dev)
            for _ in range(4000):
                call(j)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    Bd.sgqa_check()
    assert not errors, errors[0]
    assert all(torch.equal(j["out"], w) for j, w in zip(jobs, want))


# ------------------ NaN blocks, weights
def row_weights(c, s, i, g):
    """Weights [blocks] that the heads of one (query, group) give."""
    n = lambda t: t.cpu().double().numpy()  # noqa: E731
    hs = slice(g * HG, (g + 1) * HG)
    return R.attention(n(c["q"][s:s + 1, i:i + 1, hs]), R.codes_to_values(c["kv8"][s:s + 1, :, g:g + 1]),
                       n(c["sc"][s:s + 1, :, g:g + 1]), c["sel"][s:s + 1, i:i + 1, g:g + 1].cpu().numpy(),
                       c["cnt"][s:s + 1, i:i + 1, g:g + 1].cpu().numpy(), c["q0"] + i)[2][0]


@pytest.mark.parametrize("nq", [1, 2, 40])
@pytest.mark.parametrize("current", [False, True])
def test_weights_beside_nan_blocks(Bd, cuda_device, nq, current):
    # K with a NaN: the weights of every (query, group) that attends the block are NaN and not counted; V with one: the
    # weights are as ever
    c = T.make_attn(2, 2, nq, 1001, 50, cuda_device)
    bad_k, bad_v = (1001 // B, 1001 // B) if current else (37, 42)
    if not current:
        c["sel"][0, 0, 0, 0], c["sel"][0, 0, 1, 0] = bad_k, bad_v
    c["sel"] = c["sel"].sort(-1).values  # (k = 50 of 125 blocks: all lists are full)
    for s in range(2):  # an id set twice moves on to a free one
        for i in range(nq):
            for g in range(2):
                ids = sorted(set(c["sel"][s, i, g].tolist()))
                free = (x for x in range(125) if x not in ids)
                while len(ids) < 50:
                    ids.append(next(free))
                c["sel"][s, i, g] = torch.tensor(sorted(ids), dtype=torch.int32)
    want = np.zeros((2, c["cap"] // B))
    for s in range(2):
        for i in range(nq):
            for g in range(2):
                hit = s == 0 and g == 0 and ((c["q0"] + i) // B == bad_k or bool((c["sel"][s, i, g] == bad_k).any()))
                if not hit:
                    want[s] += row_weights(c, s, i, g)
    c["sc"][0, bad_k, 0, 0] = float("nan")
    c["sc"][0, bad_v, 1, 1] = float("nan")
    acc = torch.zeros((2, c["cap"] // B), dtype=torch.int64, device=cuda_device)
    out = T.run_attn(Bd, c, acc=acc)
    T.check_weights(acc, 0, want, nq * 2 * 2)
    assert torch.isnan(out[0, 0]).all() and not torch.isnan(out[1]).any()


# ------------------ lists that break the contract
@pytest.mark.parametrize("nq", [1, 40])
def test_repeated_and_unordered_ids(Bd, cuda_device, nq):
    # few queries leave out (and report) an id that is not above the one before it; many attend the set of the list
    c = T.make_attn(1, 1, nq, 400, 8, cuda_device)
    for i in range(nq):
        c["sel"][0, i, 0] = torch.tensor([3, 9, 9, 20, 30, 25, 31, 40], dtype=torch.int32)
    out = T.run_attn(Bd, c, check=False)
    if nq <= 32:
        with pytest.raises(Bd.SgqaError) as e:
            Bd.sgqa_check()
        assert e.value.code == 6
        ids = [3, 9, 20, 30, 31, 40]
    else:
        Bd.sgqa_check()
        ids = [3, 9, 20, 25, 30, 31, 40]
    c["sel"][0, :, 0, :len(ids)] = torch.tensor(ids, dtype=torch.int32, device=cuda_device)
    c["cnt"].fill_(len(ids))
    ref, tol, _ = T.reference(c)
    T.check_attn(c, out, ref, tol)


# ------------------ the softmax scale
@pytest.mark.parametrize("nq", [1, 7, 40])
@pytest.mark.parametrize("scale", [0.03125, 0.2])
def test_softmax_scale(Bd, cuda_device, nq, scale):
    c = T.make_attn(2, 2, nq, 1003, 60, cuda_device)
    n = lambda t: t.cpu().double().numpy()  # noqa: E731
    ref, tol, weights = R.attention(n(c["q"]) * (float(np.float32(scale)) * math.sqrt(D)), R.codes_to_values(c["kv8"]), n(c["sc"]),
                                    c["sel"].cpu().numpy(), c["cnt"].cpu().numpy(), c["q0"])
    p = Params(num_kv_groups=2, topk=60, scale=scale)
    out = torch.zeros_like(c["q"])
    acc = torch.zeros((2, c["cap"] // B), dtype=torch.int64, device=cuda_device)
    ws = Bd.alloc_workspace_q8(p, 2, nq, 1003 + nq, cuda_device)
    Bd.sgqa_sparse_attn_q8(p, 2, c["q0"], nq, c["q"], c["cap"], c["clen"], c["kv8"], c["sc"], c["sel"], c["cnt"], out, ws, acc=acc)
    Bd.sgqa_check()
    T.check_attn(c, out, ref, tol)
    T.check_weights(acc, 0, weights, nq * 2 * 2)


# ------------------ sinks
@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("strength", [12.0, 16.0])
def test_a_sink_leaves_the_others_weights(Bd, cuda_device, nq, strength):
    """One token with V = 0 takes e^strength of every other token's weight; the result lies in the others.

    A weight's rounding is off by at most 2^-9 of it (three E5M2 values; FP16: 2^-11), 2^-14 for its score, and 2^-27 of
    the largest weight of the row; the roundings of different tokens have nothing to do with one another, so the errors'
    mean square is at most the sum of the squares of these bounds times the values.  The result's own rounding: 2^-8 of it."""
    c = T.make_attn(1, 2, nq, 4001, 500, cuda_device, sigma=0.2)
    c["sel"][..., 0] = 0
    c["q"][..., 0] = 4.0
    one = torch.tensor(448.0).to(torch.float8_e4m3fn).view(torch.uint8).to(cuda_device)
    c["kv8"][:, :, :, 0, :, 0] = 0
    c["kv8"][:, 0, :, :, 3] = 0
    c["kv8"][:, 0, :, 0, 3, 0] = one
    c["sc"][:, :, :, 0] = 2.0 ** -10
    c["sc"][:, 0, :, 0] = strength * 192 ** 0.5 / (448 * 4)
    c["sc"][:, :, :, 1] = 2.0 ** -8
    got = T.run_attn(Bd, c, gate=False)[0].cpu().double().numpy()
    err = square = size = 0.0
    for i in range(nq):
        t = c["q0"] + i
        for g in range(2):
            ids = c["sel"][0, i, g, :c["cnt"][0, i, g]].tolist() + [t // B]
            n = len(ids) * B - (B - 1 - t % B)
            K, V = ((R.codes_to_values(c["kv8"][0, ids, g, x]) * c["sc"][0, ids, g, x].cpu().double().numpy()[:, None, None])
                    .reshape(-1, D)[:n] for x in (0, 1))
            hs = slice(g * HG, (g + 1) * HG)
            s = c["q"][0, i, hs].cpu().double().numpy() @ K.T / math.sqrt(D)
            w = np.exp(s - s.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            off = (2.0 ** -9 + 2.0 ** -14) * w + 2.0 ** -27 * w.max(1, keepdims=True)
            err += ((got[i, hs] - w @ V) ** 2).sum()
            square += (off ** 2 @ V ** 2).sum()
            size += ((w @ V) ** 2).sum()
    err, bound, size = math.sqrt(err), math.sqrt(square) + 2.0 ** -8 * math.sqrt(size), math.sqrt(size)
    assert bound < size / 4  # (zeros would not pass)
    assert err <= bound, (err, bound, size)


# ------------------ a BF16 cache
def test_evict_a_bf16_cache_by_given_weights(Bd, cuda_device):
    from sparse_long_context_sgqa_b200.api import SparseGQA
    dev, S, G, H, cap, n, part = cuda_device, 2, 2, 4, 512, 43, 3
    p = Params(num_kv_groups=G, idx_heads=H, topk=9)
    g = T.gen(6)
    r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(dev)  # noqa: E731
    m = SparseGQA(p, S, cap, 16, dev, keep_merged_f32=True)
    for t in (m.k, m.v, m.kp, m.c):
        t.copy_(r(*t.shape))
    Bd.sgqa_merge_blocks(p, S, cap, m.kp, m.c, 0, n, m.merged, m.store)
    acc = torch.randint(0, 1 << 40, (S, cap // B), generator=g).to(dev)
    length = n * B + part
    before = {x: getattr(m, x).clone() for x in ("k", "v", "kp", "c", "store", "merged")}
    acc0 = acc.cpu()
    with pytest.raises(ValueError):
        m.evict(length, 20)
    new = m.evict(length, 20, first=2, recent=4, acc=acc)
    Bd.sgqa_check()
    assert new == 20 * B + part and (m.evicted, m.pos_count) == (23, 20)
    other = SparseGQA(p, S, cap, 16, dev)
    for s in range(S):
        src, new_acc, num = R.evict(n, True, 20, 2, 4, acc0[s].tolist(), [], 0, 0)
        assert np.array_equal(acc[s].cpu().numpy(), new_acc) and m.pos[s, :20].tolist() == num
        rows = torch.cat([torch.arange(b * B, b * B + B) for b in src]).to(dev)
        for x in ("k", "v"):
            assert torch.equal(getattr(m, x)[s, :len(rows)], before[x][s, rows])
        for x in ("store", "merged"):
            assert torch.equal(getattr(m, x)[s, :20], before[x][s, src[:20]])
        for x in ("kp", "c"):
            assert torch.equal(getattr(m, x)[s, 20 * B:new], before[x][s, n * B:length])
        for x in ("k", "v", "kp", "c"):
            getattr(other, x)[s, :len(rows)] = before[x][s, rows]
        other.store[s, :20] = before["store"][s, src[:20]]
    # and the next call reads the rearranged cache
    outs = []
    q, iq, iw = r(S, 7, G * HG, D), r(S, 7, G, H, 64), r(S, 7, G, H).float()
    rows = {x: r(S, 7, *getattr(m, x).shape[2:]) for x in ("k", "v", "kp", "c")}
    for x in (m, other):
        for name, t in rows.items():
            getattr(x, name)[:, new:new + 7] = t
        out = torch.zeros_like(q)
        sel, cnt = torch.empty((S, 7, G, 9), dtype=torch.int32, device=dev), torch.empty((S, 7, G), dtype=torch.int32, device=dev)
        x.forward(new, q, iq, iw, sel, cnt, out)
        Bd.sgqa_check()
        outs.append((out, sel))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# ------------------ a shorter call after a longer one
def test_drafts_taken_back_within_the_block(Bd, cuda_device):
    # five tokens, of which the last three are replaced: `tail` holds the rows before them
    G, dev = 2, cuda_device
    k, v = T.rows(1, 21, G, 1), T.rows(1, 21, G, 2)
    p = Params(num_kv_groups=G)
    kv8, sc, tail = T.empty_cache(1, 4, G, dev)
    junk_k, junk_v = T.rows(1, 3, G, 3) * 50, T.rows(1, 3, G, 4) * 50
    T.append(Bd, p, 1, 32, [17], k, v, kv8, sc, tail, dev)
    Bd.sgqa_kv_append_q8(p, 1, 32, 17, 5, torch.cat([k[:, 17:19], junk_k], 1).to(dev), torch.cat([v[:, 17:19], junk_v], 1).to(dev),
                         tail, kv8, sc)
    Bd.sgqa_kv_append_q8(p, 1, 32, 19, 2, k[:, 19:].to(dev), v[:, 19:].to(dev), tail, kv8, sc)
    Bd.sgqa_check()
    T.check_cache(k, v, 21, kv8, sc, tail)
