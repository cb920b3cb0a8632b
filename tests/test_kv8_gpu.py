"""The 8-bit cache's operators on the GPU against plain 64-bit implementations.

Tolerances.  Codes, scales, tails and evictions are exact.  Attention output: _kv8_ref.attention derives it; scores,
exponentials and FP32 sums stay well under its 2^-10 (a score of magnitude 30 in FP32: 2^-19; exp2: 2^-22; a query
value's second E4M3: 2^-18 of the row's largest).  Accumulated weights: per (call, row, block) at most half a unit of 2^-32, and 2^-14 relative from the same FP32 sources
(a row's scores are off by at most 192 terms' rounding, 2^-15 at magnitude 30).
"""
import numpy as np
import pytest
import torch

from sparse_long_context_sgqa_b200.binding import Params
from tests import _kv8_ref as R

pytestmark = pytest.mark.gpu
D, HG, B = R.D, R.HG, R.B


@pytest.fixture(scope="module")
def Bd():
    from sparse_long_context_sgqa_b200 import binding
    return binding


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rows(S, n, G, seed):
    g = gen(seed)
    return (torch.randn((S, n, G, D), generator=g) * (torch.rand((S, n, G, 1), generator=g) * 4 + 0.01)).to(torch.bfloat16)


def empty_cache(S, blocks, G, dev, fill=0x35):
    return (torch.full((S, blocks, G, 2, B, D), fill, dtype=torch.uint8, device=dev),
            torch.full((S, blocks, G, 2), -3.0, device=dev),
            torch.full((S, 2, B, G, D), 9.0, dtype=torch.bfloat16, device=dev))


def append(Bd, p, S, cap, cuts, k, v, kv8, sc, tail, dev):
    pos = 0
    for n in cuts:
        Bd.sgqa_kv_append_q8(p, S, cap, pos, n, k[:, pos:pos + n].contiguous().to(dev), v[:, pos:pos + n].contiguous().to(dev),
                             tail, kv8, sc)
        pos += n
    Bd.sgqa_check()
    return pos


def check_cache(k, v, n, kv8, sc, tail):
    S, G = k.shape[0], k.shape[2]
    nb = -(-n // B)
    for s in range(S):
        for x, src in ((0, k), (1, v)):
            codes, scales = R.quantise_rows(src[s, :n].double().numpy())
            got = kv8[s, :nb, :, x].cpu().numpy()
            assert np.array_equal(got, codes), np.argwhere(got != codes)[:4]
            np.testing.assert_array_equal(sc[s, :nb, :, x].cpu().double().numpy(), scales)
            left = n % B
            assert torch.equal(tail[s, x, :left].cpu().view(torch.int16), src[s, n - left:n].view(torch.int16))
    # nothing behind the last block was touched
    assert (kv8[:, nb:] == 0x35).all() and (sc[:, nb:] == -3.0).all()


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("S,G,cuts", [
    (1, 4, [1]), (1, 1, [8]), (2, 4, [1] * 19), (3, 2, [5, 1, 3, 12, 2]), (1, 3, [7, 9, 64, 1]), (2, 5, [100]),
    (16, 4, [3, 1]), (1, 4, [1001]), (2, 1, [4, 4, 8, 6, 20])])
def test_append_parity(Bd, cuda_device, S, G, cuts):
    n = sum(cuts)
    cap = (n + 23) // 8 * 8
    k, v = rows(S, n, G, n), rows(S, n, G, n + 1)
    kv8, sc, tail = empty_cache(S, cap // B, G, cuda_device)
    append(Bd, Params(num_kv_groups=G), S, cap, cuts, k, v, kv8, sc, tail, cuda_device)
    check_cache(k, v, n, kv8, sc, tail)


def test_append_special_values(Bd, cuda_device):
    n, G = 64, 2
    k, v = rows(1, n, G, 3), rows(1, n, G, 4)
    k[0, 0:8] = 0                                   # a block of zeros: the smallest scale
    v[0, 0:8] = -0.0
    k[0, 8:16] = 1e-39                              # subnormal BF16
    v[0, 8:16] = torch.finfo(torch.bfloat16).max
    k[0, 17, 0, 5] = float("nan")                   # one group's K of block 2
    v[0, 18, 1, 191] = float("-inf")                # the other group's V
    k[0, 24:32] *= 2.0 ** 100
    v[0, 24:32] *= 2.0 ** -100
    for j in range(8):                              # magnitudes next to a power of two times 448
        k[0, 32 + j] = (448 if j % 2 else 450) * 2.0 ** (j - 4)
        k[0, 40 + j] = 448 * 2.0 ** -3
        v[0, 40 + j] = 450 * 2.0 ** -3
    kv8, sc, tail = empty_cache(1, 9, G, cuda_device)
    append(Bd, Params(num_kv_groups=G), 1, 72, [n], k, v, kv8, sc, tail, cuda_device)
    check_cache(k, v, n, kv8, sc, tail)
    assert torch.isnan(sc[0, 2, 0, 0]) and torch.isnan(sc[0, 2, 1, 1]) and int(torch.isnan(sc).sum()) == 2


def test_append_every_bf16_value_next_to_a_larger_one(Bd, cuda_device):
    # 64 blocks of one token each time: codes of 12288 BF16 patterns under the scale their block's largest gives
    x = torch.arange(0, 64 * 8 * D, dtype=torch.int32) * 5 % 0x7F80
    k = x.to(torch.uint16).view(torch.bfloat16).view(1, 512, 1, D)
    kv8, sc, tail = empty_cache(1, 65, 1, cuda_device)
    append(Bd, Params(num_kv_groups=1), 1, 520, [512], k, -k, kv8, sc, tail, cuda_device)
    check_cache(k, -k, 512, kv8, sc, tail)


def test_append_does_not_depend_on_the_cuts(Bd, cuda_device):
    S, G, n = 2, 4, 333
    k, v = rows(S, n, G, 1), rows(S, n, G, 2)
    got = []
    for cuts in ([n], [1] * n, [7] * 47 + [4], [100, 5, 228]):
        kv8, sc, tail = empty_cache(S, 48, G, cuda_device)
        append(Bd, Params(num_kv_groups=G), S, 384, cuts, k, v, kv8, sc, tail, cuda_device)
        got.append((kv8, sc, tail[:, :, :n % B]))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


# ------------------------------------------------------------------ attention
def make_attn(S, G, nq, q0, k, dev, seed=0, spread=4, extra=0, sigma=1.0):
    """A cache of q0 + nq + extra tokens with random codes and scales, queries and a causal selection."""
    g = gen(seed + 1000 * nq + q0)
    clen = q0 + nq + extra
    blocks = -(-clen // B) + 1
    kv8 = (torch.randn((S, blocks, G, 2, B, D), generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    sc = torch.exp2(torch.randint(-7 - spread, -6, (S, blocks, G, 2), generator=g).float())
    sc[:, -(-clen // B):] = 1.0
    q = (torch.randn((S, nq, G * HG, D), generator=g) * sigma).to(torch.bfloat16)
    sel = torch.full((S, nq, G, k), -1, dtype=torch.int32)
    cnt = torch.zeros((S, nq, G), dtype=torch.int32)
    for s in range(S):
        for i in range(nq):
            h = (q0 + i) // B
            for gg in range(G):
                c = min(k, h)
                ids = torch.randperm(h, generator=g)[:c].sort().values
                sel[s, i, gg, :c] = ids.int()
                cnt[s, i, gg] = c
    gate = torch.randn((S, nq, G * HG), generator=g).to(torch.bfloat16)
    return dict(S=S, G=G, nq=nq, q0=q0, k=k, cap=blocks * B, clen=clen, kv8=kv8.to(dev), sc=sc.to(dev), q=q.to(dev),
                sel=sel.to(dev), cnt=cnt.to(dev), gate=gate.to(dev))


def run_attn(Bd, c, gate=True, acc=None, stream=None, out=None, check=True, ws=None):
    p = Params(num_kv_groups=c["G"], topk=c["k"])
    out = torch.full_like(c["q"], 7.0) if out is None else out
    if ws is None:
        ws = Bd.alloc_workspace_q8(p, c["S"], c["nq"], c["q0"] + c["nq"], c["q"].device)
    Bd.sgqa_sparse_attn_q8(p, c["S"], c["q0"], c["nq"], c["q"], c["cap"], c["clen"], c["kv8"], c["sc"], c["sel"], c["cnt"],
                           out, ws, gate=c["gate"] if gate else None, acc=acc, stream=stream)
    if check:
        Bd.sgqa_check(stream)
    return out


def reference(c, gate=True):
    n = lambda t: t.cpu().double().numpy()  # noqa: E731
    return R.attention(n(c["q"]), R.codes_to_values(c["kv8"]), n(c["sc"]), c["sel"].cpu().numpy(), c["cnt"].cpu().numpy(),
                       c["q0"], n(c["gate"]) if gate else None)


def check_attn(c, out, ref, tol):
    R.check_out(out, ref, tol)


def check_weights(acc, before, weights, adds):
    got = (acc - before).cpu().double().numpy() * R.UNIT
    tol = adds * R.UNIT + 2.0 ** -14 * weights
    assert (np.abs(got - weights) <= tol).all(), np.abs(got - weights).max()


SHAPES = [
    # S, G, nq, q0, k
    (1, 4, 1, 0, 512),        # the first token of a sequence: nothing selected
    (2, 1, 1, 7, 4),          # a full current block
    (1, 2, 1, 8, 1),
    (3, 4, 1, 1001, 512),     # every block
    (2, 4, 1, 5003, 100),
    (1, 1, 1, 40000, 2048),
    (2, 3, 5, 0, 16),         # queries that begin at position 0
    (5, 2, 7, 2003, 60),
    (1, 4, 32, 777, 512),
    (1, 4, 33, 0, 512),
    (2, 2, 40, 8, 7),
    (1, 1, 129, 300, 33),
    (2, 4, 65, 1021, 128),
    (1, 2, 200, 4000, 300),
]


@pytest.mark.parametrize("S,G,nq,q0,k", SHAPES)
def test_attention_parity(Bd, cuda_device, S, G, nq, q0, k):
    c = make_attn(S, G, nq, q0, k, cuda_device)
    ref, tol, weights = reference(c)
    check_attn(c, run_attn(Bd, c), ref, tol)
    acc = torch.randint(0, 1 << 40, (S, c["cap"] // B), device=cuda_device)
    before = acc.clone()
    check_attn(c, run_attn(Bd, c, acc=acc), ref, tol)
    check_weights(acc, before, weights, nq * G * 2)
    # every head of every query gives 1 in all
    total = (acc - before).double().sum(1).cpu().numpy() * R.UNIT
    np.testing.assert_allclose(total, nq * G * HG, rtol=2.0 ** -14)


@pytest.mark.parametrize("S,G,nq,q0,k", [(2, 4, 1, 3001, 64), (1, 2, 70, 500, 40)])
def test_attention_ungated_and_with_tokens_behind_the_queries(Bd, cuda_device, S, G, nq, q0, k):
    c = make_attn(S, G, nq, q0, k, cuda_device, extra=21)
    ref, tol, _ = reference(c, gate=False)
    check_attn(c, run_attn(Bd, c, gate=False), ref, tol)


@pytest.mark.parametrize("nq", [1, 48])
def test_attention_sharp_and_far_scores(Bd, cuda_device, nq):
    # large queries: weights next to one-hot, scores of some hundreds, the running maximum moves
    c = make_attn(1, 2, nq, 2000, 200, cuda_device, sigma=40.0)
    ref, tol, _ = reference(c)
    # a score of magnitude 500 in FP32 is off by up to 2^-15, a weight by as much of it
    check_attn(c, run_attn(Bd, c), ref, tol)


@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("strength", [12.0, 16.0, 22.0])
def test_attention_sink(Bd, cuda_device, nq, strength):
    # one token with V = 0 takes nearly all of every row (e^12 .. e^22 of another token's weight): the result lies in the
    # small weights of all the others
    c = make_attn(1, 2, nq, 4001, 500, cuda_device, sigma=0.2)
    c["sel"][..., 0] = 0
    c["q"][..., 0] = 4.0
    c["kv8"][:, 0, :, :, 3] = 0
    c["kv8"][:, 0, :, 0, 3, 0] = torch.tensor(448.0).to(torch.float8_e4m3fn).view(torch.uint8).to(cuda_device)
    c["kv8"][:, :, :, 0, :, 0] = torch.where(c["kv8"][:, :, :, 0, :, 0] == c["kv8"][0, 0, 0, 0, 3, 0], c["kv8"][:, :, :, 0, :, 0], 0)
    c["sc"][:, 0, :, 0] = strength * 192 ** 0.5 / (448 * 4)
    ref, tol, _ = reference(c)
    check_attn(c, run_attn(Bd, c), ref, tol)


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_blocks_of_very_different_scale(Bd, cuda_device, nq):
    # V scales over 2^24: the result must be right in every head, also where the weight lies on blocks of small values
    c = make_attn(1, 2, nq, 900, 90, cuda_device, spread=24)
    ref, tol, _ = reference(c)
    check_attn(c, run_attn(Bd, c), ref, tol)
    # and blocks of zeros among them (the scale the append gives those)
    c["sc"][:, ::3, :, 1] = 2.0 ** -100
    c["kv8"][:, ::3, :, 1] = 0
    ref, tol, _ = reference(c)
    check_attn(c, run_attn(Bd, c), ref, tol)


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_scales_between_powers_of_two(Bd, cuda_device, nq):
    c = make_attn(2, 2, nq, 1500, 120, cuda_device, sigma=3.0)
    c["sc"] *= torch.rand(c["sc"].shape, generator=gen(8)).to(cuda_device) + 1
    ref, tol, weights = reference(c)
    acc = torch.zeros((2, c["cap"] // B), dtype=torch.int64, device=cuda_device)
    check_attn(c, run_attn(Bd, c, acc=acc), ref, tol)
    check_weights(acc, 0, weights, nq * 2 * 2)


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_of_queries_with_infinities(Bd, cuda_device, nq):
    c = make_attn(1, 2, nq, 500, 40, cuda_device)
    bad = c["q"].clone()
    bad[0, 0, 3, 7], bad[0, nq - 1, 20, 100] = float("inf"), float("nan")
    fine = run_attn(Bd, c)
    c["q"] = bad
    acc = torch.zeros((1, c["cap"] // B), dtype=torch.int64, device=cuda_device)
    got = run_attn(Bd, c, acc=acc)
    assert torch.isnan(got[0, 0, 3]).all() and torch.isnan(got[0, nq - 1, 20]).all()
    same = torch.ones(got.shape[:3], dtype=torch.bool, device=cuda_device)
    same[0, 0, 3] = same[0, nq - 1, 20] = False
    assert torch.equal(got[same], fine[same])
    # the other heads' weights are counted
    assert abs(float(acc.double().sum()) * R.UNIT - (nq * 2 * HG - 2)) < 1e-3


@pytest.mark.parametrize("nq", [1, 64])
def test_a_wait_that_runs_out_is_reported_and_later_calls_succeed(Bd, cuda_device, nq):
    c = make_attn(2, 4, nq, 3000, 256, cuda_device)
    acc = torch.zeros((2, c["cap"] // B), dtype=torch.int64, device=cuda_device)
    first = run_attn(Bd, c, acc=acc)
    once = acc.clone()
    try:
        Bd.sgqa_set_wait_limit_ns(1)
        with pytest.raises(Bd.SgqaError) as e:
            run_attn(Bd, c, acc=acc)
    finally:
        Bd.sgqa_set_wait_limit_ns(0)
    assert e.value.code == 5
    acc.zero_()
    assert torch.equal(run_attn(Bd, c, acc=acc), first) and torch.equal(acc, once)


@pytest.mark.parametrize("nq", [2, 40])
def test_nan_blocks_reach_only_who_attends_them(Bd, cuda_device, nq):
    c = make_attn(2, 2, nq, 1000, 50, cuda_device)
    bad = 37
    c["sc"][0, bad, 0, 0] = float("nan")
    c["sc"][0, bad + 5, 1, 1] = float("nan")
    acc = torch.zeros((2, c["cap"] // B), dtype=torch.int64, device=cuda_device)
    got = run_attn(Bd, c, acc=acc).cpu().double().view(2, nq, 2, HG, D)
    sel = c["sel"].cpu()
    c["sc"].nan_to_num_(nan=2.0 ** -7)
    ref, tol, _ = reference(c)
    ref, tol = torch.from_numpy(ref).view(got.shape), torch.from_numpy(tol).view(got.shape)
    hit = torch.zeros((2, nq, 2), dtype=torch.bool)
    hit[0, :, 0] = (sel[0, :, 0] == bad).any(-1)
    hit[0, :, 1] = (sel[0, :, 1] == bad + 5).any(-1)
    assert torch.isnan(got[hit]).all()
    fine = ~hit
    assert ((got - ref).abs() <= tol)[fine].all()
    assert (acc >= 0).all()


@pytest.mark.parametrize("nq", [1, 40])
def test_bad_selections_are_reported_and_left_out(Bd, cuda_device, nq):
    c = make_attn(1, 2, nq, 400, 8, cuda_device)
    bad = {0: -5, 1: 50, 2: 1 << 30}   # negative, the current block's own number, far outside
    good = c["sel"].clone()
    c["sel"][0, 0, 0, 7] = bad[1]
    c["sel"][0, 0, 1, 7] = bad[2]
    c["cnt"][0, nq - 1, 0] = 7 if nq > 1 else 8
    out = run_attn(Bd, c, check=False)
    with pytest.raises(Bd.SgqaError) as e:
        Bd.sgqa_check()
    assert e.value.code == 6
    c["sel"] = good
    c["cnt"][0, 0] = 7  # the bad entries left out
    ref, tol, _ = reference(c)
    check_attn(c, out, ref, tol)
    Bd.sgqa_check()


def test_counts_outside_the_list_are_clamped(Bd, cuda_device):
    c = make_attn(1, 1, 1, 800, 5, cuda_device)
    ref, tol, _ = reference(c)
    c["cnt"].fill_(1 << 30)
    check_attn(c, run_attn(Bd, c), ref, tol)
    c["cnt"].fill_(-1)
    out = run_attn(Bd, c)
    c["cnt"].fill_(0)
    ref, tol, _ = reference(c)
    check_attn(c, out, ref, tol)


@pytest.mark.parametrize("nq", [1, 6, 72])
def test_weights_and_outputs_repeat_bit_for_bit(Bd, cuda_device, nq):
    c = make_attn(3, 4, nq, 3000, 128, cuda_device)
    first = None
    for _ in range(4):
        acc = torch.zeros((3, c["cap"] // B), dtype=torch.int64, device=cuda_device)
        out = run_attn(Bd, c, acc=acc)
        if first is None:
            first = (out, acc)
        assert torch.equal(out.view(torch.int16), first[0].view(torch.int16)) and torch.equal(acc, first[1])
    assert torch.equal(run_attn(Bd, c).view(torch.int16), first[0].view(torch.int16))


@pytest.mark.parametrize("nq", [1, 40])
def test_two_streams_and_a_replayed_graph(Bd, cuda_device, nq):
    c = make_attn(2, 4, nq, 2000, 64, cuda_device)
    want = run_attn(Bd, c)
    p = Params(num_kv_groups=4, topk=64)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(want) for _ in streams]
    wss = [Bd.alloc_workspace_q8(p, 2, nq, 2000 + nq, cuda_device) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o, w in zip(streams, outs, wss):
            run_attn(Bd, c, stream=s, out=o, ws=w, check=False)
    torch.cuda.synchronize()
    Bd.sgqa_check()
    for o in outs:
        assert torch.equal(o, want)
    acc = torch.zeros((2, c["cap"] // B), dtype=torch.int64, device=cuda_device)
    run_attn(Bd, c, acc=acc)
    once = acc.clone()
    graph = torch.cuda.CUDAGraph()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run_attn(Bd, c, acc=acc, out=out, ws=wss[0], check=False)
    acc.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(acc, 3 * once)


# ------------------------------------------------------------------ eviction
def evict_case(S, n, part, B_, seed, dev, known, evicted, ties):
    g = gen(seed)
    slots = n + 1 + 3
    acc = (torch.rand((S, slots), generator=g, dtype=torch.float64) ** 4 * 2.0 ** 40).long()
    if ties:
        acc = acc % 3
    pos = torch.full((S, slots), -9, dtype=torch.int32)
    for s in range(S):
        pos[s, :known] = torch.randperm(known + evicted, generator=g)[:known].int()
    arrays = [torch.randint(0, 256, (S, slots, w), generator=g, dtype=torch.uint8).to(dev) for w in (48, 8, 3, 2, 4096)]
    tails = [torch.randint(0, 256, (S, slots, 32), generator=g, dtype=torch.uint8).to(dev)]
    return slots, acc.to(dev), pos.to(dev), arrays, tails


@pytest.mark.parametrize("S,n,part,B_,keep,first,recent,known,evicted,ties", [
    (1, 1, 1, 8, 1, 0, 0, 0, 0, False), (1, 1, 0, 8, 0, 0, 0, 0, 0, False), (1, 1, 3, 8, 0, 0, 0, 0, 0, False),
    (2, 5, 2, 8, 3, 1, 1, 0, 0, False), (3, 100, 7, 8, 60, 2, 8, 70, 40, False), (1, 100, 0, 4, 33, 0, 0, 100, 900, True),
    (2, 513, 1, 2, 400, 4, 16, 300, 77, True), (4, 2000, 5, 8, 1999, 1, 1, 0, 0, False), (1, 40, 3, 8, 40, 0, 0, 10, 3, False),
    (2, 3001, 0, 1, 1500, 10, 700, 3001, 11, True), (1, 1200, 4, 8, 600, 300, 300, 500, 5, True),
    (3, 20000, 6, 8, 15000, 4, 64, 15000, 100000, False), (1, 70000, 1, 8, 1000, 0, 0, 0, 0, True),
    (2, 64, 7, 8, 0, 0, 0, 64, 1, False), (1, 131072, 2, 8, 100000, 4, 512, 0, 0, False), (1, 140000, 0, 1, 30000, 4, 64, 9, 2, False),
    (2, 16385, 3, 8, 16000, 0, 0, 0, 0, True), (1, 131072, 0, 8, 65536, 0, 0, 131072, 7, True), (1, 4097, 1, 8, 4096, 0, 0, 0, 0, False),
    (40, 700, 1, 8, 650, 1, 1, 0, 0, False)])
def test_evict_parity(Bd, cuda_device, S, n, part, B_, keep, first, recent, known, evicted, ties):
    part = part % B_
    slots, acc, pos, arrays, tails = evict_case(S, n, part, B_, n + keep, cuda_device, known, evicted, ties)
    p = Params(block_size=B_)
    ws = Bd.alloc_evict_workspace(p, S, slots * B_, cuda_device)
    before = [a.clone() for a in arrays + tails]
    acc0, pos0 = acc.cpu(), pos.cpu()
    for in_place in (False, True):
        for a, b in zip(arrays + tails, before):
            a.copy_(b)
        ao, po = (acc, pos) if in_place else (torch.full_like(acc, -4), torch.full_like(pos, -4))
        Bd.sgqa_evict(p, S, slots * B_, n * B_ + part, keep, first, recent, acc, pos if known else None, known, evicted,
                      ao, po, arrays, ws, tail_arrays=tails)
        Bd.sgqa_check()
        for s in range(S):
            src, new_acc, num = R.evict(n, part > 0, keep, first, recent, acc0[s].tolist(), pos0[s].tolist(), known, evicted)
            assert np.array_equal(ao[s].cpu().numpy(), new_acc)
            assert po[s, :keep].tolist() == num
            assert torch.equal(po[s, keep:].cpu(), pos0[s, keep:] if in_place else torch.full((slots - keep,), -4, dtype=torch.int32))
            for a, b in zip(arrays, before):
                assert torch.equal(a[s, :len(src)], b[s, src])
            if part:
                assert torch.equal(tails[0][s, keep], before[-1][s, n])
                assert torch.equal(tails[0][s, :keep], before[-1][s, :keep])


def test_evict_without_arrays_and_negative_weights(Bd, cuda_device):
    p = Params()
    acc = torch.tensor([[-5, 3, -(1 << 62), 3, (1 << 63) - 1, 0, 1]], device=cuda_device)
    out, pos = torch.zeros_like(acc), torch.zeros((1, 7), dtype=torch.int32, device=cuda_device)
    ws = Bd.alloc_evict_workspace(p, 1, 56, cuda_device)
    Bd.sgqa_evict(p, 1, 56, 56, 4, 1, 0, acc, None, 0, 0, out, pos, [], ws)
    Bd.sgqa_check()
    assert pos[0, :4].tolist() == [0, 1, 4, 3] and out[0].tolist() == [-5, 3, (1 << 63) - 1, 3, 0, 0, 0]


def test_equal_original_numbers_are_reported(Bd, cuda_device):
    p = Params()
    acc = torch.zeros((1, 8), dtype=torch.int64, device=cuda_device)
    pos = torch.zeros((1, 8), dtype=torch.int32, device=cuda_device)
    ws = Bd.alloc_evict_workspace(p, 1, 64, cuda_device)
    data = torch.zeros((1, 8, 16), dtype=torch.uint8, device=cuda_device)
    Bd.sgqa_evict(p, 1, 64, 64, 4, 0, 0, acc, pos, 8, 0, acc.clone(), pos.clone(), [data], ws)
    with pytest.raises(Bd.SgqaError) as e:
        Bd.sgqa_check()
    assert e.value.code == 6


# ------------------------------------------------------------------ together
def test_prefill_decode_evict_decode(Bd, cuda_device):
    """A model over the 8-bit cache: a ragged prefill, token steps, an eviction, token steps, a second eviction, a step."""
    from sparse_long_context_sgqa_b200.api import SparseGQA
    dev, S, G, H = cuda_device, 2, 2, 4
    p = Params(num_kv_groups=G, idx_heads=H, topk=12)
    cap, N = 512, 347
    m = SparseGQA(p, S, cap, 100, dev, kv_dtype="e4m3", track_weights=True)
    g = gen(5)
    m.acc.zero_()

    def tokens(n):
        r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        return dict(q=r(S, n, G * HG, D).to(torch.bfloat16), idx_q=r(S, n, G, H, 64).to(torch.bfloat16),
                    idx_w=r(S, n, G, H), k=r(S, n, G, D).to(torch.bfloat16), v=r(S, n, G, D).to(torch.bfloat16),
                    kp=r(S, n, 64).to(torch.bfloat16), c=r(S, n, 64).to(torch.bfloat16))

    # the model's cache on the host: rows by slot, weights and numbers
    K, V = torch.zeros((S, cap, G, D)), torch.zeros((S, cap, G, D))
    acc = np.zeros((S, cap // B))
    adds = 0

    def step(pos, x, chunked=False):
        nonlocal acc, adds
        n = x["q"].shape[1]
        d = {a: b.to(dev) for a, b in x.items()}
        m.kp[:, pos:pos + n], m.c[:, pos:pos + n] = d["kp"], d["c"]
        out = torch.zeros_like(d["q"])
        sel = torch.full((S, n, G, p.topk), -1, dtype=torch.int32, device=dev)
        cnt = torch.zeros((S, n, G), dtype=torch.int32, device=dev)
        if chunked:  # several sequences: the selection lands in sel and cnt
            m.prefill(d["q"], d["idx_q"], d["idx_w"], out, sel, cnt, q_pos0=pos, k=d["k"], v=d["v"])
        else:
            m.forward(pos, d["q"], d["idx_q"], d["idx_w"], sel, cnt, out, k=d["k"], v=d["v"])
        Bd.sgqa_check()
        K[:, pos:pos + n], V[:, pos:pos + n] = x["k"].float(), x["v"].float()
        sizes = [min(100, n - c) for c in range(0, n, 100)]
        i = 0
        for w in sizes:  # a chunk's queries see their blocks as quantised at the chunk's end
            end = pos + i + w
            nb = -(-end // B)
            vals, scale = np.zeros((S, nb, G, 2, B, D)), np.ones((S, nb, G, 2))
            for s in range(S):
                for xx, src in ((0, K), (1, V)):
                    codes, sc = R.quantise_rows(src[s, :end].double().numpy())
                    vals[s, :, :, xx] = R.codes_to_values(torch.from_numpy(codes))
                    scale[s, :, :, xx] = sc
            sl = slice(i, i + w)
            ref, tol, wts = R.attention(x["q"][:, sl].double().numpy(), vals, scale, sel[:, sl].cpu().numpy(),
                                           cnt[:, sl].cpu().numpy(), pos + i)
            R.check_out(out[:, sl], ref, tol)
            acc[:, :nb] += wts
            adds += w * G * 2
            i += w
        assert (cnt.cpu() == torch.clamp((pos + torch.arange(n)) // B, max=p.topk)[None, :, None]).all()
        return pos + n

    def evict(length, keep, first, recent):
        nonlocal acc, K, V
        got = m.acc.cpu()
        tol = adds * R.UNIT + 2.0 ** -14 * acc
        assert (np.abs(got.double().numpy() * R.UNIT - acc) <= tol).all()
        numbers, known, gone = m.pos, m.pos_count, m.evicted
        numbers = None if numbers is None else numbers.cpu().clone()
        store, kp = m.store.clone(), m.kp.clone()
        n, part = length // B, length % B
        new = m.evict(length, keep, first, recent)
        Bd.sgqa_check()
        assert new == keep * B + part
        K2, V2 = K.clone(), V.clone()
        for s in range(S):
            src, na, num = R.evict(n, part > 0, keep, first, recent, got[s].tolist(),
                                   numbers[s].tolist() if known else [], known, gone)
            assert m.pos[s, :keep].tolist() == num
            assert np.array_equal(m.acc[s].cpu().numpy(), na)
            assert torch.equal(m.store[s, :keep], store[s, src[:keep]])
            for to, frm in enumerate(src):
                K2[s, to * B:to * B + B] = K[s, frm * B:frm * B + B]
                V2[s, to * B:to * B + B] = V[s, frm * B:frm * B + B]
            if part:
                assert torch.equal(m.kp[s, keep * B:keep * B + part], kp[s, n * B:n * B + part])
            acc[s] = na * R.UNIT
        K, V = K2, V2
        return new

    pos = step(0, tokens(N), chunked=True)
    for _ in range(3):
        pos = step(pos, tokens(1))
    pos = evict(pos, 20, 2, 4)
    assert pos == 166
    for _ in range(11):  # across a block boundary
        pos = step(pos, tokens(1))
    pos = step(pos, tokens(37))
    pos = evict(pos, 17, 1, 3)
    pos = step(pos, tokens(5))


def test_forward_host_matches_prefill(Bd, cuda_device):
    from sparse_long_context_sgqa_b200.api import SparseGQA
    S, G, N = 2, 4, 150
    p = Params(num_kv_groups=G, topk=6)
    g = gen(9)
    r = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    host = dict(q=r(S, N, G * HG, D), idx_q=r(S, N, G, 8, 64), idx_w=r(S, N, G, 8).float(), k=r(S, N, G, D), v=r(S, N, G, D),
                kp=r(S, N, 64), c=r(S, N, 64))
    pinned = {a: b.pin_memory() for a, b in host.items()}
    outs = []
    for way in range(2):
        m = SparseGQA(p, S, 160, 64, cuda_device, kv_dtype="e4m3")
        if way == 0:
            out = torch.zeros((S, N, G * HG, D), dtype=torch.bfloat16).pin_memory()
            moved = m.forward_host(pinned, out)
            torch.cuda.synchronize()
            assert moved == (sum(t.numel() * t.element_size() for t in host.values()), out.numel() * 2)
        else:
            d = {a: b.to(cuda_device) for a, b in host.items()}
            m.kp[:, :N], m.c[:, :N] = d["kp"], d["c"]
            out = torch.zeros((S, N, G * HG, D), dtype=torch.bfloat16, device=cuda_device)
            m.prefill(d["q"], d["idx_q"], d["idx_w"], out, k=d["k"], v=d["v"])
        Bd.sgqa_check()
        outs.append((out.cpu(), m.kv8.cpu(), m.kv_scale.cpu()))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
