"""The 8-bit K/V cache's operators, as cases to measure: the append that quantises new K/V rows, the sparse attention that
reads the cache (with the block weights an eviction needs), and the eviction itself.

`run` computes each operator in its plain form (elementary torch operations in FP32), or, where `own` is true, calls the
framework's entry points.  `exact` restates the definitions in FP64.

Cache layout: kv8 [S, blocks, G, 2 (K, V), 8, 192] E4M3 codes, kv_scale [S, blocks, G, 2] FP32, one scale for the eight
tokens of a block in one group's K or V.  The rows of a block that is not complete yet are also held in BF16
(tail [S, 2, 8, G, 192]), so that the block is quantised from its original rows each time it grows.
"""
import math

import torch

own = False

D, HG, B = 192, 16, 8          # head width, query heads per KV group, tokens per block
FIX = 2.0 ** -32               # one unit of an accumulated weight
SCALE = 1.0 / math.sqrt(D)


# ------------------------------------------------------------------ cases
def _append(name, S, G, pos0, n):
    return dict(name=name, op="append", S=S, G=G, pos0=pos0, n=n)


def _attn(name, S, G, nq, q_pos0, k, gate=False, weights=False):
    return dict(name=name, op="attn", S=S, G=G, nq=nq, q_pos0=q_pos0, k=k, gate=gate, weights=weights)


def _evict(name, S, G, n, part, keep, first, recent, known, evicted):
    return dict(name=name, op="evict", S=S, G=G, n=n, part=part, keep=keep, first=first, recent=recent, known=known,
                evicted=evicted)


def listed():
    return [
        # one decode step of 16 sequences: each adds a token in the middle of its block
        _append("append_token", 16, 4, 4099, 1),
        # three prompts of an odd length, continued in the middle of a block
        _append("append_ragged", 3, 4, 37, 1001),
        # one 8192-token chunk of a prefill
        _append("append_chunk", 1, 4, 8192, 8192),
        # the smallest serving call: one sequence, one token, a short context (latency)
        _attn("attn_one_1k", 1, 4, 1, 1023, 512),
        # the decode workload: 16 contexts of 262144 tokens, top-512 blocks
        _attn("attn_decode_16x256k", 16, 4, 1, 262143, 512),
        # decode of a serving batch whose cache is evicted by weight: gated, weights accumulated
        _attn("attn_decode_weights", 16, 4, 1, 32767, 512, True, True),
        # drafted tokens verified together: several queries per sequence, odd sizes, two groups
        _attn("attn_draft_5x7", 5, 2, 7, 20003, 300, False, True),
        # a prefill chunk behind a prompt of 6144 tokens
        _attn("attn_prefill_2k", 1, 4, 2048, 6144, 512),
        # two ragged prompts whose weights are accumulated for a later eviction
        _attn("attn_prefill_weights", 2, 4, 1001, 3003, 256, True, True),
        # one short sequence trimmed by an eighth (latency)
        _evict("evict_one", 1, 4, 520, 3, 456, 2, 16, 400, 64),
        # a serving batch back to 2800 of 4096 blocks
        _evict("evict_batch", 16, 4, 4096, 5, 2800, 4, 64, 2800, 9000),
        # two long contexts cut by a quarter
        _evict("evict_long", 2, 4, 65536, 0, 49152, 4, 512, 0, 0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn_large", "evict"])
    S, G = _log(rng, 1, 16), rng.choice([1, 2, 3, 4, 4])
    if op == "append":
        c = _append("", S, G, rng.randrange(0, 6000), _log(rng, 1, max(1, 24000 // (S * G))))
    elif op == "attn":
        k, nq = _log(rng, 1, 2048), rng.choice([1, 1, 1, rng.randrange(2, 33)])
        S = max(1, min(S, 40000 // (nq * G * k)))
        ctx = _log(rng, nq, max(64, min(262144, (1 << 22) // (S * G))))
        c = _attn("", S, G, nq, ctx - nq, k, rng.random() < 0.5, rng.random() < 0.5)
    elif op == "attn_large":
        S, k = rng.randrange(1, 4), _log(rng, 8, 600)
        nq = _log(rng, 33, max(34, min(2000, 4000000 // (S * G * k))))
        c = _attn("", S, G, nq, _log(rng, 1, 24000) - 1, k, rng.random() < 0.5, rng.random() < 0.5)
    else:
        n = _log(rng, 2, 131072 // (S * max(1, G // 2)))
        keep = rng.randrange((n + 2) // 3, n + 1)
        first = rng.randrange(0, min(keep, 8) + 1)
        recent = rng.randrange(0, min(keep - first, 512) + 1)
        known = rng.randrange(0, n + 1)
        c = _evict("", S, G, n, rng.randrange(0, B), keep, first, recent, known, rng.randrange(0, 5000) if known else 0)
    del c["name"]
    return c


def work(c):
    S, G = c["S"], c["G"]
    if c["op"] == "append":
        rows = S * c["n"] * G * 2
        blocks = S * G * 2 * ((c["pos0"] + c["n"] - 1) // B - c["pos0"] // B + 1)
        return {"bytes": rows * D * 3 + blocks * 4, "flops": rows * D * 2}
    if c["op"] == "attn":
        pairs = read = 0  # (query, group, token) attended; blocks of the cache read
        for i in range(c["nq"]):
            t = c["q_pos0"] + i
            cnt = min(c["k"], t // B)
            pairs += cnt * B + t % B + 1
            read += cnt + 1
        read = min(read, (c["q_pos0"] + c["nq"] + B - 1) // B)
        b = S * G * read * 2 * (B * D + 4) + S * c["nq"] * G * (HG * D * 4 + c["k"] * 4 + 4)
        b += S * c["nq"] * G * HG * 2 * c["gate"] + S * read * 16 * c["weights"]
        return {"bytes": b, "flops": S * G * pairs * 4 * D * HG}
    n, keep = c["n"], c["keep"]
    moved = keep * (n - keep) / n + (c["part"] > 0)  # kept blocks expected behind the first `keep` slots
    per = G * 2 * (B * D + 4) + 64
    return {"bytes": S * (n * 12 + keep * 12 + moved * per * 2), "flops": S * n * 2}


# ------------------------------------------------------------------ inputs
def _codes(shape, g, dev, sigma=120.0):
    """E4M3 codes of normal values: what a quantised K or V block holds."""
    out = torch.empty(shape, dtype=torch.uint8, device=dev)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        x = torch.randn(min(1 << 28, flat.numel() - i), generator=g, device=dev)
        flat[i:i + x.numel()] = (x * sigma).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    S, G = case["S"], case["G"]

    def scales(blocks):  # powers of two, as the append writes them
        e = torch.randint(-9, -5, (S, blocks, G, 2), generator=g, device=dev)
        return ((e.to(torch.int32) + 127) << 23).view(torch.float32)

    s = dict(case=dict(case))
    if case["op"] == "append":
        n, pos0 = case["n"], case["pos0"]
        blocks = (pos0 + n + B - 1) // B
        size = torch.rand((S, n, G, 1), generator=g, device=dev) * 2 + 0.25
        for x in ("k", "v"):
            s[x] = (torch.randn((S, n, G, D), generator=g, device=dev) * size).to(torch.bfloat16)
        s["tail"] = torch.randn((S, 2, B, G, D), generator=g, device=dev).to(torch.bfloat16)
        s["kv8"] = _codes((S, blocks, G, 2, B, D), g, dev)
        s["kv_scale"] = scales(blocks)
    elif case["op"] == "attn":
        nq, k, t0 = case["nq"], case["k"], case["q_pos0"]
        blocks = (t0 + nq + B - 1) // B
        s["kv8"] = _codes((S, blocks, G, 2, B, D), g, dev)
        s["kv_scale"] = scales(blocks)
        s["q"] = torch.randn((S, nq, G * HG, D), generator=g, device=dev).mul_(1.5).to(torch.bfloat16)
        # a selection: queries of a 64-query segment share most of their blocks
        hist = (t0 + nq - 1) // B
        t = torch.arange(t0, t0 + nq, device=dev)
        s["sel"] = torch.full((S, nq, G, k), -1, dtype=torch.int32, device=dev)
        s["cnt"] = torch.clamp(t // B, max=k).to(torch.int32).view(1, nq, 1).expand(S, nq, G).contiguous()
        if hist:
            base = torch.rand((S, (nq + 63) // 64, G, hist), generator=g, device=dev)
            x = base.repeat_interleave(64, 1)[:, :nq] + 0.2 * torch.rand((S, nq, G, hist), generator=g, device=dev)
            x.masked_fill_(torch.arange(hist, device=dev) >= (t // B).view(1, nq, 1, 1), -1.0)
            kk = min(k, hist)
            best, ids = x.topk(kk, -1)
            ids = torch.where(best >= 0, ids, hist).sort(-1).values
            s["sel"][..., :kk] = torch.where(ids < hist, ids, -1)
        s["gate"] = torch.randn((S, nq, G * HG), generator=g, device=dev).to(torch.bfloat16) if case["gate"] else None
        # weights that earlier calls accumulated
        s["acc"] = (torch.rand((S, blocks), generator=g, device=dev).double() * 2.0 ** 33).long() if case["weights"] else None
        s["out"] = torch.empty_like(s["q"])
    else:
        n, part = case["n"], case["part"]
        blocks = n + (part > 0)
        s["kv8"] = _codes((S, blocks, G, 2, B, D), g, dev)
        s["kv_scale"] = scales(blocks)
        s["store"] = _codes((S, blocks, 64), g, dev, 1.0)
        # attention weights fall off over many decades; some blocks are never attended, so ties occur
        w = torch.exp(3 * torch.randn((S, blocks), generator=g, device=dev).double())
        w[torch.rand((S, blocks), generator=g, device=dev) < 0.05] = 0
        s["acc"] = (w / FIX).long()
        # original block numbers of the slots an earlier eviction left behind, in no order
        known, seen = case["known"], case["known"] + case["evicted"]
        pos = torch.rand((S, max(seen, 1)), generator=g, device=dev).argsort(-1)[:, :known].to(torch.int32)
        s["pos"] = torch.cat([pos, torch.zeros((S, blocks - known), dtype=torch.int32, device=dev)], 1)
        s["acc_out"], s["pos_out"] = torch.empty_like(s["acc"]), torch.empty_like(s["pos"])
    return s


# ------------------------------------------------------------------ the framework's calls
def _run_own(s):
    from sparse_long_context_sgqa_b200 import binding as Bd
    c = s["case"]
    S, G = c["S"], c["G"]
    if "p" not in s:  # a program's parameters and workspace
        s["p"] = Bd.Params(num_kv_groups=G, topk=c.get("k", 512))
    p, cap = s["p"], s["kv8"].shape[1] * B
    if c["op"] == "append":
        Bd.sgqa_kv_append_q8(p, S, cap, c["pos0"], c["n"], s["k"], s["v"], s["tail"], s["kv8"], s["kv_scale"])
    elif c["op"] == "attn":
        if "ws" not in s:
            s["ws"] = Bd.alloc_workspace_q8(p, S, c["nq"], c["q_pos0"] + c["nq"], "cuda")
        Bd.sgqa_sparse_attn_q8(p, S, c["q_pos0"], c["nq"], s["q"], cap, c["q_pos0"] + c["nq"], s["kv8"], s["kv_scale"],
                               s["sel"], s["cnt"], s["out"], s["ws"], gate=s["gate"], acc=s["acc"])
    else:
        if "ws" not in s:
            s["ws"] = Bd.alloc_evict_workspace(p, S, cap, "cuda")
        Bd.sgqa_evict(p, S, cap, c["n"] * B + c["part"], c["keep"], c["first"], c["recent"], s["acc"], s["pos"],
                      c["known"], c["evicted"], s["acc_out"], s["pos_out"], [s["kv8"], s["kv_scale"], s["store"]], s["ws"])


# ------------------------------------------------------------------ plain forms
def _run_plain(s):
    c = s["case"]
    S, G, dev = c["S"], c["G"], s["kv8"].device
    if c["op"] == "append":
        n, pos0 = c["n"], c["pos0"]
        head, first, last = pos0 % B, pos0 // B, (pos0 + n - 1) // B
        rows = torch.cat([s["tail"][:, :, :head], torch.stack([s["k"], s["v"]], 1)], 2)
        x = torch.zeros((S, 2, (last - first + 1) * B, G, D), device=dev)
        x[:, :, :head + n] = rows.float()
        x = x.view(S, 2, -1, B, G, D).permute(0, 2, 4, 1, 3, 5)  # [S, block, G, K/V, token, D]
        amax = x.abs().amax((-2, -1))
        m, e = torch.frexp(amax / 448)
        e = (e - (m == 0.5).to(e.dtype)).clamp(min=-100)
        e = torch.where(amax > 0, e, -100)
        scale = ((e + 127) << 23).view(torch.float32)
        s["kv_scale"][:, first:last + 1] = scale
        s["kv8"][:, first:last + 1] = (x / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        left = (pos0 + n) % B
        s["tail"][:, :, :left] = rows[:, :, head + n - left:head + n]
    elif c["op"] == "attn":
        nq, k, t0 = c["nq"], c["k"], c["q_pos0"]
        t = torch.arange(t0, t0 + nq, device=dev).view(1, nq, 1, 1)
        cur = (t // B).expand(S, nq, G, 1)
        ids = torch.cat([s["sel"].long(), cur], -1)                       # [S, nq, G, k + 1]
        at = torch.arange(k + 1, device=dev)
        used = (at < s["cnt"][..., None]) | (at == k)
        tok = torch.arange(B, device=dev)
        valid = used[..., None] & ((at < k)[:, None] | (tok <= (t % B)[..., None]))  # [S, nq, G, k + 1, 8]
        ids = torch.where(used, ids, 0)
        si = torch.arange(S, device=dev).view(S, 1, 1, 1)
        gi = torch.arange(G, device=dev).view(1, 1, G, 1)
        sc = s["kv_scale"][si, ids, gi].repeat_interleave(B, -2)          # [S, nq, G, T, 2]
        K = s["kv8"][si, ids, gi, 0].view(torch.float8_e4m3fn).float().view(S, nq, G, -1, D)
        q = s["q"].float().view(S, nq, G, HG, D) * SCALE
        x = (q @ K.transpose(-1, -2)) * sc[..., 0].unsqueeze(-2)
        del K
        x.masked_fill_(~valid.view(S, nq, G, 1, -1), -torch.inf)
        x = (x - x.amax(-1, keepdim=True)).exp()
        w = x / x.sum(-1, keepdim=True)
        V = s["kv8"][si, ids, gi, 1].view(torch.float8_e4m3fn).float().view(S, nq, G, -1, D)
        o = ((w * sc[..., 1].unsqueeze(-2)) @ V).view(S, nq, G * HG, D)
        if s["gate"] is not None:
            o = o / (1 + (-s["gate"].float()).exp())[..., None]
        s["out"].copy_(o)
        if s["acc"] is not None:
            wb = w.sum(-2).view(S, nq, G, k + 1, B).sum(-1)               # weight of each block, over the heads
            fixed = (wb.double() / FIX).round().long()
            s["acc"].scatter_add_(1, ids.reshape(S, -1), fixed.view(S, -1))
    else:
        n, part, keep = c["n"], c["part"], c["keep"]
        slot = torch.arange(n, device=dev)
        pos = torch.where(slot < c["known"], s["pos"][:, :n], (slot + c["evicted"]).int())
        acc = s["acc"][:, :n]
        safe = (pos < c["first"]) | (pos >= n + c["evicted"] - c["recent"])
        by_pos = pos.sort(dim=-1, stable=True).indices                       # ties: the smaller original number stays
        rank = torch.where(safe, torch.iinfo(torch.int64).max, acc).gather(1, by_pos)
        order = by_pos.gather(1, rank.sort(dim=-1, descending=True, stable=True).indices)
        kept = torch.zeros((S, n), dtype=torch.bool, device=dev).scatter_(1, order[:, :keep], True)
        # the i-th free slot below `keep` takes the i-th kept block from behind it
        ar = slot.expand(S, n)
        hole = (~kept) & (slot < keep)
        late = kept & (slot >= keep)
        move_to = ar.masked_fill(~hole, n).sort(-1).values                # holes first, ascending
        move_from = ar.masked_fill(~late, n).sort(-1).values
        src = torch.cat([ar, ar[:, :1]], 1).scatter(1, move_to, move_from)[:, :keep]
        si = torch.arange(S, device=dev)[:, None]
        if part:
            src = torch.cat([src, torch.full((S, 1), n, device=dev)], 1)
        s["pos_out"][:, :keep] = pos.gather(1, src[:, :keep])
        s["acc_out"].zero_()
        s["acc_out"][:, :src.shape[1]] = s["acc"].gather(1, src)
        for x in ("kv8", "kv_scale", "store"):
            s[x][:, :src.shape[1]] = s[x][si, src]


def run(s):
    if own:
        _run_own(s)
    else:
        _run_plain(s)
    c = s["case"]
    e4m3 = torch.float8_e4m3fn
    if c["op"] == "append":
        first, last, left = c["pos0"] // B, (c["pos0"] + c["n"] - 1) // B, (c["pos0"] + c["n"]) % B
        return {"kv8": s["kv8"][:, first:last + 1].view(e4m3), "kv_scale": s["kv_scale"][:, first:last + 1],
                "tail": s["tail"][:, :, :left]}
    if c["op"] == "attn":
        return {"out": s["out"]} if s["acc"] is None else {"out": s["out"], "weights": s["acc"] * FIX}
    m = c["keep"] + (c["part"] > 0)
    return {"kv8": s["kv8"][:, :m].view(e4m3), "kv_scale": s["kv_scale"][:, :m], "store": s["store"][:, :m].view(e4m3),
            "acc": s["acc_out"], "pos": s["pos_out"][:, :c["keep"]]}


# ------------------------------------------------------------------ the definitions in 64 bits
def _e4m3_nearest(x):
    """E4M3 values nearest to x (|x| <= 448), ties to the even code."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))) / 8
    return torch.round(x / step) * step  # torch.round takes ties to even multiples


def exact(case, seed):
    if case["op"] == "evict":
        return None  # copies and whole numbers: nothing is computed
    s = prepare(case, seed)
    S, G = case["S"], case["G"]
    if case["op"] == "append":
        pos0, n = case["pos0"], case["n"]
        first, end = pos0 // B, pos0 + n
        codes, scales = [], []
        for name, at in (("k", 0), ("v", 1)):
            rows = torch.cat([s["tail"][:, at, :pos0 % B], s[name]], 1).double()
            rows = torch.nn.functional.pad(rows, (0, 0, 0, 0, 0, -(pos0 % B + n) % B))
            blk = rows.view(S, -1, B, G, D).transpose(2, 3)
            top = blk.abs().amax((3, 4)).clamp(min=448 * 2.0 ** -100)
            sc = torch.exp2(torch.ceil(torch.log2(top / 448)))
            sc = torch.where(sc / 2 * 448 >= top, sc / 2, sc)  # log2's own rounding
            sc = torch.where(sc * 448 < top, sc * 2, sc)
            codes.append(_e4m3_nearest(blk / sc[..., None, None]))
            scales.append(sc)
        left = end % B
        tail = s["tail"][:, :, :left].double()
        new = torch.stack([s["k"], s["v"]], 1).double()
        if left:
            fresh = min(left, n)
            tail[:, :, left - fresh:] = new[:, :, n - fresh:]
        return {"kv8": torch.stack(codes, 3), "kv_scale": torch.stack(scales, 3), "tail": tail}
    nq, k, t0 = case["nq"], case["k"], case["q_pos0"]
    out = torch.empty((S, nq, G, HG, D), dtype=torch.float64, device="cuda")
    acc = None if s["acc"] is None else s["acc"].double() * FIX
    step = max(1, (1 << 20) // ((k + 1) * B))  # queries at a time: at most about 2 GB of keys
    for b in range(S):
        for g in range(G):
            for i0 in range(0, nq, step):
                i1 = min(nq, i0 + step)
                t = torch.arange(t0 + i0, t0 + i1, device="cuda")
                ids = torch.cat([s["sel"][b, i0:i1, g].long(), (t // B)[:, None]], 1)
                live = torch.cat([torch.arange(k, device="cuda") < s["cnt"][b, i0:i1, g, None], (t >= 0)[:, None]], 1)
                ids = ids * live
                where = ids[..., None] * B + torch.arange(B, device="cuda")
                seen = live[..., None] & (where <= t[:, None, None])
                kv = s["kv8"][b, ids, g].view(torch.float8_e4m3fn).double() * s["kv_scale"][b, ids, g].double()[..., None, None]
                K, V = kv[:, :, 0].reshape(i1 - i0, -1, D), kv[:, :, 1].reshape(i1 - i0, -1, D)
                q = s["q"][b, i0:i1, g * HG:(g + 1) * HG].double()
                x = torch.einsum("qhd,qtd->qht", q, K) / math.sqrt(D)
                x = x.masked_fill(~seen.reshape(i1 - i0, 1, -1), -math.inf)
                w = torch.softmax(x, -1)
                out[b, i0:i1, g] = torch.einsum("qht,qtd->qhd", w, V)
                if acc is not None:
                    acc[b].index_add_(0, ids.reshape(-1), w.view(i1 - i0, HG, k + 1, B).sum((1, 3)).reshape(-1))
    out = out.view(S, nq, G * HG, D)
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"].double())[..., None]
    return {"out": out} if acc is None else {"out": out, "weights": acc}
