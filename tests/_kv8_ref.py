"""Plain 64-bit implementations (numpy, CPU) of the 8-bit cache's operators, for the tests.  They share no code with the
CUDA path."""
from __future__ import annotations

import math

import numpy as np
import torch

D, HG, B = 192, 16, 8
UNIT = 2.0 ** -32


def codes_to_values(codes: torch.Tensor) -> np.ndarray:
    return codes.cpu().view(torch.float8_e4m3fn).to(torch.float64).numpy()


def _nearest_e4m3():
    """All non-negative E4M3 values, ascending; index = code."""
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


E4M3 = _nearest_e4m3()


def e4m3_codes(x: np.ndarray) -> np.ndarray:
    """Codes nearest to x (|x| <= 448), ties to the even code; x = -0 keeps its sign."""
    a = np.abs(x)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up = E4M3[hi] - a
    down = a - E4M3[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(a == E4M3[hi], hi, code)
    return (code | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8)


def scale_of(amax: float) -> float:
    if amax == 0:
        return 2.0 ** -100
    e = math.frexp(amax / 448.0)
    return 2.0 ** max(-100, e[1] - 1 if e[0] == 0.5 else e[1])


def quantise_rows(rows: np.ndarray):
    """rows [n, G, D] of one sequence from position 0: codes [blocks, G, 8, D] (uint8) and scales [blocks, G]."""
    n, G, _ = rows.shape
    nb = -(-n // B)
    codes = np.zeros((nb, G, B, D), np.uint8)
    scales = np.zeros((nb, G))
    for r in range(nb):
        for g in range(G):
            x = rows[r * B:(r + 1) * B, g]
            if not np.isfinite(x).all():
                scales[r, g] = np.nan
                continue
            s = scale_of(np.abs(x).max())
            scales[r, g] = s
            codes[r, g, :x.shape[0]] = e4m3_codes(x / s)
    return codes, scales


def attention(q, kv8, scale, sel, cnt, q_pos0, gate=None):
    """q [S, nq, G*16, D], kv8 [S, blocks, G, 2, 8, D] values, scale [S, blocks, G, 2], sel [S, nq, G, k] (numpy, float64):
    out, the tolerance of out (below) and weights [S, blocks].

    Tolerance: 2^-8 |out| for the result's rounding to BF16, 2^-8 sum w |v| for the weights, 2^-10 sum w |v| for scores,
    exponentials and sums, and what is below the smallest weight a row resolves.  A weight w enters the product as w vs
    (vs: its V scale) in units in which the row's largest is at least 2^4: as FP16, whose smallest step there is 2^-24, or
    as three E5M2 values, the last in steps of 2^-22; so it is off by up to 2^-27 of the row's largest w vs, times its code."""
    S, nq = q.shape[:2]
    G = kv8.shape[2]
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    weights = np.zeros(kv8.shape[:2])
    for b in range(S):
        for i in range(nq):
            t = q_pos0 + i
            for g in range(G):
                ids = [int(x) for x in sel[b, i, g, :cnt[b, i, g]]] + [t // B]
                K = kv8[b, ids, g, 0] * scale[b, ids, g, 0][:, None, None]
                V = kv8[b, ids, g, 1] * scale[b, ids, g, 1][:, None, None]
                n = len(ids) * B - (B - 1 - t % B)  # the current block only up to t
                K, V = K.reshape(-1, D)[:n], V.reshape(-1, D)[:n]
                s = q[b, i, g * HG:(g + 1) * HG] @ K.T / math.sqrt(D)
                w = np.exp(s - s.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                out[b, i, g * HG:(g + 1) * HG] = w @ V
                vs = np.repeat(scale[b, ids, g, 1], B)[:n]
                floor = 2.0 ** -27 * (w * vs).max(1)[:, None] * np.abs(V / vs[:, None]).sum(0)
                spread[b, i, g * HG:(g + 1) * HG] = (2.0 ** -8 + 2.0 ** -10) * (w @ np.abs(V)) + floor
                per = np.zeros(len(ids) * B)
                per[:n] = w.sum(0)
                np.add.at(weights[b], ids, per.reshape(-1, B).sum(1))
    if gate is not None:
        f = 1.0 / (1.0 + np.exp(-gate))[..., None]
        out, spread = out * f, spread * f
    return out, 2.0 ** -8 * np.abs(out) + spread + 1e-30, weights


def check_out(got, ref, tol):
    got = got.cpu().double().numpy()
    assert np.isfinite(got).all()
    off = np.abs(got - ref) / tol
    at = np.unravel_index(off.argmax(), off.shape)
    assert off.max() <= 1, (off.max(), at, got[at], ref[at], int((off > 1).sum()))


def evict(n, part, keep, first, recent, acc, pos, known, evicted):
    """One sequence: source slot of every new slot (the incomplete block's last), weights and original numbers."""
    number = [int(pos[s]) if s < known else s + evicted for s in range(n)]
    safe = [p < first or p >= n + evicted - recent for p in number]
    order = sorted(range(n), key=lambda s: (not safe[s], 0 if safe[s] else -int(acc[s]), number[s]))
    kept = set(order[:keep])
    holes = [s for s in range(keep) if s not in kept]
    late = [s for s in range(keep, n) if s in kept]
    src = list(range(keep))
    for h, m in zip(holes, late):
        src[h] = m
    src = src + ([n] if part else [])
    new_acc = np.zeros(len(acc), np.int64)
    new_acc[:len(src)] = [acc[s] for s in src]
    return src, new_acc, [number[s] for s in src[:keep]]
