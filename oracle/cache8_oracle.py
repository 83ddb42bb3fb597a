"""float64 CPU oracle of the 8-bit KV cache (test infrastructure).

Codes are e4m3 bytes (sign, 4 exponent bits with bias 7, 3 fraction bits; 0x7F and 0xFF are NaN, there
is no infinity), scales powers of two, value = code * scale.  Everything is computed sequence by
sequence and head by head from the definitions.
"""

from __future__ import annotations

import math

import numpy as np


def e4m3_values() -> np.ndarray:
    """The 256 values a code stands for."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = math.nan if e == 15 and f == 7 else (f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
        out[c] = -v if c & 128 else v
    return out


VALUES = e4m3_values()
_POSITIVE = VALUES[:127]  # 0 .. 448, ascending


def encode(x) -> np.ndarray:
    """The code nearest to each x, |x| <= 448 (ties to the even code); NaN and infinities give 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    assert np.all(a <= 448.0)
    hi = np.minimum(np.searchsorted(_POSITIVE, a, side="left"), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.signbit(x), c + 128, c)
    return np.where(np.isfinite(x), c, 0x7F).astype(np.uint8)


def need(a: float) -> float:
    """The smallest 2^e, e >= -126, with a <= 448 * 2^e."""
    e = -126
    while a > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def _top(x) -> float:
    """Largest magnitude among the finite elements (0 if none)."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    x = x[np.isfinite(x)]
    return float(x.max()) if x.size else 0.0


def append(codes, scale, lens, new, block, at=None, counts=None):
    """(codes, scale, lens) of one of the two arrays after rows new [B, H, n, d] joined; bad sequences stay."""
    codes, scale, lens = codes.copy(), scale.copy(), lens.copy()
    B, H, n, _ = new.shape
    L = codes.shape[2]
    for b in range(B):
        p = int(lens[b] if at is None else at[b])
        m = int(n if counts is None else counts[b])
        if p < 0 or m < 0 or m > n or p + m > L:
            continue
        for h in range(H):
            for blk in range(p // block, (p + m - 1) // block + 1 if m else 0):
                r0, r1 = max(p, blk * block), min(p + m, (blk + 1) * block)
                rows = new[b, h, r0 - p: r1 - p].astype(np.float64)
                f = need(_top(rows))
                if blk * block < p:
                    f = max(f, float(scale[b, h, blk]))
                    ratio = float(scale[b, h, blk]) / f
                    if ratio != 1.0:
                        codes[b, h, blk * block: p] = encode(VALUES[codes[b, h, blk * block: p]] * ratio)
                codes[b, h, r0:r1] = encode(rows / f)
                scale[b, h, blk] = f
        lens[b] = p + m
    return codes, scale, lens


def values(codes, scale, block):
    """code * scale for one head: codes [L, d], scale [blocks]."""
    return VALUES[codes] * np.repeat(scale.astype(np.float64), block)[: codes.shape[0], None]


def _softmax(s):
    m = s.max()
    e = np.exp(s - m)
    return e / e.sum(), m + math.log(e.sum())


def attn(q, k, ks, v, vs, lens, block, back=0, scale=None):
    """q [B, Hq, nq, d].  Returns o, lse, w [B, Hkv, L] (the weight each token received) and, for error
    bounds, (a, a1, sk): a = sum_t p_t |v_t| and a1 = max_t p_t * sum_t |v_t| (like o), sk [B, Hq, nq] =
    scale * max over dims |q| * max_t sum over dims |k_t|."""
    B, Hq, nq, d = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    G = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    o, a, a1 = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    lse, sk = np.full((B, Hq, nq), -np.inf), np.zeros((B, Hq, nq))
    w = np.zeros((B, Hkv, L))
    for b in range(B):
        n = int(lens[b])
        n = max(n - back, 0) if 0 <= n <= L else 0
        for g in range(Hkv):
            kk, vv = values(k[b, g, :n], ks[b, g], block), values(v[b, g, :n], vs[b, g], block)
            for h in range(g * G, (g + 1) * G):
                for i in range(nq):
                    m = n - (nq - 1 - i)
                    if m <= 0:
                        continue
                    qq = q[b, h, i].astype(np.float64)
                    p, lse[b, h, i] = _softmax(scale * (kk[:m] @ qq))
                    o[b, h, i], a[b, h, i] = p @ vv[:m], p @ np.abs(vv[:m])
                    a1[b, h, i] = p.max() * np.abs(vv[:m]).sum(0)
                    sk[b, h, i] = scale * np.abs(qq).max() * np.abs(kk[:m]).sum(-1).max()
                    w[b, g, :m] += p
    return o, lse, w, (a, a1, sk)


def attn_list(q, k, ks, v, vs, lens, idx, block, scale=None):
    """q [B, Hq, d], idx [B, Hq, k]: o, lse, (a, a1, sk) as attn; a row with an entry outside [-1, lens) is empty."""
    B, Hq, d = q.shape
    G = Hq // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o, a, a1 = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    lse, sk = np.full((B, Hq), -np.inf), np.zeros((B, Hq))
    for b in range(B):
        for h in range(Hq):
            t = idx[b, h]
            if np.any(t < -1) or np.any(t >= lens[b]):
                continue
            t = t[t >= 0]
            if t.size == 0:
                continue
            kk, vv = values(k[b, h // G], ks[b, h // G], block)[t], values(v[b, h // G], vs[b, h // G], block)[t]
            qq = q[b, h].astype(np.float64)
            p, lse[b, h] = _softmax(scale * (kk @ qq))
            o[b, h], a[b, h], a1[b, h] = p @ vv, p @ np.abs(vv), p.max() * np.abs(vv).sum(0)
            sk[b, h] = scale * np.abs(qq).max() * np.abs(kk).sum(-1).max()
    return o, lse, (a, a1, sk)


def kept_tokens(weight, n: int, keep: int, recent: int) -> list[int]:
    """The rows eviction keeps of one head: weights [L], n tokens held."""
    if n <= keep:
        return list(range(n))
    old = n - recent
    # NaN above everything; equal weights (0.0 == -0.0) by the lower row
    order = sorted(range(old), key=lambda t: (0 if math.isnan(weight[t]) else 1, 0.0 if math.isnan(weight[t])
                                              else -float(weight[t]), t))
    return sorted(order[: keep - recent]) + list(range(old, n))


def evict(k, ks, v, vs, lens, weight, block, keep, recent, dst):
    """dst: dict of the destination's arrays k, ks, v, vs, lens, weight (copied, then written); returns it and idx."""
    B, H, L, _ = k.shape
    dst = {n: x.copy() for n, x in dst.items()}
    idx = np.full((B, H, keep), -1, dtype=np.int32)
    for b in range(B):
        n = int(lens[b]) if 0 <= lens[b] <= L else 0
        dst["lens"][b] = min(n, keep)
        for h in range(H):
            t = kept_tokens(weight[b, h], n, keep, recent)
            idx[b, h, : len(t)] = t
            dst["weight"][b, h, : len(t)] = weight[b, h, t]
            for codes, scale, dc, ds in ((k, ks, "k", "ks"), (v, vs, "v", "vs")):
                for r0 in range(0, len(t), block):
                    tt = np.asarray(t[r0: r0 + block])
                    x = VALUES[codes[b, h, tt]] * scale[b, h, tt // block].astype(np.float64)[:, None]
                    f = need(_top(x))
                    dst[dc][b, h, r0: r0 + len(tt)] = encode(x / f)
                    dst[ds][b, h, r0 // block] = f
    return dst, idx


def fc_gather(codes, scale, fc, block):
    """Values of the dominant dims [B, H, L, 2 nfc]: pairs' low dims, then their partners."""
    B, H, L, d = codes.shape
    out = np.empty((B, H, L, 2 * fc.shape[1]))
    for b in range(B):
        for h in range(H):
            x = values(codes[b, h], scale[b, h], block)
            out[b, h] = x[:, np.concatenate([fc[h], fc[h] + d // 2])]
    return out
