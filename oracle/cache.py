"""fp64 CPU oracle of the 8-bit page-scaled cache: append, attention, eviction.

TEST INFRASTRUCTURE (see ``oracle/__init__.py``).  numpy arrays in and out; E4M3 is held as bytes.
Written from the definitions in the C header: a byte x of page p and KV head h is e4m3(x) * scale[p][h];
an appended page's scale is the smallest power of two (at least 2^-64) that brings its largest value to
448 or less; attention is the softmax over a query's visible tokens; eviction drops the lowest scores.
"""
from __future__ import annotations

import math

import numpy as np

D = 128


def _decode_table() -> np.ndarray:
    """The 256 E4M3 values: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    t = np.empty(256, np.float64)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        t[b] = math.nan if (b & 127) == 127 else (-v if b & 128 else v)
    return t


TABLE = _decode_table()
_POS = TABLE[:127]  # ascending magnitudes, byte = index


def encode(x: np.ndarray) -> np.ndarray:
    """E4M3 bytes of x, rounded to nearest (ties to the even byte), saturating at 448; NaN and
    infinities become 0x7f."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x)
    a = np.minimum(np.abs(np.where(bad, 0.0, x)), 448.0)
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POS[hi] - a, a - _POS[lo]
    pick = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    b = pick | np.where(np.signbit(x), 128, 0)
    return np.where(bad, 127, b).astype(np.uint8)


def page_scale(amax: float) -> float:
    """The smallest 2^k, k >= -64, with amax <= 448 * 2^k."""
    if amax <= 0:
        return 2.0 ** -64
    m, e = math.frexp(amax)
    return 2.0 ** max(-64, e - 9 if m <= 0.875 else e - 8)


def append(cache, scale, new, page_table, page_ptr, kv_len, tok_ptr):
    """(cache, scale) with the new tokens: cache uint8 [P][Hkv][T][D], scale fp32 [P][Hkv], new [N][Hkv][D]."""
    cache, scale = cache.copy(), scale.astype(np.float32).copy()
    T = cache.shape[2]
    for r in range(len(kv_len)):
        n = tok_ptr[r + 1] - tok_ptr[r]
        at = kv_len[r] - n
        while at < kv_len[r]:
            end = min(kv_len[r], (at // T + 1) * T)
            p = page_table[page_ptr[r] + at // T]
            x = new[tok_ptr[r] + at - (kv_len[r] - n):][:end - at].astype(np.float64)
            a = at % T
            for h in range(cache.shape[1]):
                y = x[:, h]
                fin = np.abs(y[np.isfinite(y)])
                s = page_scale(float(fin.max()) if fin.size else 0.0)
                old = float(scale[p, h])
                if a:
                    s = max(s, old)
                    if s != old:
                        cache[p, h, :a] = encode(TABLE[cache[p, h, :a]] * (old / s))
                cache[p, h, a:a + end - at] = encode(y / s)
                scale[p, h] = s
            at = end
    return cache, scale


def attn(q, K, V, k_scale, v_scale, page_table, page_ptr, kv_len, q_ptr, softmax_scale, topk=None):
    """O, lse, page weights, and for error bounds, per (row, head): smag, the largest sum |q||k| of a visible
    token, qk, the largest max|q| sum|k| (both scaled), vtop, the largest |v|, and per element vmag, the
    weighted mean of |v|.  q [N][Hq][D] float64."""
    N, Hq, _ = q.shape
    Hkv, T = K.shape[1], K.shape[2]
    g = Hq // Hkv
    O = np.zeros((N, Hq, D))
    lse = np.full((N, Hq), -np.inf)
    weight = np.zeros((len(page_table), Hkv))
    smag = np.zeros((N, Hq))
    vmag = np.zeros((N, Hq, D))
    vtop = np.zeros((N, Hq))
    qk = np.zeros((N, Hq))
    for r in range(len(kv_len)):
        n, L = q_ptr[r + 1] - q_ptr[r], kv_len[r]
        if n == 0 or L == 0:
            continue
        pages = -(-L // T)
        phys = page_table[page_ptr[r]:page_ptr[r] + pages]
        for h in range(Hkv):
            k = (TABLE[K[phys, h]] * k_scale[phys, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:L]
            v = (TABLE[V[phys, h]] * v_scale[phys, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:L]
            for i in range(n):
                row = q_ptr[r] + i
                end = L - n + i + 1
                if end <= 0:
                    continue
                for j in range(g):
                    hq = h * g + j
                    tok = np.arange(end)
                    if topk is not None:
                        sel = topk[hq, row]
                        tok = tok[np.isin(tok // T, sel[sel >= 0])]
                    if tok.size == 0:
                        continue
                    s = (k[tok] @ q[row, hq]) * softmax_scale
                    m = s.max()
                    with np.errstate(invalid="ignore"):  # an infinite score
                        e = np.exp(s - m)
                    lse[row, hq] = m + math.log(e.sum()) if np.isfinite(e.sum()) else math.nan
                    p = e / e.sum()
                    O[row, hq] = p @ v[tok]
                    np.add.at(weight[:, h], page_ptr[r] + tok // T, p)
                    smag[row, hq] = (np.abs(k[tok]) @ np.abs(q[row, hq])).max() * softmax_scale
                    vmag[row, hq] = p @ np.abs(v[tok])
                    vtop[row, hq] = np.abs(v[tok]).max()
                    qk[row, hq] = np.abs(q[row, hq]).max() * np.abs(k[tok]).sum(axis=1).max() * softmax_scale
    return dict(o=O, lse=lse, weight=weight, smag=smag, vmag=vmag, vtop=vtop, qk=qk)


def evict(page_table, acc, weight, page_ptr, kv_len, T, budget, sink, recent, decay):
    """(page_table, acc, kv_len, page_src) after the eviction; scores rounded once to fp32."""
    table, acc_o = page_table.copy(), acc.astype(np.float32).copy()
    lens, src = kv_len.copy(), np.zeros(len(page_table), np.int32)
    for r in range(len(kv_len)):
        b, e = page_ptr[r], page_ptr[r + 1]
        used = -(-kv_len[r] // T)
        score = (decay * acc[b:b + used].astype(np.float64) +
                 weight[b:b + used].astype(np.float64).sum(axis=1)).astype(np.float32)
        free = list(range(min(sink, used), max(min(sink, used), used - recent)))
        order = sorted(free, key=lambda p: (np.isnan(score[p]), score[p] if not np.isnan(score[p]) else 0.0, p))
        gone = sorted(order[:max(0, used - budget)])
        kept = [p for p in range(used) if p not in set(gone)]
        new = kept + gone + list(range(used, e - b))
        table[b:e] = page_table[b:e][new]
        acc_o[b:e] = [score[p] if p < used and p not in set(gone) else (0.0 if p < used else acc[b + p]) for p in new]
        src[b:e] = new
        lens[r] = kv_len[r] - len(gone) * T
    return table, acc_o, lens, src
