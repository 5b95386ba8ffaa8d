"""The serving operators restated in float64 numpy, straight from their
definitions (no code in common with the CUDA path):

* ``decode``: attention of new tokens over a shared prefix and their caches;
* ``key_weight``: accumulated attention weight of each cached key;
* ``evict``: which entries of a cache stay, and where they go.
"""

from __future__ import annotations

import math

import numpy as np


def decode(q, k_cache, v_cache, cache_len, k_prefix=None, v_prefix=None, prefix_len=None):
    """Returns (out, lse, spread, lsum): ``spread`` = sum_j p_j |v_j| per
    output element (what a relative error of every term can move it by) and
    ``lsum`` = (sum_j e^{s_j - max}, sum_j |v_j|) for absolute term errors.
    Row by row, keys masked by leaving them out."""
    B, Hq, T, d = q.shape
    k0 = k_cache if k_cache is not None else k_prefix
    Hkv = k0.shape[1]
    G = Hq // Hkv
    Bp = k_prefix.shape[0] if k_prefix is not None else 1
    out = np.zeros((B, Hq, T, d))
    lse = np.full((B, Hq, T), -np.inf)
    spread = np.zeros((B, Hq, T, d))
    tiny = np.zeros((B, Hq, T, d))
    for b in range(B):
        for h in range(Hq):
            g = h // G
            for t in range(T):
                ks, vs = [], []
                if k_prefix is not None:
                    p = b // (B // Bp)
                    ks.append(k_prefix[p, g, :prefix_len[p]])
                    vs.append(v_prefix[p, g, :prefix_len[p]])
                if k_cache is not None:
                    n = max(0, cache_len[b] - (T - 1 - t))
                    ks.append(k_cache[b, g, :n])
                    vs.append(v_cache[b, g, :n])
                kk, vv = np.concatenate(ks), np.concatenate(vs)
                if len(kk) == 0:
                    continue
                s = kk @ q[b, h, t] / math.sqrt(d)
                m = s.max()
                e = np.exp(s - m)
                out[b, h, t] = e @ vv / e.sum()
                lse[b, h, t] = m + math.log(e.sum())
                spread[b, h, t] = e @ np.abs(vv) / e.sum()
                tiny[b, h, t] = np.abs(vv).sum(0) / e.sum()
    return out, lse, spread, tiny


def key_weight(q, k, lse, key_len, causal, score=None):
    """Returns (score_out, mass): ``mass`` is the weight added."""
    B, Hq, T, d = q.shape
    Bk, Hkv, C, _ = k.shape
    n, G = B // Bk, Hq // Hkv
    mass = np.zeros((Bk, Hkv, C))
    for b in range(B):
        for h in range(Hq):
            for t in range(T):
                seen = key_len[b // n] - (T - 1 - t) if causal else key_len[b // n]
                if seen <= 0 or lse[b, h, t] == -np.inf:
                    continue
                s = k[b // n, h // G, :seen] @ q[b, h, t] / math.sqrt(d)
                mass[b // n, h // G, :seen] += np.exp(s - lse[b, h, t])
    out = mass.copy()
    if score is not None:
        out += score
    for b in range(Bk):
        out[b, :, max(0, key_len[b]):] = 0.0
    return out, mass


def evict(score, pos, cache_len, budget, sink, recent):
    """Returns (kept [B, Hkv, budget], new lengths [B]): the source slot of
    every kept entry, -1 past the new length."""
    B, H, C = score.shape
    kept = np.full((B, H, budget), -1, dtype=np.int64)
    lens = np.zeros(B, dtype=np.int64)
    for b in range(B):
        m = int(cache_len[b])
        nk = min(m, budget)
        lens[b] = nk
        for h in range(H):
            if m <= budget:
                kept[b, h, :m] = np.arange(m)
                continue
            ps = pos[b, h, :m] if pos is not None else np.arange(m)
            last = int(ps.max())

            def rank(i):
                s = float(score[b, h, i])
                safe = ps[i] < sink or int(ps[i]) > last - recent
                return (0 if safe else 1, math.inf if math.isnan(s) else -s, i)

            stay = sorted(sorted(range(m), key=rank)[:nk])
            inside = set(i for i in stay if i < nk)
            late = [i for i in stay if i >= nk]
            for i in range(nk):
                kept[b, h, i] = i if i in inside else late.pop(0)
    return kept, lens
