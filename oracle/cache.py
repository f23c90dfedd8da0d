"""Attention over a serving cache of grouped heads, and eviction from it: the
definitions, one sequence at a time, in float64.

Query head h reads key head h // G, G = H / Hkv.  The query at position p sees
key j if j <= p and (window == 0 or j > p - window or j < sinks).
"""

import numpy as np


def visible(p, window, sinks):
    """The keys that a query at position ``p`` sees, in order."""
    j = np.arange(p + 1)
    return j if window == 0 else j[(j > p - window) | (j < sinks)]


def attend(q, k, v, scale):
    """One row q [D] over keys k [n, D]: out [D], lse, weights [n] (0, -inf without keys)."""
    if k.shape[0] == 0:
        return np.zeros(v.shape[1]), -np.inf, np.zeros(0)
    s = scale * (k @ q)
    m = s.max()
    e = np.exp(s - m)
    total = e.sum()
    return (e / total) @ v, m + np.log(total), e / total


def decode(q, k, v, lens, scale, window=0, sinks=0, kp=None, vp=None):
    """q [B, H, D], k, v [B, Hkv, cap, D], lens [B]; kp, vp [Hkv, P, D] shared by all sequences
    and in front of their own keys.  Returns out [B, H, D], lse [B, H] and each key's weights
    summed over its group's heads, [B, Hkv, cap] (own keys only)."""
    B, H, D = q.shape
    Hkv, cap = k.shape[1], k.shape[2]
    out, lse = np.zeros((B, H, v.shape[3])), np.full((B, H), -np.inf)
    weight = np.zeros((B, Hkv, cap))
    for b in range(B):
        n = int(lens[b])
        keys = visible(n - 1, window, sinks)
        for h in range(H):
            hk = h // (H // Hkv)
            kk, vv = k[b, hk, keys], v[b, hk, keys]
            if kp is not None:
                kk, vv = np.concatenate([kp[hk], kk]), np.concatenate([vp[hk], vv])
            out[b, h], lse[b, h], w = attend(q[b, h], kk, vv, scale)
            weight[b, hk, keys] += w[len(w) - len(keys):]
    return out, lse, weight


def prefill_row(q, k, v, p, scale, window, sinks):
    """The query q [D] at position p over one key head's k, v [L, D]: out [D] and lse."""
    keys = visible(p, window, sinks)
    return attend(q, k[keys], v[keys], scale)[:2]


def kept_rows(weight, n, keep, sinks, recent):
    """Rows of a sequence of n that stay, ascending: the first ``sinks``, the last ``recent`` and
    the heaviest between (equal weights: lower index first; NaN below every number)."""
    if n <= keep:
        return np.arange(n)
    first = min(sinks, n)
    last = max(first, n - recent)
    need = keep - first - (n - last)
    w = weight[first:last].astype(np.float64)
    nan = np.isnan(w)
    order = np.lexsort((np.arange(last - first), -np.where(nan, 0.0, w), nan))
    return np.sort(np.concatenate([np.arange(first), first + order[:need], np.arange(last, n)]))


def score_error(q, k, scale):
    """How far an fp32 score of 16-bit rows can be from its value: each of the D products is exact
    in fp32; the D additions and the multiplication by the scale each lose up to 2^-23 of the
    sum of magnitudes (truncating additions included).  q [..., D], k [n, D]: the largest."""
    D = q.shape[-1]
    if k.shape[0] == 0:
        return 0.0
    return (D + 4) * 2.0 ** -23 * abs(scale) * float((np.abs(q) @ np.abs(k).T).max())
