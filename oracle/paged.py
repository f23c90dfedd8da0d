"""A serving step over a paged cache: the definitions, request by request, in float64.

Pages hold ``page`` rows of every key head, kp and vp [P, Hkv, page, D]; table [B, width] lists each
request's pages in order.
"""

import numpy as np

from . import cache


def pages(n, page):
    return -(-n // page)


def page_tables(lens, news, table, stack, n_free, page, tokens):
    """One request after the other.  Returns starts, positions, slots, the new lengths, the number of
    free pages left, the table and the stack."""
    table, stack = np.array(table), np.array(stack)
    B, width = table.shape
    n = min(max(int(n_free), 0), len(stack))
    lens = [max(0, int(x)) for x in lens]
    held = [min(pages(x, page), width) for x in lens]
    for b in range(B):
        if news[b] < 0:
            for i in range(held[b]):
                if n < len(stack):
                    stack[n] = table[b, i]
                    n += 1
    starts, positions, slots, lens_out, dry = [0], [], [], [], False
    for b in range(B):
        if news[b] < 0:
            lens_out.append(0)
            starts.append(starts[-1])
            continue
        new = int(news[b])
        total = pages(lens[b] + new, page)
        fits = total <= width
        if fits and total > held[b] and (dry or total - held[b] > n):
            fits, dry = False, True
        for i in range(held[b], total if fits else held[b]):
            n -= 1
            table[b, i] = stack[n]
        lens_out.append(lens[b] + new if fits else lens[b])
        starts.append(starts[-1] + new)
        for p in range(lens[b], lens[b] + new):
            positions.append(p)
            slots.append(table[b, p // page] * page + p % page if fits else -1)
    positions = (positions + [0] * tokens)[:tokens]
    slots = (slots + [-1] * tokens)[:tokens]
    return (np.array(starts), np.array(positions), np.array(slots), np.array(lens_out), n, table, stack)


def norm_rope(x, weight, eps, positions, freq, axis=None, interleaved=False):
    """x [T, heads, D], positions [axes, T], freq [R / 2], axis [R / 2]: normed (with a weight), then
    rotated.  Returns the result and, for error bounds, the size |a| + |b| of each value's pair."""
    x = np.asarray(x, np.float64)
    y = x if weight is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    R = 2 * len(freq)
    axis = np.zeros(R // 2, int) if axis is None else np.clip(axis, 0, len(positions) - 1)
    out, size = y.copy(), np.abs(y)
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        t = positions[axis[i]].astype(np.float64)[:, None] * float(freq[i])
        out[..., a] = y[..., a] * np.cos(t) - y[..., b] * np.sin(t)
        out[..., b] = y[..., b] * np.cos(t) + y[..., a] * np.sin(t)
        size[..., a] = size[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, size


def gather(pages_of, table_row, n):
    """Rows 0 .. n - 1 of a request, [Hkv, n, D]; a page outside the cache reads as zeros."""
    P, Hkv, page, D = pages_of.shape
    out = np.zeros((Hkv, n, D))
    for i in range(pages(n, page)):
        rows = min(page, n - i * page)
        if 0 <= table_row[i] < P:
            out[:, i * page:i * page + rows] = pages_of[table_row[i], :, :rows]
    return out


def attend(q, kp, vp, table, starts, lens, scale, window=0, sinks=0):
    """q [T, H, D]: out [T, H, D] and lse [T, H]; NaN in rows that belong to no request."""
    T, H, D = q.shape
    G = H // kp.shape[1]
    out, lse = np.full((T, H, D), np.nan), np.full((T, H), np.nan)
    for b in range(len(lens)):
        L, N = int(lens[b]), int(starts[b + 1] - starts[b])
        k, v = gather(kp, table[b], L), gather(vp, table[b], L)
        for i in range(N):
            keys = cache.visible(L - N + i, window, sinks) if L - N + i >= 0 else []
            for h in range(H):
                out[starts[b] + i, h], lse[starts[b] + i, h], _ = cache.attend(
                    q[starts[b] + i, h], k[h // G][keys], v[h // G][keys], scale)
    return out, lse
