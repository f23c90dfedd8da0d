"""Inputs for the tests of the calls over a paged cache."""

import random

import numpy as np
import torch


def tables(B, page, held, width, free, seed, spare=2):
    """A pool whose pages are scattered: table [B, width] (-1 behind the pages in use), the stack of
    ``free`` free ones (and -1 above) and the number of pages."""
    rng = random.Random(seed)
    P = sum(held) + free + spare
    ids = rng.sample(range(P), P)
    table, at = np.full((B, width), -1, np.int32), 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    stack = np.full(P, -1, np.int32)
    stack[:free] = ids[at:at + free]
    return table, stack, P


def i32(x, dev="cuda"):
    return torch.tensor(np.asarray(x, np.int32), device=dev)


def paged_cache(lens, Hkv, page, seed, dtype=torch.bfloat16, D=128, width=None, fill=float("nan")):
    """kp, vp [P, Hkv, page, D] and a table of requests of ``lens`` keys; rows that no request uses
    hold ``fill``."""
    held = [-(-n // page) for n in lens]
    table, _, P = tables(len(lens), page, held, width or max(max(held), 1), 0, seed)
    g = torch.Generator().manual_seed(seed)
    pages = []
    for _ in range(2):
        x = torch.full((P, Hkv, page, D), fill, dtype=dtype)
        for b, n in enumerate(lens):
            rows = torch.randn(Hkv, n, D, generator=g).to(dtype)
            for i in range(held[b]):
                m = min(page, n - i * page)
                x[table[b, i], :, :m] = rows[:, i * page:i * page + m]
        pages.append(x)
    return pages[0], pages[1], table


def few_rows(B, H, Hkv, max_new, max_len, sms=None):
    """Rows per key head (new tokens * H / Hkv) up to which a request of a call of these sizes has its
    weights in two 16-bit terms, as the header file documents it."""
    sms = sms or torch.cuda.get_device_properties(0).multi_processor_count
    G = H // Hkv
    if max_new * G <= 64 and B * Hkv * -(-max_new * G // 16) * -(-max_len // 64) <= 32 * sms:
        return 64
    return min(64, 32 * G // max(g for g in (8, 4, 2, 1) if G % g == 0))
