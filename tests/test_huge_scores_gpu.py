"""Scores of any finite size, in the calls over a serving cache; of up to 2^31 in the causal prefill.

Rows of q hold one value, a power of two, and keys one of 129 .. 255 units, so that scores are whole
multiples of a large unit, exact in fp32 (and not in log2 units); two that differ do so by a thousand.  So a row's weights are equal on the keys
of its highest score and 0 elsewhere: out is the mean of their values, lse the score plus the logarithm of
their number.

Tolerance: the weight of a highest score is 1 but for the rounding of the score in log2 units, the same for
all of them; its rounding to 16 bits and that of the output are half a step each; the sum, its inverse and the
product less than 2^-19.  lse: the scale in log2 units, the score and the logarithm, each rounded to
fp32, less than 2^-21 of the score."""

import math

import numpy as np
import pytest
import torch

import cascaded_reductions_gb300 as rf
from cache_helpers import DT, HALF_STEP, assert_within
from helpers import f64
from oracle import cache as C
from paged_helpers import i32, tables

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5
# of q's values and of a key's unit: scores up to 2^33 in fp16, 2^118 in bf16, in log2 units
GAINS = {"bf16": (2.0 ** 46, [1.0, 2.0 ** 20, 2.0 ** 60]), "fp16": (2.0 ** 7, [1.0, 2.0 ** 8, 2.0 ** 15])}


def queries(dtype, seed, *shape):
    gains = np.array(GAINS[dtype][1])
    rng = np.random.default_rng(seed)
    x = gains[rng.integers(0, len(gains), shape)] * rng.choice([-1.0, 1.0], shape)
    return torch.from_numpy(np.repeat(x[..., None], 128, -1)).to(DT[dtype])


def keys(dtype, seed, *shape):
    rng = np.random.default_rng(seed)
    x = GAINS[dtype][0] * rng.integers(129, 256, shape)
    return torch.from_numpy(np.repeat(x[..., None], 128, -1)).to(DT[dtype])


def values(dtype, seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).integers(-8, 9, (*shape, 128)) / 8.0).to(DT[dtype])


def check_row(out, lse, q, k, v, what):
    """One row against keys k and values v [n, 128], all float64; ``out`` in the type of the result."""
    s = k[:, 0] * q[0] * 128
    top = s == s.max()
    mean = v[top].mean(0)
    assert_within(f64(out), mean, (2.01 * HALF_STEP[out.dtype]) * np.abs(mean) + 2.0 ** -19, what)
    want = s.max() * SCALE + math.log(top.sum())
    assert_within(f64(lse), want, 2.0 ** -21 * abs(want) + 2.0 ** -16, "lse " + what)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5)])
@pytest.mark.parametrize("B,news,max_len", [(6, 1, 640), (6, 3, 640), (80, 2, 9600), (6, 70, 640), (3, 300, 640)])
def test_paged(B, news, max_len, window, sinks, dtype):
    """Small calls, a queue of units, the pair kernel, whole and in parts."""
    H, Hkv, page = 8, 2, 32
    lens = [news + (97 * b) % 330 for b in range(B)]
    table, _, P = tables(B, page, [-(-n // page) for n in lens], max_len // page, 0, 1)
    kp, vp = keys(dtype, 2, P, Hkv, page), values(dtype, 3, P, Hkv, page)
    q = queries(dtype, 4, B * news, H)
    plan = rf.paged_plan(i32(np.arange(B + 1) * news), i32(lens), B * news, H, Hkv, news, max_len, window, sinks)
    out, lse = rf.attn_paged(q.cuda(), kp.cuda(), vp.cuda(), i32(table), plan)
    out, lse = out.cpu(), lse.cpu()
    for b, L in enumerate(lens):
        at = np.arange(L)
        kd, vd = (f64(x[table[b, at // page], :, at % page]) for x in (kp, vp))       # [L, Hkv, 128]
        for i in sorted({0, 1 % news, 33 % news, news - 1}):
            seen = C.visible(L - news + i, window, sinks)
            for h in range(H):
                check_row(out[b * news + i, h], lse[b * news + i, h], f64(q[b * news + i, h]), kd[seen, h // 4],
                          vd[seen, h // 4], f"request {b}, row {i}, head {h}")
    assert rf.rf_device_error() == 0


def test_paged_parts_of_a_tile():
    """One tile over many keys, cut between clusters, whose parts have maxima that differ hugely."""
    L, news, page = 20000, 65, 64
    n = -(-L // page)
    kp, vp = keys("bf16", 2, n, 1, page), values("bf16", 3, n, 1, page)
    kp[: n // 2] = -kp[: n // 2]
    q = queries("bf16", 4, news, 4)
    table = torch.arange(n, dtype=torch.int32)[None]
    plan = rf.paged_plan(i32([0, news]), i32([L]), news, 4, 1, news, n * page)
    out, lse = rf.attn_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), plan)
    kd, vd = (f64(x).reshape(-1, 128) for x in (kp, vp))
    for i in (0, 31, 64):
        for h in range(4):
            check_row(out[i, h].cpu(), lse[i, h].cpu(), f64(q[i, h]), kd[:L - news + i + 1], vd[:L - news + i + 1],
                      f"row {i}, head {h}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5), (257, 100)])
@pytest.mark.parametrize("N,L", [(20, 40), (700, 1000)])
def test_windowed_prefill(N, L, window, sinks, dtype):
    q, k, v = queries(dtype, 5, 1, 8, N), keys(dtype, 6, 1, 2, L), values(dtype, 7, 1, 2, L)
    out, lse = (x.cpu() for x in rf.attn_prefill_window(q.cuda(), k.cuda(), v.cuda(), window=window, sinks=sinks))
    for i in sorted({0, 19, N // 2, N - 33 % N, N - 1}):
        seen = C.visible(L - N + i, window, sinks)
        for h in range(8):
            check_row(out[0, h, i], lse[0, h, i], f64(q[0, h, i]), f64(k[0, h // 4])[seen], f64(v[0, h // 4])[seen],
                      f"row {i}, head {h}")


def test_causal_prefill():
    """Up to 2^30 in log2 units."""
    q, k = queries("fp16", 8, 1, 2, 600).bfloat16(), keys("fp16", 9, 1, 2, 600).bfloat16() / 16
    v = values("bf16", 10, 1, 2, 600)
    out, lse = (x.cpu() for x in rf.attn_prefill(q.cuda(), k.cuda(), v.cuda(), causal=True, scale=SCALE))
    for i in (0, 1, 127, 255, 256, 500, 599):
        for h in range(2):
            check_row(out[0, h, i], lse[0, h, i], f64(q[0, h, i]), f64(k[0, h])[:i + 1], f64(v[0, h])[:i + 1],
                      f"row {i}, head {h}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("B,prefix", [(3, 50), (200, 3000)])
def test_shared_prefix(B, prefix, dtype):
    """The prefix as each sequence's first keys, and read once by the pair kernel."""
    H, Hkv, cap = 8, 2, 120
    lens = [(37 * b) % (cap + 1) for b in range(B)]
    q = queries(dtype, 11, B, H)
    kp, vp = keys(dtype, 12, Hkv, prefix), values(dtype, 13, Hkv, prefix)
    k, v = keys(dtype, 14, B, Hkv, cap), values(dtype, 15, B, Hkv, cap)
    out, lse = (x.cpu() for x in rf.attn_decode_shared(q.cuda(), kp.cuda(), vp.cuda(), k.cuda(), v.cuda(), i32(lens)))
    for b in range(0, B, 1 + B // 30):
        for h in range(H):
            kk, vv = (np.concatenate([f64(x[h // 4]), f64(y[b, h // 4, :lens[b]])]) for x, y in ((kp, k), (vp, v)))
            check_row(out[b, h], lse[b, h], f64(q[b, h]), kk, vv, f"sequence {b}, head {h}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_over_a_dense_cache(dtype):
    lens = [1, 40, 700, 333]
    q, k, v = queries(dtype, 16, 4, 8), keys(dtype, 17, 4, 2, 700), values(dtype, 18, 4, 2, 700)
    out, lse = (x.cpu() for x in rf.attn_decode_window(q.cuda(), k.cuda(), v.cuda(), i32(lens)))
    for b, n in enumerate(lens):
        for h in range(8):
            check_row(out[b, h], lse[b, h], f64(q[b, h]), f64(k[b, h // 4, :n]), f64(v[b, h // 4, :n]),
                      f"sequence {b}, head {h}")
