"""Values of +inf and -inf in rows that a query sees, in the calls over a serving cache.

Every weight is positive, so an output column with an infinite value is that infinity, and NaN
where both signs meet; the other columns stay within the bounds of cache_helpers.  Each call runs
at a size of either kernel that it may take.
"""

import numpy as np
import pytest
import torch

from cache_helpers import DT, HALF_STEP, assert_within, normal, out_bound
from helpers import f64
from oracle import cache as C

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5
INF = float("inf")


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def check_rows(got, q, k, v, p_step, what):
    """got [n, D] and q [n, D] over the keys k, v [keys, D] that they see."""
    q, k, v, out = f64(q), f64(k), f64(v), f64(got)
    with np.errstate(invalid="ignore"):
        ref = np.stack([C.attend(x, k, v, SCALE)[0] for x in q])
    assert not np.isfinite(ref).all(), f"{what}: nothing infinite is seen"
    vmax = float(np.abs(np.where(np.isfinite(v), v, 0)).max())
    fine = np.where(np.isfinite(ref), ref, 0)
    bound = out_bound(fine, C.score_error(q, k, SCALE), vmax, got.dtype, p_step)
    assert_within(out, ref, np.where(np.isfinite(ref), bound, 0), what)


def spoil(v, bad, n):
    """Of one key head's values [rows, D], n in use: columns 5..69 of a row in the middle, column 3 of
    both signs, column 100 of the last row alone."""
    v[n // 2, 5:70] = bad
    v[0, 3], v[n - 1, 3] = INF, -INF
    v[n - 1, 100] = bad


def sequences(rf, large):
    """Batch of key heads 8 (large: more row groups than two CTAs per SM, rows in several pieces)."""
    if not large:
        return 2, 300, [300, 1]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return 2 * sms // 8 + 1, 1700, None


@pytest.mark.parametrize("bad", [INF, -INF])
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("large", [False, True])
def test_decode(rf, large, dtype, bad):
    B, cap, lens = sequences(rf, large)
    lens = lens or [1700 if b % 2 else 1550 for b in range(B - 1)] + [1]
    H, Hkv = 16, 8
    q = normal(1, B, H, 128, dtype=DT[dtype]).cuda()
    k, v = normal(2, B, Hkv, cap, 128, dtype=DT[dtype]).cuda(), normal(3, B, Hkv, cap, 128, dtype=DT[dtype]).cuda()
    clean = rf.attn_decode_window(q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=SCALE)
    spoil(v[0, 2], bad, lens[0])
    v[-1, 5, 0] = bad                                    # the only key of its sequence
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for out_dtype in (None, torch.float32):
        out, lse = rf.attn_decode_window(q, k, v, n, scale=SCALE, out_dtype=out_dtype)
        check_rows(out[0, 4:6], q[0, 4:6], k[0, 2, :lens[0]], v[0, 2, :lens[0]], 2.0 ** -16, "sequence 0")
        check_rows(out[-1, 10:12], q[-1, 10:12], k[-1, 5, :1], v[-1, 5, :1], 2.0 ** -16, "one key")
        assert torch.equal(lse, clean[1])
        if out_dtype is None:
            other = torch.ones(B, H, dtype=torch.bool)
            other[0, 4:6], other[-1, 10:12] = False, False
            assert torch.equal(out[other], clean[0][other])


@pytest.mark.parametrize("bad", [INF, -INF])
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("B", [4, 160])
def test_shared_prefix(rf, B, dtype, bad):
    H, Hkv, prefix, cap = 8, 2, 300, 20
    q = normal(11, B, H, 128, dtype=DT[dtype]).cuda()
    kp, vp = (normal(s, Hkv, prefix, 128, dtype=DT[dtype]).cuda() for s in (12, 13))
    k, v = (normal(s, B, Hkv, cap, 128, dtype=DT[dtype]).cuda() for s in (14, 15))
    lens = torch.full((B,), cap, dtype=torch.int32, device="cuda")
    spoil(vp[1], bad, prefix)                            # seen by heads 4..7 of every sequence
    spoil(v[1, 0], bad, cap)                             # by heads 0..3 of sequence 1
    out, lse = rf.attn_decode_shared(q, kp, vp, k, v, lens, scale=SCALE)
    for b in (0, 1, B - 1):
        for hk in (0, 1):
            if hk or b == 1:
                rows = slice(4 * hk, 4 * hk + 4)
                check_rows(out[b, rows], q[b, rows], torch.cat([kp[hk], k[b, hk]]),
                           torch.cat([vp[hk], v[b, hk]]), HALF_STEP[DT[dtype]], (b, hk))
    assert out[:1, :4].isfinite().all() and out[2:, :4].isfinite().all() and lse.isfinite().all()


@pytest.mark.parametrize("bad", [INF, -INF])
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("N", [1, 6, 400])
def test_prefill(rf, N, dtype, bad):
    H, Hkv, L, window, sinks = 8, 2, 500, 90, 3
    q = normal(21, 1, H, N, 128, dtype=DT[dtype]).cuda()
    k, v = (normal(s, 1, Hkv, L, 128, dtype=DT[dtype]).cuda() for s in (22, 23))
    v[0, 1, 1, 3], v[0, 1, L - 1, 3] = INF, -INF         # a sink and the last position's own
    v[0, 1, L - 1 - N // 2, 5:70] = bad
    out, lse = rf.attn_prefill_window(q, k, v, window=window, sinks=sinks, scale=SCALE)
    for i in sorted({0, N // 2, N - 1}):
        keys = C.visible(L - N + i, window, sinks)
        check_rows(out[0, 4:, i], q[0, 4:, i], k[0, 1, keys], v[0, 1, keys], HALF_STEP[DT[dtype]], i)
    assert out[0, :4].isfinite().all() and lse.isfinite().all()


@pytest.mark.parametrize("dtype", sorted(DT))
def test_one_key(rf, dtype):
    """The smallest call: the output is the value itself."""
    q, k, v = (normal(s, 1, 1, 1, 128, dtype=DT[dtype]).cuda() for s in (31, 32, 33))
    v[..., :3] = torch.tensor([INF, -INF, float("nan")])
    out, _ = rf.attn_prefill_window(q, k, v)
    assert torch.equal(out.nan_to_num(7), v.nan_to_num(7)) and out[..., 2].isnan().all()
    out, _ = rf.attn_decode_window(q[0], k, v)
    assert torch.equal(out.nan_to_num(7), v[0].nan_to_num(7)) and out[..., 2].isnan().all()
