"""Norm and rotation of query and key heads, and the write into pages, against float64.

Tolerance: the norm's factor is off by less than 2^-19 of itself (16 products and 4 sums of squares,
each a rounding of 2^-24, halved by the root; the mean, eps, rsqrt's 2 ulp and two products), sine and
cosine by less than 2^-21 (2 ulp, and half a step of the fp32 angle), the rotation's two terms by a
rounding each: in all less than 2^-18 of |a| + |b|.  Rounding the result adds half a step of it."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import cascaded_reductions_gb300 as rf
from cache_helpers import DT, HALF_STEP, assert_within, normal
from helpers import f64
from oracle import paged
from paged_helpers import i32

pytestmark = pytest.mark.gpu


def bound(ref, size, dtype):
    moved = 2.0 ** -18 * size
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133     # half the smallest step
    return HALF_STEP[dtype] * (np.abs(ref) + moved) + moved + tiny


def inputs(T, H, Hkv, D, dtype, seed, weights=True, w_dtype=None):
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn(T, (H + 2 * Hkv) * D, generator=g).to(dtype)
    qw, kw = (1 + 0.2 * torch.randn(D, generator=g) for _ in range(2))
    q, k, v = rows.cuda().split([H * D, Hkv * D, Hkv * D], 1)
    w = [x.to(w_dtype or dtype).cuda() if weights else None for x in (qw, kw)]
    return q.view(T, H, D), k.view(T, Hkv, D), v.view(T, Hkv, D), *w


def freqs(R, base=10000.0):
    return (base ** (-torch.arange(R // 2, dtype=torch.float64) * 2 / R)).float().cuda()


def check(q, k, qw, kw, pos, freq, axis=None, interleaved=False, eps=1e-6):
    qo, ko = rf.qk_norm_rope(q, k, pos, freq, qw, kw, axis=axis, interleaved=interleaved, eps=eps)
    for x, w, y, name in ((q, qw, qo, "q"), (k, kw, ko, "k")):
        ref, size = paged.norm_rope(f64(x), None if w is None else f64(w), eps, pos.cpu().numpy(), f64(freq),
                                    None if axis is None else axis.cpu().numpy(), interleaved)
        assert_within(f64(y), ref, bound(ref, size, x.dtype), name)
    return qo, ko


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 48), (256, 256), (256, 112)])
def test_widths(D, R, interleaved, dtype):
    q, k, _, qw, kw = inputs(7, 5, 3, D, DT[dtype], D + R)
    pos = i32([[0, 1, 2, 77, 4095, 131071, 1000000]])
    check(q, k, qw, kw, pos, freqs(R), interleaved=interleaved)


@pytest.mark.parametrize("T,H,Hkv", [(1, 1, 1), (1, 32, 8), (2, 7, 7), (33, 40, 8), (700, 3, 1), (5000, 4, 2),
                                     (2500, 32, 4)])
def test_sizes(T, H, Hkv):
    """From one token, whose heads several CTAs share, to CTAs of several tokens."""
    q, k, _, qw, kw = inputs(T, H, Hkv, 128, torch.bfloat16, T)
    check(q, k, qw, kw, i32(np.arange(T)[None] * 13 + 5), freqs(128))


def test_axes_and_numbers_outside():
    T, R = 50, 128
    q, k, _, qw, kw = inputs(T, 4, 4, 128, torch.float16, 9)
    rng = np.random.default_rng(9)
    pos = i32(rng.integers(0, 5000, (3, T)))
    check(q, k, qw, kw, pos, freqs(R), axis=i32(np.arange(R // 2) % 3))
    check(q, k, qw, kw, pos, freqs(R), axis=i32(np.arange(R // 2) - 30))       # below 0 and above 2


def test_far_and_negative_positions():
    T = 64
    q, k, _, qw, kw = inputs(T, 3, 2, 128, torch.float16, 11)
    rng = np.random.default_rng(11)
    check(q, k, qw, kw, i32(rng.integers(-2 ** 31, 2 ** 31 - 1, (1, T))), freqs(128))


def test_frequencies_of_whole_turns_and_large_ones():
    q, k, _, qw, kw = inputs(5, 3, 2, 64, torch.float16, 12)
    f = torch.tensor([0.0, -0.5, 6.2831855, 3.0, 100.25, -7.5, 1e-9, 1.0] * 2, device="cuda")
    check(q, k, qw, kw, i32([[0, 1, 5, 1000, 99999]]), f)


@pytest.mark.parametrize("w_dtype", [None, torch.float32])
def test_weights(w_dtype):
    q, k, _, qw, kw = inputs(9, 4, 2, 128, torch.bfloat16, 13, w_dtype=w_dtype)
    pos = i32(np.arange(9)[None])
    check(q, k, qw, kw, pos, freqs(128), eps=0.1)
    check(q, k, None, None, pos, freqs(128))
    check(q, k, None, kw, pos, freqs(128))


def test_zero_rows_and_rows_that_are_not_finite():
    q, k, _, qw, kw = inputs(6, 4, 2, 128, torch.bfloat16, 14)
    q, k = q.contiguous(), k.contiguous()
    q[0] = 0
    k[1, 0, 5] = float("inf")
    q[2, 3, 100] = float("nan")
    qo, ko = rf.qk_norm_rope(q, k, i32([[0, 1, 2, 3, 4, 5]]), freqs(128), qw, kw)
    assert torch.equal(qo[0], torch.zeros_like(qo[0]))
    bad = torch.zeros(6, 4, dtype=torch.bool)
    bad[2, 3] = True
    assert torch.equal(torch.isnan(qo).any(-1).cpu(), bad)              # one head, not its neighbours
    assert not torch.isnan(ko[0]).any() and not torch.isnan(ko[1, 1]).any()


@pytest.mark.parametrize("page", [1, 16, 24, 128])
@pytest.mark.parametrize("T", [1, 45, 1300])
def test_cache_write(T, page):
    H, Hkv, D, dt = 8, 2, 128, torch.bfloat16
    q, k, v, qw, kw = inputs(T, H, Hkv, D, dt, T + page)
    P = -(-T // page) + 3
    kp, vp = (torch.full((P, Hkv, page, D), x, dtype=dt, device="cuda") for x in (3.0, 4.0))
    g = torch.Generator().manual_seed(1)
    slots = torch.randperm(P * page, generator=g)[:T].int()
    slots[::5] = -1                                     # tokens without a place
    if T > 3:
        slots[1], slots[2], slots[3] = P * page, 2 ** 31 - 1, -2 ** 31
    pos = i32(np.arange(T)[None] + 100)
    qo = rf.qk_norm_rope(q, k, pos, freqs(D), qw, kw, v=v, slots=slots.cuda(), kp=kp, vp=vp)
    ref_q, ref_k = rf.qk_norm_rope(q, k, pos, freqs(D), qw, kw)
    assert torch.equal(qo, ref_q)
    want_k, want_v = torch.full_like(kp, 3.0), torch.full_like(vp, 4.0)
    for t in range(T):
        s = int(slots[t])
        if 0 <= s < P * page:
            want_k[s // page, :, s % page] = ref_k[t]
            want_v[s // page, :, s % page] = v[t]
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)


def test_in_place_and_dense_rows():
    q, k, _, qw, kw = inputs(70, 4, 2, 128, torch.float16, 15)
    pos = i32(np.arange(70)[None])
    want = rf.qk_norm_rope(q, k, pos, freqs(128), qw, kw)
    q, k = q.contiguous(), k.contiguous()
    rf.rf_qk_norm_rope(q, k, None, qw, kw, 1e-6, pos, freqs(128), None, False, None, q, k, None)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_far_rows():
    """Rows 2^20 elements apart: offsets past 2^31 bytes."""
    T, H, D = 2100, 2, 64
    rows = torch.zeros(T, 1 << 20, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rows[:, :3 * H * D] = torch.randn(T, 3 * H * D, generator=g, device="cuda").bfloat16()
    q, k = rows[:, :H * D].view(T, H, D), rows[:, H * D:2 * H * D].view(T, H, D)
    pos = i32(np.arange(T)[None])
    a = rf.qk_norm_rope(q, k, pos, freqs(64))
    b = rf.qk_norm_rope(q.contiguous(), k.contiguous(), pos, freqs(64))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_in_place_of_one_token_and_outputs_between_the_rows():
    """What the check of overlapping buffers lets through."""
    q, k, _, qw, kw = inputs(1, 4, 2, 128, torch.bfloat16, 16)          # steps of a longer row, T = 1
    pos = i32([[77]])
    want = rf.qk_norm_rope(q, k, pos, freqs(128), qw, kw)
    q, k = q.clone(), k.clone()
    rf.rf_qk_norm_rope(q, k, None, qw, kw, 1e-6, pos, freqs(128), None, False, None, q, k, None)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    # two tokens 64 KiB apart, both outputs in the gap
    wide = torch.zeros(2, 32768, dtype=torch.bfloat16, device="cuda")
    rows = normal(17, 2, 6, 128).cuda()
    wide[:, :768] = rows.view(2, 768)
    q, k = wide[:, :512].view(2, 4, 128), wide[:, 512:768].view(2, 2, 128)
    q_out, k_out = wide[0, 4096:5120].view(2, 4, 128), wide[0, 768:1280].view(2, 2, 128)
    pos = i32([[5, 6]])
    want = rf.qk_norm_rope(q, k, pos, freqs(128), qw, kw)
    rf.rf_qk_norm_rope(q, k, None, qw, kw, 1e-6, pos, freqs(128), None, False, None, q_out, k_out, None)
    assert torch.equal(q_out, want[0]) and torch.equal(k_out, want[1])
    with pytest.raises(rf.RFError):                                     # half a row over the second token's key
        rf.rf_qk_norm_rope(q, k, None, qw, kw, 1e-6, pos, freqs(128), None, False, None, q_out,
                           wide.view(-1)[32768 + 704:32768 + 1216].view(2, 2, 128), None)


TURN = Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257242")    # 2 pi


@pytest.mark.parametrize("top", [1.0, 6.2831855, 100.0, 30000.0])
def test_angles_at_the_farthest_positions(top):
    """Against the exact product, taken mod a turn: off by |pos| max(1, |f|) 2^-52 rad and what the other
    tests allow the rest (sine and cosine 2^-18 of 1, half a step of the result)."""
    T, R = 40, 32
    rng = np.random.default_rng(int(top))
    pos = rng.integers(-2 ** 31, 2 ** 31 - 1, T)
    freq = np.float32(top * rng.random(R // 2))
    freq[0] = -top
    x = torch.zeros(T, 1, 64, dtype=torch.float16, device="cuda")
    x[..., :R // 2] = 1                                                     # (1, 0) turns to (cos, sin)
    out = f64(rf.qk_norm_rope(x, x, i32(pos[None]), torch.from_numpy(freq).cuda())[0])[:, 0]
    for t in range(T):
        for i in range(R // 2):
            f = float(freq[i])
            angle = float(Fraction(f) * int(pos[t]) % TURN)
            far = abs(int(pos[t])) * max(1.0, abs(f)) * 2.0 ** -52 + 2.0 ** -18
            got, want = out[t, [i, i + R // 2]], np.array([np.cos(angle), np.sin(angle)])
            assert_within(got, want, far + 2.0 ** -11 * (np.abs(want) + far) + 2.0 ** -25, f"token {t}, pair {i}")
