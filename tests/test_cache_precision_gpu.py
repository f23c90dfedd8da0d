"""Calls over a serving cache whose weights keep two 16-bit terms, told from one term: half of the
keys weigh 1 and hold -round16(w), the others weigh w and hold 1, so that the output is the
rounding error of w.  With one term it would be 0, with two it is w's to 2^-16 (bf16).

A key's score has one nonzero product, which is exact.
"""

import numpy as np
import pytest
import torch

from cache_helpers import DT, HALF_STEP, assert_within, normal, out_bound
from helpers import f64
from oracle import cache as C

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def worst_scale(dtype):
    """A scale whose w = exp(-scale) is about half a step from its neighbours of the type."""
    x = np.linspace(0.1, 0.6, 5001).astype(np.float32).astype(np.float64)
    w = torch.from_numpy(np.exp(-x))
    return float(x[((w - w.to(dtype).double()).abs() / w).argmax()])


def keys_and_values(dtype, *shape):
    """k, v [..., n, 128] of both kinds of keys in turn."""
    k, v = torch.zeros(*shape, 128, dtype=dtype), torch.ones(*shape, 128, dtype=dtype)
    k[..., 1::2, 0] = -1
    v[..., 0::2, :] = -torch.tensor(np.exp(-worst_scale(dtype))).to(dtype)
    return k, v


def query(dtype, *shape):
    q = torch.zeros(*shape, 128, dtype=dtype)
    q[..., 0] = 1
    return q


def bound(ref, scale, out_dtype, p_step):
    # the score loses 2^-23 to each of the scale's two roundings; the largest value is 1
    return out_bound(ref, 2.0 ** -22 * scale, 1.0, out_dtype, p_step)


def check(out, k, v, dtype, p_step=2.0 ** -16):
    """out [..., 128], every row the same: over k, v [n, 128]."""
    scale = worst_scale(dtype)
    ref = C.attend(f64(query(dtype)), f64(k), f64(v), scale)[0]
    assert_within(f64(out), np.broadcast_to(ref, out.shape), bound(ref, scale, out.dtype, p_step), "out")


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("n", [2, 300])
def test_one_term_is_outside_the_bound(dtype, n):
    k, v = keys_and_values(DT[dtype], n)
    scale = worst_scale(DT[dtype])
    ref, _, w = C.attend(f64(query(DT[dtype])), f64(k), f64(v), scale)
    p = torch.from_numpy(w / w.max())
    hi = p.to(DT[dtype]).double()
    lo = (p - hi).to(DT[dtype]).double()
    one, two = ((x.numpy() / p.sum().item()) @ f64(v) for x in (hi, hi + lo))
    limit = bound(ref, scale, DT[dtype], 2.0 ** -16)
    assert np.all(np.abs(two - ref) <= limit) and np.all(np.abs(one - ref) > 4 * limit)


@gpu
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 2), (20, 1)])
@pytest.mark.parametrize("N,L,window,sinks", [(1, 2, 0, 0), (3, 300, 0, 0), (5, 900, 256, 4), (7, 64, 20, 2)])
def test_few_rows(rf, N, L, window, sinks, H, Hkv, dtype):
    k, v = keys_and_values(DT[dtype], 2, Hkv, L)
    out, _ = rf.attn_prefill_window(query(DT[dtype], 2, H, N).cuda(), k.cuda(), v.cuda(), window=window,
                                    sinks=sinks, scale=worst_scale(DT[dtype]))
    for i in range(N):
        keys = C.visible(L - N + i, window, sinks)
        check(out[:, :, i], k[0, 0, keys], v[0, 0, keys], DT[dtype])


@gpu
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("B,H,Hkv,prefix,cap", [(1, 1, 1, 1, 1), (2, 16, 2, 200, 40), (5, 8, 2, 333, 17),
                                                (3, 20, 1, 640, 1)])
def test_small_shared_prefix(rf, B, H, Hkv, prefix, cap, dtype):
    kp, vp = keys_and_values(DT[dtype], Hkv, prefix)
    k, v = keys_and_values(DT[dtype], B, Hkv, cap)
    lens = [cap * b // B for b in range(B)]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for out_dtype in (torch.float32, None):
        out, _ = rf.attn_decode_shared(query(DT[dtype], B, H).cuda(), kp.cuda(), vp.cuda(), k.cuda(), v.cuda(), n,
                                       scale=worst_scale(DT[dtype]), out_dtype=out_dtype)
        for b, m in enumerate(lens):
            check(out[b], torch.cat([kp[0], k[b, 0, :m]]), torch.cat([vp[0], v[b, 0, :m]]), DT[dtype])


@gpu
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("B,cap", [(2, 300), (330, 1700)])
def test_decode(rf, B, cap, dtype):
    k, v = keys_and_values(DT[dtype], 1, cap)
    lens = [2, cap] + [cap - 3 * b for b in range(2, B)]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kb, vb = (t.cuda().expand(B, 1, cap, 128).contiguous() for t in (k, v))
    for out_dtype in (torch.float32, None):
        out, _ = rf.attn_decode_window(query(DT[dtype], B, 3).cuda(), kb, vb, n, scale=worst_scale(DT[dtype]),
                                       out_dtype=out_dtype)
        for b in {0, 1, B // 2, B - 1}:
            check(out[b], k[0, :lens[b]], v[0, :lens[b]], DT[dtype])


@gpu
def test_causal_prefills_agree(rf):
    """The windowed prefill without a window and the causal one round every weight once to bf16 and
    the output once: both stay within that bound of the definition, not only near each other."""
    scale = 128 ** -0.5
    q, k, v = (normal(s, 1, 2, 500, 128).cuda() for s in (9, 10, 11))
    for out, lse in (rf.attn_prefill_window(q, k, v, scale=scale), rf.attn_prefill(q, k, v, causal=True, scale=scale)):
        for h in range(2):
            qd, kd, vd = f64(q[0, h]), f64(k[0, h]), f64(v[0, h])
            ref = [C.prefill_row(qd[i], kd, vd, i, scale, 0, 0) for i in range(500)]
            ro, rl = np.stack([x[0] for x in ref]), np.array([x[1] for x in ref])
            delta = C.score_error(qd, kd, scale)
            assert_within(f64(out[0, h]), ro, out_bound(ro, delta, float(np.abs(vd).max()), out.dtype,
                                                        HALF_STEP[torch.bfloat16]), "out")
            assert_within(f64(lse[0, h]), rl, delta + 2.0 ** -19 + 2.0 ** -22 * np.abs(rl), "lse")
