"""Scores of 10^6 to 10^8, where fp32 counts in units: the largest one's value is the output, in both
types and whichever kernel a call of that size runs on.

The scores are 1 to 256 times the scale, so that each is behind the next by thousands."""

import numpy as np
import pytest
import torch

from cache_helpers import DT, HALF_STEP, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def keys(n, dtype, *lead):
    k = torch.zeros(*lead, n, 128, dtype=dtype)
    k[..., 0] = (torch.arange(n) % 256 + 1).to(dtype)    # 1 .. 256, exact
    return k.cuda()


def query(dtype, *shape):
    q = torch.zeros(*shape, 128, dtype=dtype)
    q[..., 0] = 1
    return q.cuda()


def same(out, v, dtype):
    """A weight of one, rounded once to 16 bits with its sum not rounded, and the output's rounding."""
    a, b = out.double(), v.double()
    return bool(((a - b).abs() <= 4 * HALF_STEP[dtype] * b.abs() + 2.0 ** -24).all())


# to where 15 is less than a step of the largest score
SCALES = [3000.0, 3333.3, 5000.0, 40000.0, 77777.7, 150000.0, 222222.2, 300000.0]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("B", [2, 320])
def test_decode(rf, B, dtype, scale):
    n, t = 256, DT[dtype]
    v = normal(1, B, 1, n, 128, dtype=t).cuda()
    out, lse = rf.attn_decode_window(query(t, B, 2), keys(n, t, B, 1), v, scale=scale)
    assert same(out, v[:, 0, n - 1][:, None].expand_as(out), t)
    assert torch.all((lse - 256 * scale).abs() <= 256 * scale * 2.0 ** -21)
    out, _ = rf.attn_decode_window(query(t, B, 2), keys(n, t, B, 1), v, scale=-scale)
    assert same(out, v[:, 0, 0][:, None].expand_as(out), t)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("N", [3, 256])
def test_prefill(rf, N, dtype, scale):
    n, t = 256, DT[dtype]
    v = normal(2, 1, 1, n, 128, dtype=t).cuda()
    for window in (0, 20):
        out, _ = rf.attn_prefill_window(query(t, 1, 2, N), keys(n, t, 1, 1), v, window=window, scale=scale)
        assert same(out, v[:, :, n - N:].expand_as(out), t)
    # descending: the window's first key is the largest
    out, _ = rf.attn_prefill_window(-query(t, 1, 2, N), keys(n, t, 1, 1), v, window=20, scale=scale)
    first = (torch.arange(n - N, n) - 19).clamp(min=0).cuda()
    assert same(out, v[:, :, first].expand_as(out), t)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("B", [2, 320])
def test_shared_prefix(rf, B, dtype, scale):
    n, t = 600, DT[dtype]
    vp, v = normal(3, 1, n, 128, dtype=t).cuda(), normal(4, B, 1, 10, 128, dtype=t).cuda()
    # twice 1 .. 256, then 1 .. 88: the largest score occurs twice; own keys 1 .. 10
    out, _ = rf.attn_decode_shared(query(t, B, 2), keys(n, t, 1), vp, keys(10, t, B, 1), v, scale=scale)
    assert same(out, ((vp[0, 255].double() + vp[0, 511].double()) / 2).expand_as(out), t)
    out, _ = rf.attn_decode_shared(query(t, B, 2), keys(n, t, 1)[:, :255].contiguous(), vp[:, :255].contiguous(),
                                   2 * keys(256, t, B, 1), v.repeat(1, 1, 26, 1)[:, :, :256].contiguous(), scale=scale)
    assert same(out, v[:, 0, 255 % 10][:, None].expand_as(out), t)
