"""Rows whose every visible score is -inf have no weight to give: out = 0 and lse = -inf, as for
a row without visible keys, whichever kernel a call of that size runs on."""

import pytest
import torch

from cache_helpers import DT, normal

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def empty(out, lse):
    return torch.all(out == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("N", [4, 300])
def test_prefill(rf, N, dtype):
    q = normal(1, 1, 4, N, 128, dtype=DT[dtype]).cuda()
    k, v = (normal(s, 1, 2, 600, 128, dtype=DT[dtype]).cuda() for s in (2, 3))
    q[..., 0] = 1
    k[0, 0, :, 0] = float("-inf")                        # all of head 0's keys
    k[0, 1, 600 - N:, 0] = float("-inf")                 # of head 1's only the last ones
    out, lse = rf.attn_prefill_window(q, k, v, window=50, sinks=2, scale=SCALE)
    assert empty(out[0, :2], lse[0, :2])
    assert out[0, 2:].isfinite().all() and lse[0, 2:].isfinite().all()
    out, lse = rf.attn_prefill_window(q, k, v, window=2, sinks=0, scale=SCALE)
    assert empty(out[0, 2:, 1:], lse[0, 2:, 1:]) and lse[0, 2:, 0].isfinite().all()


@pytest.mark.parametrize("B", [3, 320])
def test_decode_and_prefix(rf, B):
    q = normal(4, B, 2, 128).cuda()
    kp, vp = (normal(s, 1, 300, 128).cuda() for s in (5, 6))
    k, v = (normal(s, B, 1, 90, 128).cuda() for s in (7, 8))
    q[..., 0] = 1
    k[0, ..., 0] = float("-inf")
    out, lse = rf.attn_decode_window(q, k, v, scale=SCALE)
    assert empty(out[0], lse[0]) and out[1:].isfinite().all() and lse[1:].isfinite().all()
    kp[..., 0] = float("-inf")
    both, lse2 = rf.attn_decode_shared(q, kp, vp, k, v, scale=SCALE)
    assert empty(both[0], lse2[0])
    assert torch.allclose(lse2[1:], lse[1:], rtol=0, atol=1e-5)
