"""Counts near the largest int, and Python counts that do not fit one: taken as the largest or
refused, never cut to their low bits."""

import pytest
import torch

from cache_helpers import normal

pytestmark = pytest.mark.gpu

MOST = (1 << 31) - 1


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def test_segment_proposals_at_the_largest_counts(rf):
    for groups in (1, 8, 304, 305, MOST):
        want = rf.rf_decode_segments(groups, 1 << 30)
        assert 1 <= want <= 4096
        for keys in (MOST - 800, MOST - 64, MOST - 63, MOST - 62, MOST):
            assert rf.rf_decode_segments(groups, keys) == want, (groups, keys)


def test_prefix_proposals_at_the_largest_counts(rf):
    assert rf.rf_prefix_segments(1, 8, 2, 1 << 30) >= 2
    assert rf.rf_prefix_segments(1, 8, 2, (1 << 30) + 1) == 0      # longer than the call takes
    assert rf.rf_prefix_segments(1, 8, 2, MOST) == 0
    assert rf.rf_prefix_segments(MOST, 1, 1, 1000) >= 2


def test_python_counts_beyond_an_int(rf):
    for keys in (1 << 31, 1 << 32, (1 << 32) + 5):
        assert rf.rf_decode_segments(8, keys) == rf.rf_decode_segments(8, MOST)
    assert rf.rf_decode_segments((1 << 32) + 1, 1000) == rf.rf_decode_segments(MOST, 1000)
    assert rf.rf_decode_segments(-(1 << 32) + 8, 1000) == rf.rf_decode_segments(1, 1000)
    assert rf.rf_prefix_segments((1 << 32) + 1, 8, 2, 100) == 0
    assert rf.rf_prefix_segments(1, 8, 2, (1 << 32) + 100) == 0


@pytest.mark.parametrize("extension", [True, False])
@pytest.mark.parametrize("given", [True, False])
def test_eviction_counts(rf, monkeypatch, extension, given):
    if not extension:
        monkeypatch.setattr(rf, "_calls", None)
    k, w = normal(1, 1, 2, 50, 128).cuda(), normal(2, 1, 2, 50, dtype=torch.float32).cuda()
    out = [torch.zeros_like(k[:, :, :20]), torch.zeros_like(k[:, :, :20]), torch.zeros_like(w[:, :, :20])]
    for bad in ({"sinks": (1 << 32) + 2}, {"recent": (1 << 32) + 5}, {"sinks": -(1 << 32) + 2}, {"recent": 1 << 31}):
        with pytest.raises(rf.RFError):
            rf.cache_evict(k, k.clone(), w, None, 20, **{"sinks": 1, "recent": 1, **bad}, out=out if given else None)
    assert all(torch.all(t == 0) for t in out)


def test_tensor_sizes_beyond_an_int(rf):
    # 2^32 + 8 columns of which the low 32 bits are a size that the call takes: 8 GiB a tensor
    D = (1 << 32) + 8
    k = torch.zeros(1, 1, 1, D, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1, 1, 1, device="cuda")
    out = [torch.zeros_like(k), None, torch.zeros_like(w)]
    with pytest.raises(rf.RFError):
        rf.cache_evict(k, None, w, None, 1, out=out)
    assert torch.all(out[2] == 0)
