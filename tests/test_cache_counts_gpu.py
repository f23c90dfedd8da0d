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
