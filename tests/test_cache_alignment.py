"""Buffers that the calls over a serving cache access in vectors are refused where they do not begin
on 16 bytes, before any CUDA call: no GPU is needed."""

import pytest

from test_cache_abi import ODD, P, lib, shared_args, weights_args, window_args   # noqa: F401


@pytest.mark.parametrize("address", [0x10004, 0x10008, 0x1000c])
def test_scores(lib, address):                                               # noqa: F811
    # pairs of scores are stored eight bytes at a time
    for cap in (100, 101):
        assert lib.rf_attn_decode_weights(*weights_args(scores=P(address), cap=cap)) == 3


def test_every_vector_buffer(lib):                                           # noqa: F811
    for f, args in ((lib.rf_attn_decode_window, window_args), (lib.rf_attn_decode_weights, weights_args),
                    (lib.rf_attn_decode_shared, shared_args)):
        for name in ("q", "k", "v", "out", "seg_acc"):
            assert f(*args(**{name: ODD})) == 3, name
