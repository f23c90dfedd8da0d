"""Refusals of the calls over a serving cache: every call below is rejected by
the host checks before any CUDA call is made, so they run without a GPU."""

import ctypes

import pytest

P = ctypes.c_void_p
F = ctypes.c_float
FAKE, ODD, NULL = P(0x10000), P(0x10004), P(0)


@pytest.fixture(scope="module")
def lib():
    from conftest import load_builder
    return ctypes.CDLL(load_builder().build())


def window_args(**o):
    return [o.get("q", FAKE), o.get("k", FAKE), o.get("v", FAKE), o.get("lens", NULL), o.get("B", 2),
            o.get("H", 8), o.get("Hkv", 2), o.get("cap", 100), o.get("D", 128), o.get("window", 0),
            o.get("sinks", 0), o.get("S", 4), F(o.get("scale", 0.1)), o.get("dtype", 1),
            o.get("seg_m", FAKE), o.get("seg_l", FAKE), o.get("seg_acc", FAKE), o.get("counters", FAKE),
            o.get("out", FAKE), o.get("out_dtype", 1), NULL, NULL]


def weights_args(**o):
    return [o.get("q", FAKE), o.get("k", FAKE), o.get("v", FAKE), NULL, o.get("B", 2), o.get("H", 8),
            o.get("Hkv", 2), o.get("cap", 100), o.get("D", 128), o.get("S", 4), F(o.get("scale", 0.1)),
            o.get("dtype", 1), o.get("seg_m", FAKE), o.get("seg_l", FAKE), o.get("seg_acc", FAKE),
            o.get("counters", FAKE), o.get("scores", FAKE), o.get("out", FAKE), o.get("out_dtype", 1),
            NULL, o.get("weight", NULL), o.get("weight_out", FAKE), NULL]


@pytest.mark.parametrize("call,args", [("rf_attn_decode_window", window_args),
                                       ("rf_attn_decode_weights", weights_args)])
def test_decode_refusals(lib, call, args):
    f = getattr(lib, call)
    for name in ("q", "k", "v", "seg_m", "seg_l", "seg_acc", "counters", "out"):
        assert f(*args(**{name: NULL})) == 1, name
    for name in ("B", "H", "Hkv", "cap", "D"):
        assert f(*args(**{name: 0})) == 1, name
        assert f(*args(**{name: -4})) == 1, name
    assert f(*args(H=7)) == 1                       # not a multiple of Hkv
    assert f(*args(S=0)) == 1
    assert f(*args(scale=float("nan"))) == 1
    assert f(*args(scale=float("inf"))) == 1
    assert f(*args(dtype=3)) == 1
    assert f(*args(out_dtype=2)) == 1               # fp16 out of bf16 inputs
    assert f(*args(dtype=2, out_dtype=1)) == 1
    assert f(*args(D=64)) == 2
    assert f(*args(dtype=0, out_dtype=0)) == 2      # fp32 inputs
    assert f(*args(S=4097)) == 2
    assert f(*args(cap=(1 << 30) + 1)) == 2
    assert f(*args(B=1 << 30, S=4096)) == 2         # too many CTAs
    assert f(*args(B=(1 << 31) - 1, H=2147483646, Hkv=2147483646)) == 2
    for name in ("q", "k", "v", "out", "seg_acc"):
        assert f(*args(**{name: ODD})) == 3, name


def test_window_refusals(lib):
    assert lib.rf_attn_decode_window(*window_args(window=-1)) == 1
    assert lib.rf_attn_decode_window(*window_args(sinks=-1)) == 1


def test_weights_refusals(lib):
    f = lib.rf_attn_decode_weights
    assert f(*weights_args(scores=NULL)) == 1
    assert f(*weights_args(weight_out=NULL)) == 1
    assert f(*weights_args(weight=P(0x10010), weight_out=FAKE)) == 1     # overlapping, not in place
    assert f(*weights_args(B=1 << 15, Hkv=1 << 11, H=1 << 11, S=1, cap=1 << 30)) == 2


def evict_args(**o):
    """Buffers far apart (1 TiB), so that only what a case asks for overlaps."""
    at = lambda i: P((i + 1) << 40)                                      # noqa: E731
    return [o.get("k", at(0)), o.get("v", at(1)), o.get("weight", at(2)), o.get("lens", at(3)),
            o.get("B", 2), o.get("Hkv", 2), o.get("cap", 100), o.get("D", 128), o.get("dtype", 1),
            o.get("keep", 50), o.get("sinks", 4), o.get("recent", 10), o.get("cap_out", 50),
            o.get("k_out", at(4)), o.get("v_out", at(5)), o.get("weight_out", at(6)),
            o.get("lens_out", at(7)), o.get("kept", at(8)), NULL]


def test_evict_refusals(lib):
    f = lib.rf_cache_evict
    for name in ("k", "weight", "k_out", "weight_out", "lens_out", "kept", "v", "v_out"):
        assert f(*evict_args(**{name: NULL})) == 1, name
    for name in ("B", "Hkv", "cap", "D", "keep"):
        assert f(*evict_args(**{name: 0})) == 1, name
    assert f(*evict_args(sinks=-1)) == 1
    assert f(*evict_args(recent=-1)) == 1
    assert f(*evict_args(sinks=41)) == 1            # sinks + recent > keep
    assert f(*evict_args(sinks=2147483647, recent=2147483647)) == 1
    assert f(*evict_args(keep=51)) == 1             # more than cap_out
    assert f(*evict_args(dtype=5)) == 1
    assert f(*evict_args(D=4)) == 2                 # rows of 8 bytes
    assert f(*evict_args(D=65536)) == 2
    assert f(*evict_args(cap=(1 << 30) + 1)) == 2
    for name in ("k", "v", "k_out", "v_out"):
        assert f(*evict_args(**{name: P((20 << 40) + 4)})) == 3, name
    base = (1 << 40)
    assert f(*evict_args(k_out=P(base))) == 1                            # in place
    assert f(*evict_args(k_out=P(base + 2 * 2 * 100 * 256 - 16))) == 1   # its first row on k's last
    assert f(*evict_args(lens_out=P(4 << 40))) == 1                      # lens_out is lens
    assert f(*evict_args(kept=P(8 << 40))) == 1                          # kept is lens_out


def test_segment_proposal_is_positive_or_zero_without_a_device(lib):
    assert 0 <= lib.rf_decode_segments(64, 4096) <= 64


def prefill_args(**o):
    return [o.get("q", FAKE), o.get("k", FAKE), o.get("v", FAKE), o.get("B", 2), o.get("H", 8),
            o.get("Hkv", 2), o.get("N", 10), o.get("cap", 100), o.get("D", 128), o.get("window", 0),
            o.get("sinks", 0), F(o.get("scale", 0.1)), o.get("dtype", 1), o.get("out", FAKE), NULL, NULL]


def test_prefill_refusals(lib):
    f = lib.rf_attn_prefill_window
    for name in ("q", "k", "v", "out"):
        assert f(*prefill_args(**{name: NULL})) == 1, name
        assert f(*prefill_args(**{name: ODD})) == 3, name
    for name in ("B", "H", "Hkv", "N", "cap", "D"):
        assert f(*prefill_args(**{name: 0})) == 1, name
    assert f(*prefill_args(N=101)) == 1             # more rows than positions
    assert f(*prefill_args(H=7)) == 1
    assert f(*prefill_args(window=-1)) == 1
    assert f(*prefill_args(sinks=-1)) == 1
    assert f(*prefill_args(scale=float("nan"))) == 1
    assert f(*prefill_args(dtype=3)) == 1
    assert f(*prefill_args(dtype=0)) == 2           # fp32
    assert f(*prefill_args(D=64)) == 2
    assert f(*prefill_args(scale=0.0)) == 2
    assert f(*prefill_args(scale=-0.1)) == 2
    assert f(*prefill_args(B=1 << 20, H=1 << 10, Hkv=1 << 10, N=4, cap=4)) == 2
    assert f(*prefill_args(cap=(1 << 30) + 1)) == 2


def shared_args(**o):
    return [o.get("q", FAKE), o.get("kp", FAKE), o.get("vp", FAKE), o.get("prefix", 1000), o.get("k", FAKE),
            o.get("v", FAKE), NULL, o.get("B", 2), o.get("H", 8), o.get("Hkv", 2), o.get("cap", 100),
            o.get("D", 128), o.get("Sp", 4), o.get("S", 4), F(o.get("scale", 0.1)), o.get("dtype", 1),
            o.get("seg_m", FAKE), o.get("seg_l", FAKE), o.get("seg_acc", FAKE), o.get("counters", FAKE),
            o.get("out", FAKE), o.get("out_dtype", 1), NULL, NULL]


def test_shared_refusals(lib):
    f = lib.rf_attn_decode_shared
    for name in ("q", "kp", "vp", "k", "v", "seg_m", "seg_l", "seg_acc", "counters", "out"):
        assert f(*shared_args(**{name: NULL})) == 1, name
    for name in ("B", "H", "Hkv", "cap", "D", "prefix"):
        assert f(*shared_args(**{name: 0})) == 1, name
    assert f(*shared_args(Sp=1)) == 1
    assert f(*shared_args(S=0)) == 1
    assert f(*shared_args(H=7)) == 1
    assert f(*shared_args(out_dtype=2)) == 1
    assert f(*shared_args(scale=float("inf"))) == 1
    assert f(*shared_args(Sp=4097)) == 2
    assert f(*shared_args(S=4097)) == 2
    assert f(*shared_args(scale=0.0)) == 2
    assert f(*shared_args(scale=-1.0)) == 2
    assert f(*shared_args(H=129, Hkv=1)) == 2       # more query heads than a tile has rows
    assert f(*shared_args(prefix=(1 << 30) + 1)) == 2
    assert f(*shared_args(dtype=0, out_dtype=0)) == 2
    assert f(*shared_args(D=64)) == 2
    for name in ("q", "kp", "vp", "k", "v", "out", "seg_acc"):
        assert f(*shared_args(**{name: ODD})) == 3, name


def test_prefix_segments_refuses_bad_sizes(lib):
    for a in ((0, 8, 2, 10), (2, 7, 2, 10), (2, 8, 2, 0), (2, 129, 1, 10), (-1, 8, 2, 10)):
        assert lib.rf_prefix_segments(*a) == 0


# ------------------------------------------------ refusals of the Python layer --

def test_python_layer_refuses_cpu_tensors_and_bad_shapes():
    import torch
    import cascaded_reductions_gb300 as rf
    q, k = torch.zeros(2, 8, 128, dtype=torch.bfloat16), torch.zeros(2, 2, 10, 128, dtype=torch.bfloat16)
    w = torch.zeros(2, 2, 10)
    for call in (lambda: rf.attn_decode_window(q, k, k), lambda: rf.attn_decode_weights(q, k, k),
                 lambda: rf.attn_decode_shared(q, k[0], k[0], k, k),
                 lambda: rf.attn_prefill_window(k, k, k), lambda: rf.cache_evict(k, k, w, None, 5),
                 lambda: rf.attn_decode_window(q[0], k, k), lambda: rf.decode_workspace(2, 7, 2, 10)):
        with pytest.raises(ValueError):
            call()


def test_quick_calls_leave_what_they_cannot_take_to_python():
    import torch

    from conftest import load_builder
    load_builder().build()
    import cascaded_reductions_gb300 as rf
    if rf._calls is None:
        pytest.skip("the extension is not built here")
    q, k = torch.zeros(2, 8, 128), torch.zeros(2, 2, 100, 128)
    w, sizes = torch.zeros(2, 2, 100), (0, 2, 8, 2, 128)
    fn, work = rf._DECODE_WINDOW, (1, 1, 1, 1)
    good = (fn, q, k, k, None, 0, 0, None, 1, sizes, work)
    assert rf._calls.decode_window(*good) is None                      # tensors on the CPU
    for i in range(len(good)):
        for bad in (None, "x", 1.5, (), [1], object()):
            assert rf._calls.decode_window(*good[:i], bad, *good[i + 1:]) is None
    assert rf._calls.decode_window(*good[:-1]) is None
    assert rf._calls.decode_window() is None
    assert rf._calls.decode_shared(fn, q, k[0], k[0], k, k, None, None, 0, 1, sizes, work) is None
    assert rf._calls.decode_weights(fn, q, k, k, None, w, None, 1, sizes, work, w) is None
    assert rf._calls.prefill_window(fn, q[None], k, k, 0, 0, None) is None
    assert rf._calls.cache_evict(fn, k, k, w, None, 10, 0, 0, k, k, w) is None
    with pytest.raises(ValueError):
        rf.attn_prefill_window(k, k, k)
