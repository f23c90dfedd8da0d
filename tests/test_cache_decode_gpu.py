"""Single-token decode over a cache of grouped heads (rf_attn_decode_window) and
its weight-accumulating form (rf_attn_decode_weights) against the definition in
float64.  Rows that a call must not read (behind a sequence's end, outside its
window) hold NaN in every case.

The output bound counts the score's fp32 rounding, the weights (two 16-bit
terms: 2^-16 of a bf16 weight) and one rounding of the output.
"""

import numpy as np
import pytest
import torch

from cache_helpers import DT, assert_within, check_decode, normal
from helpers import f64
from oracle import cache as C

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def make(seed, B, H, Hkv, cap, lens, window, sinks, dtype, gain=1.0):
    q = normal(seed, B, H, 128, dtype=dtype) * gain
    k, v = normal(seed + 1, B, Hkv, cap, 128, dtype=dtype), normal(seed + 2, B, Hkv, cap, 128, dtype=dtype)
    for b, n in enumerate(lens):
        hidden = np.setdiff1d(np.arange(cap), C.visible(n - 1, window, sinks))
        k[b, :, hidden] = float("nan")
        v[b, :, hidden] = float("nan")
    return q.cuda(), k.cuda(), v.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


# (H, Hkv): a key head each; groups of 4, 7 and 16; more than 16 query heads on one key head
HEADS = [(4, 4), (8, 2), (7, 1), (16, 1), (40, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,Hkv", HEADS)
def test_ragged_lengths(rf, H, Hkv, dtype):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 129, 333]
    q, k, v, n = make(H, len(lens), H, Hkv, 333, lens, 0, 0, DT[dtype])
    out, lse = rf.attn_decode_window(q, k, v, n, scale=SCALE)
    check_decode(out, lse, q, k, v, lens, SCALE)
    assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[0]))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (16, 4), (50, 3), (100, 64), (500, 4),
                                          (64, 500)])
def test_window_and_sinks(rf, window, sinks):
    lens = [1, 16, 51, 64, 160, 299]
    q, k, v, n = make(window, len(lens), 8, 2, 300, lens, window, sinks, torch.bfloat16)
    out, lse = rf.attn_decode_window(q, k, v, n, window=window, sinks=sinks, scale=SCALE)
    check_decode(out, lse, q, k, v, lens, SCALE, window, sinks)


@pytest.mark.parametrize("S", [1, 2, 5, 33, 70, 4096])
def test_segment_counts(rf, S):
    lens = [5000, 77, 0]
    q, k, v, n = make(S, 3, 8, 2, 5000, lens, 0, 0, torch.bfloat16)
    work = rf.decode_workspace(3, 8, 2, 5000, S=S)
    for _ in range(2):                                   # the counters come back to zero
        out, lse = rf.attn_decode_window(q, k, v, n, scale=SCALE, work=work)
        check_decode(out, lse, q, k, v, lens, SCALE)
    assert torch.all(work.counters == 0)


@pytest.mark.parametrize("S", [None, 1, 2, 3, 9, 60, 4096])
@pytest.mark.parametrize("lens", [[2100, 0, 1, 17, 1600, 2099], [2100] * 6, [0, 0, 0, 0, 0, 1500]])
def test_large_calls(rf, lens, S):
    # enough tiles (48 groups of up to 132) for the warps to share them across groups
    q, k, v, n = make(3, 6, 16, 8, 2100, lens, 0, 0, torch.bfloat16)
    work = rf.decode_workspace(6, 16, 8, 2100, S=S)
    for _ in range(2):
        out, lse = rf.attn_decode_window(q, k, v, n, scale=SCALE, work=work)
    check_decode(out, lse, q, k, v, lens, SCALE)
    assert torch.all(work.counters == 0)


def test_large_batch_of_short_sequences(rf):
    # more sequences than a block has threads, most of a tile or less
    lens = [(5 * b) % 37 for b in range(700)]
    lens[333] = 300
    q, k, v, n = make(4, 700, 8, 4, 300, lens, 0, 0, torch.float16)
    out, lse = rf.attn_decode_window(q, k, v, n, scale=SCALE)
    check_decode(out, lse, q, k, v, lens, SCALE)


def test_large_windowed_call_with_many_query_heads(rf):
    lens = [3000, 1, 700, 2999, 64]
    q, k, v, n = make(5, 5, 40, 2, 3000, lens, 2500, 33, torch.bfloat16)
    out, lse = rf.attn_decode_window(q, k, v, n, window=2500, sinks=33, scale=SCALE)
    check_decode(out, lse, q, k, v, lens, SCALE, 2500, 33)


def test_fp32_output_whole_cache_and_peaked_scores(rf):
    # no lengths: every sequence holds cap keys; large queries move the maximum often
    q, k, v, _ = make(5, 2, 4, 1, 777, [777, 777], 0, 0, torch.float16, gain=8.0)
    out, lse = rf.attn_decode_window(q, k, v, scale=SCALE, out_dtype=torch.float32)
    assert out.dtype == torch.float32
    check_decode(out, lse, q, k, v, [777, 777], SCALE)


def test_lengths_outside_the_cache_are_clamped(rf):
    q, k, v, _ = make(6, 2, 4, 2, 40, [40, 0], 0, 0, torch.bfloat16)
    n = torch.tensor([1000, -3], dtype=torch.int32, device="cuda")
    out, lse = rf.attn_decode_window(q, k, v, n, scale=SCALE)
    check_decode(out, lse, q, k, v, [40, 0], SCALE)


def test_a_nan_key_reaches_only_its_own_rows(rf):
    q, k, v, n = make(7, 2, 4, 2, 200, [200, 150], 0, 0, torch.bfloat16)
    k[0, 1, 13] = float("nan")
    out, lse = rf.attn_decode_window(q, k, v, n, scale=SCALE)
    assert torch.all(torch.isnan(out[0, 2:])) and torch.all(torch.isnan(lse[0, 2:]))
    assert torch.all(torch.isfinite(out[0, :2])) and torch.all(torch.isfinite(out[1]))


def test_cache_beyond_32_bit_offsets(rf):
    # 2^32 bytes lie before the last key head's rows
    cap, Hkv = 1 << 19, 34
    k = torch.zeros(1, Hkv, cap, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[0, -1, -5:], v[0, -1, -5:] = normal(8, 5, 128).cuda(), normal(9, 5, 128).cuda()
    q = normal(10, 1, Hkv, 128).cuda()
    out, lse = rf.attn_decode_window(q, k, v, window=5, scale=SCALE)
    ref, rl = out[:, -1:], lse[:, -1:]
    check_decode(ref, rl, q[:, -1:], k[:, -1:, -5:], v[:, -1:, -5:], [5], SCALE)
    assert torch.all(out[:, :-1] == 0)


def test_the_same_bits_every_time(rf):
    q, k, v, n = make(11, 4, 32, 8, 3001, [3001, 2000, 1, 77], 0, 0, torch.bfloat16)
    first = rf.attn_decode_window(q, k, v, n, scale=SCALE)
    for _ in range(5):
        again = rf.attn_decode_window(q, k, v, n, scale=SCALE)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ----------------------------------------------------------------- weights --

def check_weights(total, before, w, q, lens, delta):
    """A weight is off by exp(2 delta) - 1 + 2^-19 of itself (see cache_helpers), the lse it is
    normalised by rounded in fp32 (2^-20 covers |lse| < 4 units in the last place of 8), and each
    of the G additions rounds the running total."""
    G = q.shape[1] // before.shape[1]
    exact = before + w
    share = np.expm1(2 * delta) + 2.0 ** -18
    assert_within(f64(total), exact, w * share + (G + 1) * 2.0 ** -24 * np.abs(exact) + 1e-30, "weight")
    for b, n in enumerate(lens):
        assert np.array_equal(f64(total)[b, :, n:], before[b, :, n:])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,Hkv", HEADS)
def test_weights(rf, H, Hkv, dtype):
    lens = [0, 1, 16, 65, 200, 201]
    q, k, v, n = make(20 + H, len(lens), H, Hkv, 201, lens, 0, 0, DT[dtype])
    before = torch.rand(len(lens), Hkv, 201, generator=torch.Generator().manual_seed(1))
    out, lse, total = rf.attn_decode_weights(q, k, v, n, weight=before.cuda(), scale=SCALE)
    w, delta = check_decode(out, lse, q, k, v, lens, SCALE)
    check_weights(total, f64(before), w, q, lens, delta)


def test_weights_from_zero_and_in_place(rf):
    lens = [300, 41]
    q, k, v, n = make(30, 2, 8, 2, 300, lens, 0, 0, torch.bfloat16)
    out, lse, total = rf.attn_decode_weights(q, k, v, n, scale=SCALE)
    w, delta = check_decode(out, lse, q, k, v, lens, SCALE)
    check_weights(total, np.zeros_like(w), w, q, lens, delta)
    # every head's weights sum to 1; the check's own sum in float64
    assert np.allclose(f64(total).sum(-1), 4.0, rtol=1e-5)
    kept = total.clone()
    rf.attn_decode_weights(q, k, v, n, weight=total, weight_out=total, scale=SCALE)
    check_weights(total, f64(kept), w, q, lens, delta)


def test_weights_one_segment_and_many(rf):
    lens = [2000, 3]
    q, k, v, n = make(31, 2, 8, 2, 2000, lens, 0, 0, torch.bfloat16)
    for S in (1, 7, 31):
        work = rf.decode_workspace(2, 8, 2, 2000, weights=True, S=S)
        out, lse, total = rf.attn_decode_weights(q, k, v, n, scale=SCALE, work=work)
        w, delta = check_decode(out, lse, q, k, v, lens, SCALE)
        check_weights(total, np.zeros_like(w), w, q, lens, delta)


# ---------------------------------------------------- graphs, streams, wrap --

def test_captured_and_replayed(rf):
    B, H, Hkv, cap = 3, 8, 2, 500
    q, k, v, n = make(40, B, H, Hkv, cap, [cap] * B, 0, 0, torch.bfloat16)
    work = rf.decode_workspace(B, H, Hkv, cap, weights=True)
    total = torch.zeros(B, Hkv, cap, device="cuda")

    def step():
        return rf.attn_decode_weights(q, k, v, n, weight=total, scale=SCALE, work=work)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse, after = step()
    for seed, lens in ((41, [500, 1, 0]), (42, [33, 499, 250])):
        q2, k2, v2, n2 = make(seed, B, H, Hkv, cap, lens, 0, 0, torch.bfloat16)
        for dst, src in ((q, q2), (k, k2), (v, v2), (n, n2)):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        w, delta = check_decode(out, lse, q, k, v, lens, SCALE)
        check_weights(after, np.zeros_like(w), w, q, lens, delta)


def test_on_another_stream(rf):
    lens = [700, 20]
    q, k, v, n = make(50, 2, 8, 2, 700, lens, 0, 0, torch.bfloat16)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out, lse = rf.attn_decode_window(q, k, v, n, scale=SCALE, stream=st)
    st.synchronize()
    check_decode(out, lse, q, k, v, lens, SCALE)


def test_python_layer_refusals(rf):
    q, k, v, n = make(60, 2, 8, 2, 50, [50, 3], 0, 0, torch.bfloat16)
    work = rf.decode_workspace(2, 8, 2, 50)
    for bad in (lambda: rf.attn_decode_window(q, k.transpose(1, 2), v, n),          # not contiguous
                lambda: rf.attn_decode_window(q, k.half(), v, n),                   # another type
                lambda: rf.attn_decode_window(q, k, v[:, :, :40].contiguous(), n),  # another shape
                lambda: rf.attn_decode_window(q, k, v, n.long()),
                lambda: rf.attn_decode_window(q, k, v, n.cpu()),
                lambda: rf.attn_decode_window(q[:1].contiguous(), k[:1].contiguous(),
                                              v[:1].contiguous(), n[:1].contiguous(), work=work),
                lambda: rf.attn_decode_weights(q, k, v, n, work=work)):             # no scores in it
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: rf.attn_decode_window(q, k, v, n, window=-1),
                lambda: rf.attn_decode_window(q, k, v, n, out_dtype=torch.float16),
                lambda: rf.attn_decode_window(q[..., :64].contiguous(), k[..., :64].contiguous(),
                                              v[..., :64].contiguous(), n)):
        with pytest.raises(rf.RFError):
            bad()
