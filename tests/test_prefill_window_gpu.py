"""Prefill with a sliding window and sinks (rf_attn_prefill_window) against the
definition in float64, row by row.

The output bound counts the score's fp32 rounding, the weights' rounding to 16
bits for the second product (half a step each: 2^-8 or 2^-11 of a weight) and
one rounding of the output.
"""

import numpy as np
import pytest
import torch

from cache_helpers import DT, HALF_STEP, assert_within, normal, out_bound
from helpers import f64
from oracle import cache as C

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def make(seed, B, H, Hkv, N, L, dtype, gain=1.0):
    return ((normal(seed, B, H, N, 128, dtype=dtype) * gain).cuda(),
            normal(seed + 1, B, Hkv, L, 128, dtype=dtype).cuda(),
            normal(seed + 2, B, Hkv, L, 128, dtype=dtype).cuda())


def check(out, lse, q, k, v, window, sinks, scale=SCALE, rows=None):
    """Every row, or the listed ones; NaN in a reference row has to be NaN in the result."""
    B, H, N, D = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    qd, kd, vd, od, ld = f64(q), f64(k), f64(v), f64(out), f64(lse)
    rows = range(N) if rows is None else rows
    for b in range(B):
        for h in range(H):
            kk, vv = kd[b, h // (H // Hkv)], vd[b, h // (H // Hkv)]
            fk, fv = np.nan_to_num(kk, posinf=0, neginf=0), np.nan_to_num(vv, posinf=0, neginf=0)
            delta = C.score_error(qd[b, h], fk, scale)
            vmax = float(np.abs(fv).max())
            with np.errstate(invalid="ignore"):
                ref = [C.prefill_row(qd[b, h, i], kk, vv, L - N + i, scale, window, sinks) for i in rows]
            ro, rl = np.stack([x[0] for x in ref]), np.array([x[1] for x in ref])
            got, gl = od[b, h, list(rows)], ld[b, h, list(rows)]
            assert_within(got, ro, out_bound(ro, delta, vmax, out.dtype, HALF_STEP[out.dtype]), f"out {b},{h}")
            assert_within(gl, rl, delta + 2.0 ** -19 + 2.0 ** -22 * np.abs(rl), f"lse {b},{h}")


def run(rf, q, k, v, window, sinks, scale=SCALE):
    out, lse = rf.attn_prefill_window(q, k, v, window=window, sinks=sinks, scale=scale)
    torch.cuda.synchronize()
    assert rf.rf_device_error() == 0
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("N", [1, 2, 127, 128, 129, 255, 256, 257, 600])
def test_whole_prompts(rf, N, dtype):
    q, k, v = make(N, 1, 2, 1, N, N, DT[dtype])
    for window, sinks in ((0, 0), (1, 0), (100, 4)):
        out, lse = run(rf, q, k, v, window, sinks)
        check(out, lse, q, k, v, window, sinks)


@pytest.mark.parametrize("window,sinks", [(1, 1), (2, 0), (64, 16), (255, 1), (256, 4), (257, 0), (300, 300),
                                          (511, 257), (900, 4), (5000, 7), (0, 9)])
def test_windows_and_sinks(rf, window, sinks):
    q, k, v = make(window, 1, 2, 2, 1100, 1100, torch.bfloat16)
    out, lse = run(rf, q, k, v, window, sinks)
    check(out, lse, q, k, v, window, sinks, rows=list(range(0, 1100, 7)) + [255, 256, 257, 511, 1099])


@pytest.mark.parametrize("N,L", [(1, 1000), (3, 700), (130, 1001), (256, 2000), (300, 813)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (333, 4), (16, 600)])
def test_chunks_behind_a_cache(rf, N, L, window, sinks):
    q, k, v = make(N, 2, 3, 1, N, L, torch.bfloat16)
    out, lse = run(rf, q, k, v, window, sinks)
    check(out, lse, q, k, v, window, sinks, rows=sorted({*range(0, N, 5), N - 1}))


@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (7, 1), (6, 3), (8, 1), (12, 1), (32, 2)])
def test_head_groups(rf, H, Hkv):
    q, k, v = make(H, 2, H, Hkv, 200, 333, torch.float16)
    out, lse = run(rf, q, k, v, 90, 3)
    check(out, lse, q, k, v, 90, 3, rows=range(0, 200, 9))


def test_more_items_than_clusters(rf):
    # several items per cluster: epilogues fall into the next item's first block
    q, k, v = make(3, 2, 32, 8, 1000, 1000, torch.bfloat16)
    out, lse = run(rf, q, k, v, 200, 4)
    check(out, lse, q, k, v, 200, 4, rows=list(range(0, 1000, 97)) + [255, 256, 999])


def test_peaked_scores(rf):
    q, k, v = make(4, 1, 2, 1, 520, 520, torch.bfloat16, gain=12.0)
    out, lse = run(rf, q, k, v, 250, 5)
    check(out, lse, q, k, v, 250, 5, rows=range(0, 520, 3))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_row_reaches_only_the_rows_that_see_it(rf, bad, dtype):
    q, k, v = make(5, 1, 4, 2, 700, 700, DT[dtype])
    v[0, 0, 300, 5:70] = bad             # seen by rows 300..399 of heads 0 and 1
    v[0, 1, 699] = bad                   # by the last row alone
    window, sinks = 100, 2
    out, lse = run(rf, q, k, v, window, sinks)
    check(out, lse, q, k, v, window, sinks, rows=[0, 250, 299, 300, 399, 400, 401, 512, 640, 698, 699])
    fine = torch.isfinite(out[0, 0])
    assert torch.equal(fine.all(-1).nonzero().flatten().cpu(),
                       torch.cat([torch.arange(300), torch.arange(400, 700)]))
    k[0, 0, 120] = float("nan")          # a key row: rows 120..219
    out, lse = run(rf, q, k, v, window, sinks)
    assert torch.equal(torch.isnan(lse[0, 0]).nonzero().flatten().cpu(), torch.arange(120, 220))


@pytest.mark.parametrize("window,sinks", [(64, 4), (0, 0)])
def test_a_bad_first_key_and_bad_queries(rf, window, sinks):
    q, k, v = make(8, 2, 8, 2, 1100, 1100, torch.bfloat16)
    v[:, 0, 0] = float("nan")            # seen by every row of heads 0..3
    v[:, 1, 1, 3] = float("nan")         # one column alone, by all rows but the first
    q[:, 4:, 1000:] = float("nan")
    out, lse = run(rf, q, k, v, window, sinks)
    assert out[:, :4].isnan().all() and lse[:, :4].isfinite().all()
    assert out[:, 4:, 1000:].isnan().all() and lse[:, 4:, 1000:].isnan().all()
    assert lse[:, 4:, :1000].isfinite().all() and out[:, 4:, 0].isfinite().all()
    nan = out[:, 4:, 1:1000].isnan()
    assert nan[..., 3].all() and not nan[..., :3].any() and not nan[..., 4:].any()


def test_padding_may_hold_anything(rf):
    # a prompt of 300 in a buffer of 512: its rows never see what lies behind
    q, k, v = make(6, 1, 2, 1, 512, 512, torch.bfloat16)
    for t in (q, k, v):
        t[:, :, 300:] = float("nan")
    out, lse = run(rf, q, k, v, 64, 4)
    check(out[:, :, :300], lse[:, :, :300], q[:, :, :300], k[:, :, :300], v[:, :, :300], 64, 4,
          rows=range(0, 300, 7))


def test_agrees_with_the_causal_prefill(rf):
    q, k, v = make(7, 2, 4, 4, 777, 777, torch.bfloat16)
    out, lse = run(rf, q, k, v, 0, 0)
    ref, rl = rf.attn_prefill(q, k, v, causal=True, scale=SCALE)
    # two results of the same bounds: each within half a step of the weights and of the output
    assert torch.all((out.double() - ref.double()).abs() <= 2 ** -6 * ref.double().abs() + 2 ** -6 * v.abs().max())
    assert torch.all((lse - rl).abs() <= 1e-4)


def test_long_window_over_many_blocks(rf):
    q, k, v = make(8, 1, 1, 1, 40, 20000, torch.bfloat16)
    out, lse = run(rf, q, k, v, 15000, 300)
    check(out, lse, q, k, v, 15000, 300, rows=[0, 1, 20, 39])


def test_the_same_bits_every_time(rf):
    q, k, v = make(9, 2, 8, 2, 900, 900, torch.bfloat16)
    first = run(rf, q, k, v, 128, 4)
    for _ in range(4):
        again = run(rf, q, k, v, 128, 4)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_captured_and_replayed(rf):
    q, k, v = make(10, 1, 4, 2, 300, 500, torch.bfloat16)
    run(rf, q, k, v, 100, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = rf.attn_prefill_window(q, k, v, window=100, sinks=4, scale=SCALE)
    for seed in (11, 12):
        for dst, src in zip((q, k, v), make(seed, 1, 4, 2, 300, 500, torch.bfloat16)):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        check(out, lse, q, k, v, 100, 4, rows=range(0, 300, 11))


def test_prompt_then_tokens(rf):
    """As a serving loop uses them: a prompt in two chunks, then single tokens over the same cache;
    the last chunk's last row and a decode of the same query agree."""
    B, H, Hkv, cap, window, sinks = 1, 8, 2, 700, 200, 4
    q, k, v = make(20, B, H, Hkv, 600, cap, torch.bfloat16)
    first, _ = run(rf, q[:, :, :350].contiguous(), k[:, :, :350].contiguous(), v[:, :, :350].contiguous(),
                   window, sinks)
    second, lse2 = run(rf, q[:, :, 350:].contiguous(), k[:, :, :600].contiguous(),
                       v[:, :, :600].contiguous(), window, sinks)
    whole, lse = run(rf, q, k[:, :, :600].contiguous(), v[:, :, :600].contiguous(), window, sinks)
    check(torch.cat([first, second], 2), lse, q, k[:, :, :600], v[:, :, :600], window, sinks,
          rows=range(0, 600, 23))
    n = torch.tensor([600], dtype=torch.int32, device="cuda")
    out, l1 = rf.attn_decode_window(q[:, :, 599].contiguous(), k, v, n, window=window, sinks=sinks, scale=SCALE)
    check(out[:, :, None], l1[:, :, None], q[:, :, 599:600], k[:, :, :600], v[:, :, :600], window, sinks)


@pytest.mark.parametrize("N,L,window,sinks", [(1, 1, 0, 0), (5, 400, 300, 2), (33, 33, 7, 1), (70, 391, 256, 64),
                                              (200, 900, 512, 70), (65, 2000, 1984, 65)])
def test_query_heads_of_a_group_share_blocks(rf, N, L, window, sinks):
    # 8, 4 and 2 query heads to an item: covers that end in a narrow block and that do not
    for H, Hkv in ((8, 1), (8, 2), (4, 2)):
        q, k, v = make(N + H, 1, H, Hkv, N, L, torch.bfloat16)
        out, lse = run(rf, q, k, v, window, sinks)
        check(out, lse, q, k, v, window, sinks, rows=sorted({*range(0, N, 13), N - 1}))


# few rows of few heads: a CTA per position and group of query heads
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (8, 2), (16, 1), (17, 1), (40, 1), (128, 4)])
@pytest.mark.parametrize("N,L,window,sinks", [(1, 1, 0, 0), (1, 300, 1, 0), (2, 2, 1, 1), (5, 250, 0, 4),
                                              (7, 5000, 200, 56), (33, 33, 20, 2), (9, 64, 64, 64),
                                              (2, 2000, 900, 64)])
def test_few_rows(rf, H, Hkv, N, L, window, sinks):
    q, k, v = make(N + H, 2, H, Hkv, N, L, torch.bfloat16 if H % 2 else torch.float16)
    out, lse = run(rf, q, k, v, window, sinks)
    check(out, lse, q, k, v, window, sinks)


# as few rows of more heads (over 304 groups): the pair kernel
@pytest.mark.parametrize("B,H,Hkv", [(20, 32, 16), (160, 6, 2), (40, 64, 8)])
@pytest.mark.parametrize("N,L,window,sinks", [(1, 1, 0, 0), (1, 300, 1, 0), (2, 2, 1, 1), (5, 250, 0, 4),
                                              (3, 700, 200, 56), (3, 64, 64, 64)])
def test_few_rows_of_many_heads(rf, B, H, Hkv, N, L, window, sinks):
    q, k, v = make(N + H, B, H, Hkv, N, L, torch.bfloat16)
    out, lse = run(rf, q, k, v, window, sinks)
    pick = slice(0, None, 13)
    check(out[pick], lse[pick], q[pick], k[pick], v[pick], window, sinks)


def test_few_rows_see_nothing_else(rf):
    q, k, v = make(12, 1, 8, 2, 6, 400, torch.bfloat16)
    out, lse = run(rf, q, k, v, 50, 3)
    far = torch.ones(400, dtype=torch.bool)
    far[:3], far[345:] = False, False                    # rows 394..399 see 0..2 and 345..399
    k[:, :, far], v[:, :, far] = float("nan"), float("inf")
    again, lse2 = run(rf, q, k, v, 50, 3)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    v[:, :, 399] = float("nan")                          # the last position's own
    last, _ = run(rf, q, k, v, 50, 3)
    assert last[:, :, 5].isnan().all() and torch.equal(last[:, :, :5], out[:, :, :5])
