"""Attention over a paged cache against the definition in float64, row by row.

Bounds as for the calls over a dense cache: the score's fp32 rounding, the weights' rounding for the
second product (requests of few rows per key head: two 16-bit terms, 2^-16; larger ones, where each
weight is rounded once to the 16-bit type: half a step of it) and one rounding of the output.  Rows of the pages that no request uses hold
NaN."""

import numpy as np
import pytest
import torch

import cascaded_reductions_gb300 as rf
from cache_helpers import DT, HALF_STEP, assert_within, normal, out_bound
from helpers import f64
from oracle import cache as C
from oracle import paged
from paged_helpers import few_rows, i32, paged_cache

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


def make(lens, news, H, Hkv, page, dtype=torch.bfloat16, seed=0, gain=1.0, extra=0, fill=float("nan")):
    kp, vp, table = paged_cache(lens, Hkv, page, seed, dtype, fill=fill)
    starts = np.concatenate([[0], np.cumsum(news)])
    q = (normal(seed + 7, int(starts[-1]) + extra, H, 128, dtype=dtype) * gain)
    return dict(q=q.cuda(), kp=kp.cuda(), vp=vp.cuda(), table=i32(table), starts=i32(starts), lens=i32(lens))


def call(x, window=0, sinks=0, scale=SCALE, max_new=None, max_len=None, plan=None):
    kp, st = x["kp"], x["starts"].tolist()
    news = [b - a for a, b in zip(st, st[1:])]
    max_new, max_len = max_new or max(max(news), 1), max_len or x["table"].shape[1] * kp.shape[2]
    x["few"] = few_rows(len(news), x["q"].shape[1], kp.shape[1], max_new, max_len)
    plan = rf.paged_plan(x["starts"], x["lens"], x["q"].shape[0], x["q"].shape[1], kp.shape[1], max_new, max_len,
                         window, sinks, plan=plan)
    out, lse = rf.attn_paged(x["q"], kp, x["vp"], x["table"], plan, scale=scale)
    torch.cuda.synchronize()
    assert rf.rf_device_error() == 0
    return out, lse


def check(x, out, lse, window=0, sinks=0, scale=SCALE, rows=None, finite=True):
    """Every row of every request, or of each the listed ones (from its end where negative)."""
    q, kp, vp, od, ld = (f64(t) for t in (x["q"], x["kp"], x["vp"], out, lse))
    table, starts, lens = (x[k].cpu().numpy() for k in ("table", "starts", "lens"))
    H, G = q.shape[1], q.shape[1] // kp.shape[1]
    for b, L in enumerate(lens):
        N = starts[b + 1] - starts[b]
        if N == 0:
            continue
        k, v = paged.gather(kp, table[b], L), paged.gather(vp, table[b], L)
        fk, fv = (np.nan_to_num(t, posinf=0, neginf=0) for t in (k, v))
        p_step = 2.0 ** -16 if N * G <= x["few"] else HALF_STEP[out.dtype]
        vmax = float(np.abs(fv).max()) if L else 0.0
        mine = range(N) if rows is None else sorted({r % N for r in rows})
        for h in range(H):
            delta = C.score_error(q[starts[b]:starts[b + 1], h], fk[h // G], scale)
            for i in mine:
                keys = C.visible(L - N + i, window, sinks) if L - N + i >= 0 else []
                with np.errstate(invalid="ignore"):
                    ro, rl, _ = C.attend(q[starts[b] + i, h], k[h // G][keys], v[h // G][keys], scale)
                what = f"request {b} (L {L}, N {N}), row {i}, head {h}"
                fine = np.where(np.isfinite(ro), ro, 0)
                bound = np.where(np.isfinite(ro), out_bound(fine, delta, vmax, out.dtype, p_step), 0)
                assert_within(od[starts[b] + i, h], ro, bound, what)
                if np.isneginf(rl):
                    assert np.isneginf(ld[starts[b] + i, h]), what
                elif finite or np.isfinite(rl):
                    assert_within(ld[starts[b] + i, h], rl, delta + 2.0 ** -19 + 2.0 ** -22 * np.abs(rl), "lse " + what)


def run(lens, news, H, Hkv, page, window=0, sinks=0, rows=None, **o):
    x = make(lens, news, H, Hkv, page, **o)
    out, lse = call(x, window, sinks)
    check(x, out, lse, window, sinks, rows=rows)
    return x, out, lse


# ------------------------------------------------------------ single tokens --

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (5, 1), (32, 2), (40, 2), (1, 1)])
def test_single_tokens(H, Hkv, page, dtype):
    lens = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 255, 256, 257, 600]
    run(lens, [1] * len(lens), H, Hkv, page, dtype=DT[dtype], seed=page + H)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 16), (100, 17), (333, 64), (5000, 4), (0, 9),
                                          (40, 900)])
@pytest.mark.parametrize("news", [1, 3, 40])
def test_windows_and_sinks(window, sinks, news):
    """Single tokens, drafts and chunks (40 tokens of 4 heads: the pair kernel)."""
    lens = [n for n in (1, 17, 40, 64, 65, 300, 1111) if n >= news]
    run(lens, [news] * len(lens), 8, 2, 16, window, sinks, seed=window)


def test_one_long_request_in_pieces():
    run([20000], [1], 8, 2, 64, seed=1)
    run([9000], [1], 32, 8, 16, window=8000, sinks=4, seed=2)


def test_many_requests():
    """More pieces than the device holds at once, taken from the queue; whole and divided rows."""
    lens = [4000 - 37 * b for b in range(100)]
    run(lens, [1] * 100, 8, 8, 128, rows=[0], seed=3)
    lens[50] = 30000
    x, out, lse = run(lens, [1] * 100, 16, 8, 32, rows=[0], seed=4)
    again = call(x)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_small_call_of_more_units_than_ctas():
    lens = [200 - b for b in range(60)]
    x, out, lse = run(lens, [1] * 60, 16, 8, 16, rows=[0], seed=5)
    again = call(x)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("top,news", [(16, 1), (40, 1), (70, 3), (300, 2)])
def test_many_short_requests_where_long_ones_may_come(top, news):
    """A large call by its sizes (a queue of units) of units with fewer keys than are kept in flight."""
    lens = [max(news, 1 + (37 * b) % top) for b in range(90)]
    x = make(lens, [news] * 90, 16, 8, 16, seed=top)
    out, lse = call(x, max_len=x["table"].shape[1] * 16)
    x["table"] = torch.cat([x["table"], torch.full((90, 512), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    for _ in range(2):
        out, lse = call(x)
        check(x, out, lse, rows=[0, -1])


@pytest.mark.parametrize("news", [1, 5, 100])
def test_window_that_hides_nothing_and_sinks_without_one(news):
    """The same bits as without: no row is as far from its first key."""
    x = make([300, 150], [news, news], 8, 2, 32, seed=news)
    want = call(x)
    for window, sinks in ((320, 4), (2 ** 31 - 1, 2 ** 31 - 1), (0, 7)):
        got = call(x, window, sinks)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(x, *call(x, 299, 2 ** 31 - 1), 299, 400, rows=[0, -1])


# -------------------------------------------------------------- few and many --

@pytest.mark.parametrize("H,Hkv,news", [(32, 8, 8), (32, 8, 9), (16, 16, 33), (12, 4, 11), (12, 4, 22), (64, 2, 2)])
def test_rows_on_either_side_of_few_in_a_large_call(H, Hkv, news):
    """Requests of 32 to 96 rows per key head, one to four times what one reading of the keys serves."""
    lens = [2000, 700, 1300, news, 64, 900, 1111, 257, 300, 800, 1500, 600, 999, 1024]
    x, out, lse = run(lens, [news] * 14, H, Hkv, 64, rows=[0, -1], seed=news)
    assert x["few"] < 64 or news * H // Hkv > 64 or H == 64 or H == 12
    assert torch.equal(out, call(x)[0])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,Hkv,news", [(4, 1, 2), (8, 2, 4), (8, 8, 9), (5, 1, 7), (64, 4, 3), (4, 1, 16), (7, 7, 64)])
def test_few_tokens(H, Hkv, news, dtype):
    lens = [news, news + 1, news + 15, 100, 257, 700]
    run(lens, [news] * len(lens), H, Hkv, 32, dtype=DT[dtype], seed=news)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (4, 2), (4, 1), (8, 1), (5, 1)])
def test_whole_prompts(H, Hkv, page, dtype):
    lens = [65, 66, 127, 128, 129, 255, 256, 257, 300, 513]
    run(lens, lens, H, Hkv, page, dtype=DT[dtype], seed=page + H, rows=[0, 1, 31, 32, 63, 64, 128, 200, -2, -1])


@pytest.mark.parametrize("page", [16, 256])
def test_chunks_behind_a_cache(page):
    news = [70, 100, 33, 200, 64, 129]
    lens = [n + past for n, past in zip(news, (1, 250, 256, 777, 1500, 4000))]
    run(lens, news, 8, 2, page, seed=page, rows=[0, 1, 31, 32, 62, 63, -2, -1])


@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 4), (256, 300), (255, 1), (1000, 513), (700, 0)])
def test_windowed_chunks(window, sinks):
    news = [300, 513, 100]
    lens = [300, 2200, 1999]
    run(lens, news, 4, 1, 32, window, sinks, seed=window, rows=[0, 1, 63, 64, 100, 255, 256, -2, -1])


@pytest.mark.parametrize("page", [16, 64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(300, 1), (257, 64), (700, 65), (200, 128), (640, 190), (129, 200)])
def test_sinks_in_the_window_s_lowest_block(window, sinks, page):
    """Tiles whose lowest block begins with room for the sinks, and tiles beside them without."""
    run([1500, 900, 777], [400, 130, 777], 8, 1, page, window, sinks, seed=window + page, rows=list(range(0, 400, 13)))


def test_mixed_batch():
    news = [1, 200, 0, 5, 1, 77, 0, 1, 16, 300]
    lens = [900, 500, 40, 5, 1, 1300, 0, 256, 16, 300]
    run(lens, news, 8, 2, 64, seed=5, rows=[0, 1, 17, 64, -1])
    run(lens, news, 8, 2, 16, 90, 5, seed=6, dtype=torch.float16, rows=[0, 1, 17, 64, -1])


def test_few_tiles_over_many_keys():
    """A tile's blocks are cut between many clusters."""
    run([30000], [65], 4, 1, 64, seed=7, rows=[0, 33, -1])
    run([9000, 7000], [128, 40], 8, 4, 16, seed=8, rows=[0, 33, -1], dtype=torch.float16)


def test_long_prompts_in_rounds():
    """More keys than a round's: blocks are dealt out in several."""
    x, out, lse = run([9000, 8000, 3000], [9000, 6000, 3000], 16, 8, 128, seed=9, rows=[0, 999, 2047, -1])
    again = call(x)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


# ------------------------------------------------------------------- masks --

@pytest.mark.parametrize("B,L,N,H,Hkv", [(16, 3165, 340, 64, 32), (11, 5276, 1181, 32, 16)])
def test_equal_prompts_in_rounds(B, L, N, H, Hkv):
    """Requests that are all the same, over the same pages: tiles of equal length, whose ends all
    ranges of a cluster miss in the same direction.  Each request against the first, which is against
    the definition; the plan's memory holds 3e9 before, so that a part which nobody wrote shows (NaN columns are
    computed again)."""
    x = make([L], [N], H, Hkv, 64, seed=B)
    x = dict(x, q=x["q"].repeat(B, 1, 1), table=x["table"].repeat(B, 1), starts=i32(np.arange(B + 1) * N),
             lens=i32([L] * B))
    plan = rf.paged_plan(x["starts"], x["lens"], B * N, H, Hkv, N, x["table"].shape[1] * 64)
    plan.plan.view(torch.uint8).fill_(0x4f)
    out, lse = call(x, plan=plan)
    one = dict(x, q=x["q"][:N], table=x["table"][:1], starts=i32([0, N]), lens=i32([L]))
    check(one, out[:N], lse[:N], rows=[0, 100, 255, -1])
    q, k = f64(one["q"]), paged.gather(f64(x["kp"]), x["table"][0].cpu().numpy(), L)
    delta = max(C.score_error(q[:, h], k[h // (H // Hkv)], SCALE) for h in range(H))
    vmax = float(np.abs(np.nan_to_num(f64(x["vp"]))).max())
    out, lse = out.view(B, N, H, 128).float(), lse.view(B, N, H)
    # both are off by their bounds at most, and so is the value that a bound is taken of
    off = torch.from_numpy(np.float32(1.01 * out_bound(f64(out[0]), delta, vmax, torch.bfloat16, HALF_STEP[torch.bfloat16])))
    off, off_lse = off.cuda(), delta + 2.0 ** -19 + 2.0 ** -22 * lse[0].abs()
    for b in range(1, B):
        assert ((out[b] - out[0]).abs() <= 2 * off).all(), b
        assert ((lse[b] - lse[0]).abs() <= 2 * off_lse).all(), b


@pytest.mark.parametrize("news", [1, 3, 70])
def test_rows_without_keys_and_empty_requests(news):
    """New tokens that are not in the cache (lens < new) stand at negative positions."""
    x = make([max(1, news - 2), 40, 0, 100], [news, 0, news, 2], 4, 2, 16, seed=news)
    out, lse = call(x)
    check(x, out, lse)


@pytest.mark.parametrize("news", [2, 100])
def test_scores_of_minus_infinity(news):
    x = make([100, 100], [news, news], 4, 1, 16, seed=1)
    x["q"] = x["q"].abs()
    x["q"][1] = 0                                # this row's scores are NaN (0 * -inf)
    x["kp"][x["table"][0].long()] = -float("inf")
    out, lse = call(x)
    seen = torch.arange(news) != 1
    assert (out[:news][seen] == 0).all() and torch.isneginf(lse[:news][seen]).all()
    assert torch.isnan(out[1]).all()
    x["starts"], x["q"] = i32([0, 0, news]), x["q"][news:]
    check(x, out[news:], lse[news:])


@pytest.mark.parametrize("news,H", [(1, 8), (4, 8), (60, 8), (300, 4)])
@pytest.mark.parametrize("page", [16, 256])
def test_values_that_are_not_finite(page, news, H):
    lens = [news + 300, news + 77]
    x = make(lens, [news, news], H, 2, page, seed=news, dtype=torch.float16)
    vp, kp, table = x["vp"], x["kp"], x["table"].tolist()
    at = lambda b, t: (table[b][t // page], slice(None), t % page)                      # noqa: E731
    vp[at(0, 5)][:, 3] = float("inf")            # seen by all
    vp[at(0, 6)][:, 4] = float("nan")
    vp[at(0, lens[0] - 1)][:, 7] = float("nan")  # by the last row alone
    vp[at(0, lens[0] - news // 2 - 1)][:, 9] = -float("inf")
    kp[at(1, lens[1] - news // 2 - 1)] = float("nan")
    out, lse = call(x)
    check(x, out, lse, finite=False, rows=[0, 1, news // 2 - 1, news // 2, news // 2 + 1, -2, -1])
    check(x, *call(x, 64, 4), 64, 4, finite=False, rows=[0, 1, news // 2, -2, -1])


def test_nan_in_an_early_key_of_a_long_prompt():
    x = make([3000], [3000], 8, 2, 64, seed=2)
    x["vp"][x["table"][0, 0].item(), :, 1, 5] = float("nan")
    out, lse = call(x)
    check(x, out, lse, rows=[0, 1, 2, 500, 2999])
    assert torch.isnan(out[1:, :, 5]).all() and not torch.isnan(out[:, :, :5]).any()
    # the note of it does not stay
    x["vp"][x["table"][0, 0].item(), :, 1, 5] = 0
    out, lse = call(x)
    check(x, out, lse, rows=[0, 1, 2999])


@pytest.mark.parametrize("news", [1, 90])
def test_page_numbers_outside_the_cache_read_as_zeros(news):
    lens = [news + 100, news + 40]
    x = make(lens, [news, news], 8, 2, 16, seed=3)
    for i, bad in enumerate((-1, x["kp"].shape[0], 2 ** 31 - 1, -2 ** 31)):
        x["table"][0, i] = bad
    out, lse = call(x)
    check(x, out, lse)


def test_large_scores():
    for news in (1, 100):
        run([500], [news], 4, 2, 16, seed=4, gain=300.0, dtype=torch.float16, rows=[0, 50, -1])
        run([500], [news], 4, 2, 16, seed=4, gain=1e6, rows=[0, 50, -1])


def test_dominant_key():
    """One key far above thousands: small fp16 weights are not lost."""
    for news in (1, 65):
        x = make([9000], [news], 4, 1, 64, seed=5, dtype=torch.float16)
        x["kp"].mul_(0.01)
        x["q"].fill_(1.0)
        x["kp"][x["table"][0, 0].item(), 0, 0] = 1.2
        out, lse = call(x)
        check(x, out, lse, rows=[0, 33, -1])


# ----------------------------------------------------------------- the call --

def test_rows_of_no_request_are_left():
    x = make([50, 200, 70], [1, 100, 2], 8, 2, 16, extra=9, seed=6)
    x["few"] = few_rows(len(x["lens"]), 8, 2, 100, 208)
    plan = rf.paged_plan(x["starts"], x["lens"], x["q"].shape[0], 8, 2, 100, 208)
    out, lse = torch.full_like(x["q"], 7.0), torch.full((112, 8), 7.0, device="cuda")
    rf.rf_attn_paged(x["q"], x["kp"], x["vp"], x["table"], plan.plan, 100, 208, 0, 0, SCALE, out, lse)
    check(x, out, lse, rows=[0, 31, 96, -1])
    assert (out[103:] == 7).all() and (lse[103:] == 7).all()
    rf.rf_attn_paged(x["q"], x["kp"], x["vp"], x["table"], plan.plan, 100, 208, 0, 0, SCALE, out, None)
    check(x, out, lse, rows=[-1])


def test_plan_of_other_sizes_is_not_used():
    x = make([50, 200], [1, 100], 8, 2, 16, seed=6)
    plan = rf.paged_plan(x["starts"], x["lens"], 101, 8, 2, 100, 300)
    out = torch.full_like(x["q"], 7.0)
    rf.rf_attn_paged(x["q"], x["kp"], x["vp"], x["table"], plan.plan, 100, 200, 0, 0, SCALE, out)
    rf.rf_attn_paged(x["q"], x["kp"], x["vp"], x["table"], torch.zeros_like(plan.plan), 100, 208, 0, 0, SCALE, out)
    assert (out == 7).all()
    with pytest.raises(ValueError):
        rf.attn_paged(x["q"][:50], x["kp"], x["vp"], x["table"], plan)
    with pytest.raises(ValueError):
        rf.paged_plan(x["starts"], x["lens"], 101, 8, 2, 100, 301, plan=plan)
    with pytest.raises(rf.RFError):
        rf.rf_attn_paged(x["q"], x["kp"], x["vp"], x["table"], plan.plan[:1024], 100, 208, 0, 0, SCALE, out)


def test_sizes_above_the_lengths_and_lengths_above_them():
    x = make([100, 30], [2, 1], 8, 2, 16, seed=7)
    check(x, *call(x, max_new=3, max_len=100))
    y = dict(x, lens=i32([100, 2 ** 31 - 1]), starts=i32([-5, 2, 2 ** 31 - 1]))     # cut to 112 keys, 3 rows
    out, lse = call(y, max_new=3)
    check(dict(x, starts=i32([0, 2, 2])), out, lse)


def test_on_another_stream():
    x = make([3000, 700], [130, 1], 8, 2, 64, seed=8)
    want = call(dict(x))
    s = torch.cuda.Stream()
    for _ in range(5):
        y = {k: torch.zeros_like(v) for k, v in x.items()}
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
            for k in y:
                y[k].copy_(x[k])
        plan = rf.paged_plan(y["starts"], y["lens"], 131, 8, 2, 130, 3008, stream=s)
        out, lse = rf.attn_paged(y["q"], y["kp"], y["vp"], y["table"], plan, stream=s)
        s.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_captured_and_replayed_with_other_lengths():
    """Plan and attention in a graph; the lengths and rows change between replays."""
    x = make([300, 300, 300], [90, 90, 90], 8, 2, 32, seed=9, fill=0.0)
    call(x)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            plan = rf.paged_plan(x["starts"], x["lens"], 270, 8, 2, 90, 320)
            out, lse = rf.attn_paged(x["q"], x["kp"], x["vp"], x["table"], plan)
    x["few"] = few_rows(3, 8, 2, 90, 320)
    for lens, starts in (([300, 300, 300], [0, 90, 180, 270]), ([1, 77, 256], [0, 1, 1, 30]), ([300, 16, 9], [0, 80, 90, 99])):
        x["lens"].copy_(i32(lens))
        x["starts"].copy_(i32(starts))
        g.replay()
        torch.cuda.synchronize()
        check(x, out, lse, rows=[0, 5, 33, -1])


# --------------------------------------------------------- requests without pages --

@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 3)])
@pytest.mark.parametrize("B,news,keys", [(5, 1, 64), (5, 3, 64), (90, 2, 9000), (5, 70, 64), (5, 300, 64)])
def test_requests_without_pages(B, news, keys, window, sinks):
    """Small calls, a queue of units, the pair kernel: rows of a request whose first slot is negative get
    0 and -inf, those beside it what they get without it."""
    lens = [news + (37 * b) % 400 for b in range(B)]
    x = make(lens, [news] * B, 8, 2, 16, seed=news + B)
    width = max(x["table"].shape[1], keys // 16)
    x["table"] = torch.nn.functional.pad(x["table"], (0, width - x["table"].shape[1]), value=-1)
    T = B * news
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    refused = [0, 2, B - 1]
    for b in refused:
        slots[b * news:(b + 1) * news] = -1
    want = call(x, window, sinks)
    plan = rf.paged_plan(x["starts"], x["lens"], T, 8, 2, news, width * 16, window, sinks, slots=slots)
    out, lse = rf.attn_paged(x["q"], x["kp"], x["vp"], x["table"], plan)
    off = torch.zeros(B, dtype=torch.bool, device="cuda")
    off[refused] = True
    off = off.repeat_interleave(news)
    assert (out[off] == 0).all() and torch.isneginf(lse[off]).all()
    x["lens"] = torch.where(torch.isin(torch.arange(B, device="cuda"), torch.tensor(refused, device="cuda")), 0, x["lens"])
    check(x, out, lse, window, sinks, rows=[0, -1])
    # the same plan's memory again, for a step in which all have their places
    rf.paged_plan(x["starts"], i32(lens), T, 8, 2, news, width * 16, window, sinks, plan=plan, slots=torch.arange(
        T, dtype=torch.int32, device="cuda"))
    out, lse = rf.attn_paged(x["q"], x["kp"], x["vp"], x["table"], plan)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_slots_of_another_size_are_refused():
    with pytest.raises(ValueError):
        rf.paged_plan(i32([0, 4]), i32([9]), 4, 8, 2, 4, 16, slots=i32([1, 2, 3]))


@pytest.mark.parametrize("H,Hkv,news,kernel", [(32, 8, 8, "streaming"), (32, 8, 9, "pairs"), (16, 16, 32, "streaming"),
                                               (16, 16, 33, "pairs"), (12, 4, 21, "streaming"), (12, 4, 22, "pairs"),
                                               (64, 2, 2, "streaming"), (64, 2, 3, "pairs")])
def test_rows_at_the_limit_of_a_large_call(H, Hkv, news, kernel):
    """On either side of the rows per key head up to which a large call streams, 32 times G over the heads
    that the other kernel packs (32 at G = 4 and 1; 64 at most, 63 and 66 rows at G = 3; 64 and 96 at G = 32):
    weights in two 16-bit terms up to it."""
    G, sms = H // Hkv, torch.cuda.get_device_properties(0).multi_processor_count
    lens = [2000, 700, 1300, news, 64, 900, 1111, 257, 300, 800, 1500, 600, 999, 1024]
    x = make(lens, [news] * 14, H, Hkv, 64, seed=news + H)
    max_len = 64 * x["table"].shape[1]
    while 14 * Hkv * -(-news * G // 16) * -(-max_len // 64) <= 32 * sms:      # small: room for longer requests
        max_len += 6400
    width = max_len // 64
    x["table"] = torch.nn.functional.pad(x["table"], (0, width - x["table"].shape[1]), value=-1)
    out, lse = call(x)
    # the documented rule: a large call, and the request on the side of it that the case is for
    few = few_rows(14, H, Hkv, news, max_len)
    assert few == x["few"] == min(64, 32 * G // max(g for g in (8, 4, 2, 1) if G % g == 0))
    assert not (news * G <= 64 and 14 * Hkv * -(-news * G // 16) * -(-max_len // 64) <= 32 * sms)
    assert kernel == ("streaming" if news * G <= few else "pairs")
    check(x, out, lse, rows=[0, -1])


def test_scratch_goes_by_what_is_divided():
    """States are kept of divided tiles alone, however many requests there are."""
    for B, Hkv in ((1024, 8), (1024, 32), (8192, 8)):
        size = rf.rf_paged_plan_bytes(B, B + 4096, 32, Hkv, 4096, 32768)
        assert 0 < size < 80 << 20, size
    # whole tiles between divided ones, behind memory that holds 3e9
    lens = [9000 if b % 97 == 5 else 1 + b % 60 for b in range(700)]
    x = make(lens, [1] * 700, 16, 8, 16, seed=700)
    plan = rf.paged_plan(x["starts"], x["lens"], 700, 16, 8, 1, x["table"].shape[1] * 16)
    plan.plan.fill_(0x4f)
    out, lse = call(x, plan=plan)
    some = [0, 4, 5, 6, 101, 102, 103, 296, 399, 493, 684, 699]
    starts = np.arange(len(some) + 1)
    at = torch.tensor(some, device="cuda")
    check(dict(q=x["q"][at], kp=x["kp"], vp=x["vp"], table=x["table"][at], starts=i32(starts), lens=x["lens"][at],
               few=x["few"]), out[at], lse[at])
