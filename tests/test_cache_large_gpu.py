"""Large calls over a serving cache: rows divided into pieces whose states a launch of its own
merges, with scores and with totals of four keys per thread, alone and as a chain.

A call is small where its pieces fit one wave of two CTAs per SM.  Every case here has more row
groups than that, and asks the library: the pieces that it proposes for them would need more.
"""

import numpy as np
import pytest
import torch

from cache_helpers import DT, assert_within, check_decode, normal
from helpers import f64

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5
CAP = 1700


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def batch(rf, G, Hkv, keys):
    """Sequences of Hkv key heads that make a large call of rows of up to ``keys`` in pieces."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = -(-G // 16)
    B = 2 * sms // (Hkv * tiles) + 1
    S = rf.rf_decode_segments(B * Hkv * tiles, keys)
    assert B * Hkv * tiles * S > 2 * sms and B * Hkv * tiles > 2 * sms, "a small call"
    assert S > 1, "whole rows"
    return B


def lengths(B, cap=CAP):
    """Rows of one, two and three pieces, their limits, and none at all."""
    some = [cap, 0, 1, 767, 768, 769, 1535, 1536, 1537, cap - 1, 64, 65, 1600]
    return [some[b % len(some)] for b in range(B)]


def make(seed, B, H, Hkv, cap, lens, dtype):
    q = normal(seed, B, H, 128, dtype=dtype)
    k, v = normal(seed + 1, B, Hkv, cap, 128, dtype=dtype), normal(seed + 2, B, Hkv, cap, 128, dtype=dtype)
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = float("nan"), float("nan")
    return q.cuda(), k.cuda(), v.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


# groups of one to twenty query heads; S proposed, fewer and more than a row has
@pytest.mark.parametrize("G,Hkv,S,dtype", [(1, 8, None, "bf16"), (4, 8, 2, "fp16"), (3, 8, 3, "bf16"),
                                           (16, 4, 20, "fp16"), (20, 2, None, "bf16"), (4, 8, 1, "bf16")])
def test_rows_in_pieces(rf, G, Hkv, S, dtype):
    B = batch(rf, G, Hkv, CAP)
    lens = lengths(B)
    q, k, v, n = make(1, B, G * Hkv, Hkv, CAP, lens, DT[dtype])
    work = rf.decode_workspace(B, G * Hkv, Hkv, CAP, S=S)
    for t in (work.seg_m, work.seg_l, work.seg_acc):
        t.fill_(float("nan"))                            # whatever the scratch held must not show
    for _ in range(2):
        out, lse = rf.attn_decode_window(q, k, v, n, scale=SCALE, work=work)
    check_decode(out, lse, q, k, v, lens, SCALE)
    assert torch.all(work.counters == 0)


def test_many_pieces_by_row(rf):
    # nine pieces a row: more states than a warp merges per group
    cap, Hkv = 6200, 1
    B = batch(rf, 2, Hkv, cap)
    lens = [cap if b % 9 == 0 else 40 * b % cap for b in range(B)]
    q, k, v, n = make(2, B, 2, Hkv, cap, lens, torch.bfloat16)
    out, lse = rf.attn_decode_window(q, k, v, n, scale=SCALE)
    check_decode(out, lse, q, k, v, lens, SCALE)


def test_window_and_sinks_in_pieces(rf):
    B, window, sinks = batch(rf, 4, 8, 1620), 1600, 20
    lens = lengths(B, 1900)
    q, k, v, n = make(3, B, 32, 8, 1900, lens, torch.bfloat16)
    for b, length in enumerate(lens):
        k[b, :, sinks:max(sinks, length - window)] = float("nan")
        v[b, :, sinks:max(sinks, length - window)] = float("nan")
    out, lse = rf.attn_decode_window(q, k, v, n, window=window, sinks=sinks, scale=SCALE)
    check_decode(out, lse, q, k, v, lens, SCALE, window, sinks)


def check_totals(total, before, w, lens, G, delta):
    """As for the small calls: each weight's share of error, and G + 1 roundings of the total."""
    exact = before + w
    share = np.expm1(2 * delta) + 2.0 ** -18
    assert_within(f64(total), exact, w * share + (G + 1) * 2.0 ** -24 * np.abs(exact) + 1e-30, "weight")
    for b, n in enumerate(lens):
        assert np.array_equal(f64(total)[b, :, n:], before[b, :, n:])


# 2^19 totals and more, rows that stay aligned: four keys per thread; an odd cap: one
@pytest.mark.parametrize("G,cap,dtype", [(4, 1700, "bf16"), (5, 1700, "fp16"), (2, 1701, "bf16"),
                                         (9, 1703, "fp16")])
def test_totals(rf, G, cap, dtype):
    Hkv = 8
    B = batch(rf, G, Hkv, cap)
    assert B * Hkv * cap >= 1 << 19
    lens = lengths(B, cap)
    q, k, v, n = make(4 + G, B, G * Hkv, Hkv, cap, lens, DT[dtype])
    before = torch.rand(B, Hkv, cap, generator=torch.Generator().manual_seed(1))
    work = rf.decode_workspace(B, G * Hkv, Hkv, cap, weights=True)
    for t in (work.seg_m, work.seg_l, work.seg_acc, work.scores):
        t.fill_(float("nan"))
    out, lse, total = rf.attn_decode_weights(q, k, v, n, weight=before.cuda(), scale=SCALE, work=work)
    w, delta = check_decode(out, lse, q, k, v, lens, SCALE)
    check_totals(total, f64(before), w, lens, G, delta)
    # in place, and from nothing
    rf.attn_decode_weights(q, k, v, n, weight=total, weight_out=total, scale=SCALE, work=work)
    check_totals(total, f64(before) + w, w, lens, 2 * G, 2 * delta)
    *_, fresh = rf.attn_decode_weights(q, k, v, n, scale=SCALE, work=work)
    check_totals(fresh, np.zeros_like(w), w, lens, G, delta)


def test_totals_of_many_states(rf):
    # merged by rows, with scores
    cap, Hkv = 6200, 1
    B = batch(rf, 2, Hkv, cap)
    lens = [cap if b % 9 == 0 else 40 * b % cap for b in range(B)]
    q, k, v, n = make(5, B, 2, Hkv, cap, lens, torch.float16)
    out, lse, total = rf.attn_decode_weights(q, k, v, n, scale=SCALE)
    w, delta = check_decode(out, lse, q, k, v, lens, SCALE)
    check_totals(total, np.zeros_like(w), w, lens, 2, delta)


def test_the_same_bits_every_time(rf):
    B = batch(rf, 4, 8, CAP)
    q, k, v, n = make(6, B, 32, 8, CAP, lengths(B), torch.bfloat16)
    first = rf.attn_decode_weights(q, k, v, n, scale=SCALE)
    for _ in range(4):
        assert all(torch.equal(x.nan_to_num(), y.nan_to_num())
                   for x, y in zip(first, rf.attn_decode_weights(q, k, v, n, scale=SCALE)))


# ------------------------------------------------------------------- chain --

class Loop:
    """Decode -> totals -> eviction -> decode of what was kept -> shared prefix, every call's output
    the next one's input and all of them over the same scratch, of large calls alone."""

    def __init__(self, rf):
        self.rf, Hkv, cap, keep, prefix = rf, 8, CAP, 1600, 700
        self.B = batch(rf, 2, Hkv, keep)
        self.keep = keep
        self.q = normal(1, self.B, 16, 128).cuda()
        self.k0, self.v0 = (normal(s, self.B, Hkv, cap, 128).cuda() for s in (2, 3))
        self.kp, self.vp = (normal(s, Hkv, prefix, 128).cuda() for s in (4, 5))
        self.lens0 = torch.tensor([cap - 5 * b for b in range(self.B)], dtype=torch.int32).cuda()
        self.k, self.v, self.lens = (torch.empty_like(t) for t in (self.k0, self.v0, self.lens0))
        # scratch for the most states and scores; every call takes the same
        self.work = rf.decode_workspace(self.B, 16, Hkv, cap, prefix=prefix, weights=True)
        self.kept = [torch.zeros(self.B, Hkv, keep, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.kept.append(torch.zeros(self.B, Hkv, keep, device="cuda"))

    def fill(self):
        self.k.copy_(self.k0)
        self.v.copy_(self.v0)
        self.lens.copy_(self.lens0)

    def empty(self):
        for t in (self.k, self.v, self.lens, *self.kept):
            t.zero_()
        for t in (self.work.seg_m, self.work.seg_l, self.work.seg_acc, self.work.scores):
            t.fill_(float("nan"))
        torch.cuda.synchronize()

    def steps(self, pause):
        rf, q, outs = self.rf, self.q, []
        for _ in range(2):
            a, _ = rf.attn_decode_window(q, self.k, self.v, self.lens, work=self.work)
            pause()
            b, lse, total = rf.attn_decode_weights(a, self.k, self.v, self.lens, work=self.work)
            pause()
            *_, lens, kept = rf.cache_evict(self.k, self.v, total, self.lens, self.keep, sinks=4, recent=32,
                                            out=self.kept)
            pause()
            c, _ = rf.attn_decode_window(b, self.kept[0], self.kept[1], lens, work=self.work)
            pause()
            q, _ = rf.attn_decode_shared(c, self.kp, self.vp, self.kept[0], self.kept[1], lens, work=self.work)
            pause()
            outs += [a, b, lse, total.clone(), lens, kept, c, q]
        return outs


def test_chain_over_one_workspace(rf):
    loop = Loop(rf)
    loop.empty()
    loop.fill()
    want = [x.clone() for x in loop.steps(torch.cuda.synchronize)]
    assert all(x.isfinite().all() for x in want)
    for _ in range(4):
        loop.empty()
        loop.fill()
        got = loop.steps(lambda: None)
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), i
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    loop.empty()
    with torch.cuda.graph(graph, stream=side):
        loop.fill()
        got = loop.steps(lambda: None)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), i
