"""Steps of a serving loop over a paged cache, every call reading what the one before wrote: page tables,
norm and rotation into the pages, a plan, attention in two layers.  Requests come, send prompts in
chunks, decode, end and give their pages to others."""

import threading

import numpy as np
import pytest
import torch

import cascaded_reductions_gb300 as rf
from cache_helpers import assert_within, normal
from helpers import f64
from oracle import paged
from paged_helpers import few_rows, i32
from test_paged_attn_gpu import check as check_attn
from test_qk_norm_rope_gpu import bound as rope_bound

pytestmark = pytest.mark.gpu

H, HKV, D, PAGE, WIDTH, LAYERS = 8, 2, 128, 16, 24, 2
FREQ = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float()


class Server:
    """A loop's buffers.  ``rows`` are the projection's rows of a step's tokens, per layer."""

    def __init__(self, B, pages, tokens, max_new, window=0, sinks=0, seed=0):
        self.B, self.tokens, self.max_new, self.window, self.sinks = B, tokens, max_new, window, sinks
        new = dict(device="cuda", dtype=torch.int32)
        self.lens, self.news = torch.zeros(B, **new), torch.zeros(B, **new)
        self.table = torch.full((B, WIDTH), -1, **new)
        g = torch.Generator().manual_seed(seed)
        self.stack = torch.randperm(pages, generator=g).int().cuda()
        self.n_free = torch.full((1,), pages, **new)
        # pages as an allocator leaves them: anything, NaN among it
        self.kp, self.vp = (torch.full((LAYERS, pages, HKV, PAGE, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                            for _ in range(2))
        self.weights = [(1 + 0.1 * normal(seed + i, D, dtype=torch.float32)).cuda() for i in (1, 2)]
        self.freq = FREQ.cuda()
        self.plan = None
        self.rows = torch.zeros(LAYERS, tokens, (H + 2 * HKV) * D, dtype=torch.bfloat16, device="cuda")

    def step(self):
        starts, pos, slots, _, _ = rf.page_tables(self.lens, self.news, self.table, self.stack, self.n_free, PAGE,
                                                  self.tokens, lens_out=self.lens, n_free_out=self.n_free)
        self.plan = rf.paged_plan(starts, self.lens, self.tokens, H, HKV, self.max_new, WIDTH * PAGE, self.window,
                                  self.sinks, plan=self.plan)
        outs = []
        for layer in range(LAYERS):
            q, k, v = self.rows[layer].split([H * D, HKV * D, HKV * D], 1)
            q = rf.qk_norm_rope(q.view(-1, H, D), k.view(-1, HKV, D), pos[None], self.freq, *self.weights,
                                v=v.view(-1, HKV, D), slots=slots, kp=self.kp[layer], vp=self.vp[layer])
            outs.append((q, *rf.attn_paged(q, self.kp[layer], self.vp[layer], self.table, self.plan)))
        return starts, pos, slots, outs


SCRIPT = [  # new tokens per request; -1: it has ended
    [5, 0, 100, 1], [1, 40, 70, 1], [1, 1, 1, 17], [90, 1, -1, 1], [1, -1, 200, 1], [1, 130, 1, 3], [-1, 1, 1, 1],
    [16, 1, 0, 33], [1, 1, 4, 1]]


def feed(s, history, news, step):
    """The step's rows, and each request's raw keys and values so far."""
    total = sum(max(0, n) for n in news)
    rows = normal(100 + step, LAYERS, s.tokens, (H + 2 * HKV) * D)
    s.rows.copy_(rows)
    s.news.copy_(i32(news))
    at = 0
    for b, n in enumerate(news):
        if n < 0:
            history[b] = rows[:, :0, H * D:]
        else:
            history[b] = torch.cat([history[b], rows[:, at:at + n, H * D:]], 1)
            at += n
    return total


def check(s, history, starts, outs, news):
    lens = [h.shape[1] for h in history]
    assert s.lens.tolist() == lens
    table = s.table.cpu().numpy()
    kw, freq = f64(s.weights[1]), f64(s.freq)
    for layer, (q, out, lse) in enumerate(outs):
        kp, vp = f64(s.kp[layer]), f64(s.vp[layer])
        for b, L in enumerate(lens):
            if L == 0:
                continue
            raw = f64(history[b][layer]).reshape(L, 2, HKV, D)
            ref, size = paged.norm_rope(raw[:, 0], kw, 1e-6, np.arange(L)[None], freq)
            assert_within(paged.gather(kp, table[b], L).transpose(1, 0, 2), ref,
                          rope_bound(ref, size, torch.bfloat16), f"keys of request {b}")
            assert np.array_equal(paged.gather(vp, table[b], L).transpose(1, 0, 2), raw[:, 1])
        x = dict(q=q, kp=s.kp[layer], vp=s.vp[layer], table=s.table, starts=starts, lens=s.lens,
                 few=few_rows(len(lens), H, HKV, s.max_new, WIDTH * PAGE))
        check_attn(x, out, lse, s.window, s.sinks, rows=[0, 1, 40, 63, 64, -2, -1])


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_steps(window, sinks):
    s = Server(4, 60, 240, 200, window, sinks)
    history = [torch.zeros(LAYERS, 0, 2 * HKV * D, dtype=torch.bfloat16)] * 4
    for step, news in enumerate(SCRIPT):
        feed(s, history, news, step)
        starts, _, _, outs = s.step()
        check(s, history, starts, outs, news)
    assert rf.rf_device_error() == 0


def test_single_tokens_of_a_batch():
    """A loop of decodes alone, behind prompts: the small call's kernel."""
    s = Server(5, 80, 300, 120, seed=3)
    history = [torch.zeros(LAYERS, 0, 2 * HKV * D, dtype=torch.bfloat16)] * 5
    feed(s, history, [100, 17, 1, 64, 118], 0)
    s.step()
    s.plan, s.tokens, s.max_new, s.rows = None, 5, 1, s.rows[:, :5].contiguous()
    for step in range(1, 20):
        feed(s, history, [1] * 5, step)
        starts, _, _, outs = s.step()
    check(s, history, starts, outs, [1] * 5)


def test_captured_step_replayed():
    """One graph of a whole step, replayed with other lengths, chunks and rows."""
    s, eager = Server(4, 60, 240, 200), Server(4, 60, 240, 200)
    s.step(), eager.step()                                     # one-time set-up, and the plans
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            got = s.step()
    history = [torch.zeros(LAYERS, 0, 2 * HKV * D, dtype=torch.bfloat16)] * 4
    mirror = list(history)
    for step, news in enumerate(SCRIPT):
        total = feed(s, history, news, step)
        feed(eager, mirror, news, step)
        torch.cuda.synchronize()
        g.replay()
        want = eager.step()
        torch.cuda.synchronize()
        for a, b in zip(got[:3], want[:3]):
            assert torch.equal(a, b)
        for a, b in zip(got[3], want[3]):
            for x, y in zip(a, b):
                assert torch.equal(x[:total], y[:total])
        assert torch.equal(s.lens, eager.lens) and torch.equal(s.n_free, eager.n_free)
        assert torch.equal(s.table, eager.table)
    check(s, history, got[0], got[3], SCRIPT[-1])


def test_two_threads_with_loops_of_their_own():
    want = []
    for seed in (0, 1):
        s = Server(4, 60, 240, 200, seed=seed)
        history = [torch.zeros(LAYERS, 0, 2 * HKV * D, dtype=torch.bfloat16)] * 4
        for step, news in enumerate(SCRIPT):
            feed(s, history, news, step)
            out = s.step()
        want.append([t.clone() for t in out[3][1][1:]])
    got, errors = [None, None], []

    def loop(seed):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                s = Server(4, 60, 240, 200, seed=seed)
                history = [torch.zeros(LAYERS, 0, 2 * HKV * D, dtype=torch.bfloat16)] * 4
                for step, news in enumerate(SCRIPT):
                    feed(s, history, news, step)
                    out = s.step()
                st.synchronize()
                got[seed] = out[3][1][1:]
        except Exception as e:                                  # noqa: BLE001 (reported below)
            errors.append(e)

    threads = [threading.Thread(target=loop, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    total = sum(SCRIPT[-1])
    for a, b in zip(got, want):
        assert torch.equal(a[0][:total], b[0][:total]) and torch.equal(a[1][:total], b[1][:total])


def test_python_and_quick_calls_agree(monkeypatch):
    if rf._calls is None:
        pytest.skip("the extension is not built")
    runs = []
    for calls in (rf._calls, None):
        monkeypatch.setattr(rf, "_calls", calls)
        s = Server(4, 60, 240, 200)
        history = [torch.zeros(LAYERS, 0, 2 * HKV * D, dtype=torch.bfloat16)] * 4
        feed(s, history, SCRIPT[0], 0)
        starts, pos, slots, lens, n_free = rf.page_tables(s.lens, s.news, s.table, s.stack, s.n_free, PAGE, s.tokens)
        s.lens, s.n_free = lens, n_free
        s.plan = rf.paged_plan(starts, s.lens, s.tokens, H, HKV, s.max_new, WIDTH * PAGE)
        q, k, v = s.rows[0].split([H * D, HKV * D, HKV * D], 1)
        q, k, v = q.view(-1, H, D), k.view(-1, HKV, D), v.view(-1, HKV, D)
        plain = rf.qk_norm_rope(q, k, pos[None], s.freq, s.weights[0])
        q = rf.qk_norm_rope(q, k, pos[None], s.freq, *s.weights, v=v, slots=slots, kp=s.kp[0], vp=s.vp[0])
        out, lse = rf.attn_paged(q, s.kp[0], s.vp[0], s.table, s.plan)
        runs.append([starts, pos, slots, lens, n_free, *plain, q, out[:106], lse[:106], torch.nan_to_num(s.kp[0])])
        # refused by the library
        with pytest.raises(rf.RFError):
            rf.page_tables(s.lens, s.news, s.table, s.stack, s.n_free, 0, s.tokens)
        with pytest.raises(rf.RFError):
            rf.attn_paged(q, s.kp[0], s.vp[0], s.table, s.plan, scale=-1.0)
        with pytest.raises(rf.RFError):
            rf.qk_norm_rope(q, k, pos[None], s.freq[:60].contiguous())
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_pages_whose_offsets_pass_32_bits():
    """A request in the last pages of a cache of 2^31 elements and more."""
    heads, page, pages = 8, 64, 34000
    kp, vp = (torch.zeros(pages, heads, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = 5
    kp[-n:], vp[-n:] = normal(1, n, heads, page, D).cuda(), normal(2, n, heads, page, D).cuda()
    table = i32([[pages - 1 - i for i in range(n)]])
    small = i32([[n - 1 - i for i in range(n)]])
    for new in (1, 7, 200):
        q = normal(3, new, 16, D).cuda()
        starts, lens = i32([0, new]), i32([300])
        plan = rf.paged_plan(starts, lens, new, 16, heads, new, n * page)
        out, lse = rf.attn_paged(q, kp, vp, table, plan)
        ref, rl = rf.attn_paged(q, kp[-n:].contiguous(), vp[-n:].contiguous(), small, plan)
        assert torch.equal(out, ref) and torch.equal(lse, rl) and out.abs().max() > 0
    slots = i32([pages * page - 1 - i for i in range(7)])
    k = normal(5, 7, heads, D).cuda()
    q = normal(6, 7, 16, D).cuda()
    rf.qk_norm_rope(q, k, i32([[0] * 7]), FREQ.cuda(), v=k, slots=slots, kp=kp, vp=vp)
    assert torch.equal(vp[-1, :, -7:].transpose(0, 1).flip(0), k) and torch.equal(kp[-1, :, -7:], vp[-1, :, -7:])
    torch.cuda.empty_cache()


class Tight(Server):
    """A loop whose pool may run out: its plan takes the slots."""

    def step(self):
        starts, pos, slots, _, _ = rf.page_tables(self.lens, self.news, self.table, self.stack, self.n_free, PAGE,
                                                  self.tokens, lens_out=self.lens, n_free_out=self.n_free)
        self.plan = rf.paged_plan(starts, self.lens, self.tokens, H, HKV, self.max_new, WIDTH * PAGE, self.window,
                                  self.sinks, plan=self.plan, slots=slots)
        outs = []
        for layer in range(LAYERS):
            q, k, v = self.rows[layer].split([H * D, HKV * D, HKV * D], 1)
            q = rf.qk_norm_rope(q.view(-1, H, D), k.view(-1, HKV, D), pos[None], self.freq, *self.weights,
                                v=v.view(-1, HKV, D), slots=slots, kp=self.kp[layer], vp=self.vp[layer])
            outs.append((q, *rf.attn_paged(q, self.kp[layer], self.vp[layer], self.table, self.plan)))
        return starts, pos, slots, outs


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_steps_without_enough_pages(window, sinks):
    """Twelve pages: chunks and single tokens that get none, and come again once a request has ended."""
    s = Tight(4, 12, 240, 200, window, sinks, seed=5)
    history = [torch.zeros(LAYERS, 0, 2 * HKV * D, dtype=torch.bfloat16)] * 4
    script = [([100, 5, 30, 1], []), ([70, 1, 40, 1], [0, 2]), ([0, 1, 40, 14], [2]), ([-1, 1, 40, 70], []),
              ([200, 1, 9, 1], [0]), ([0, 190, 0, 1], [1]), ([0, 7, 1, 1], []), ([1, -1, 0, 1], [])]
    for step, (news, refused) in enumerate(script):
        old = list(history)
        feed(s, history, news, 200 + step)
        for b in refused:
            history[b] = old[b]
        starts, _, slots, outs = s.step()
        at, lens = starts.tolist(), [h.shape[1] for h in history]
        assert s.lens.tolist() == lens
        for b, n in enumerate(news):
            assert ((slots[at[b]:at[b + 1]] < 0) == (b in refused)).all(), (step, b)
        # the oracle's request without pages has no keys
        seen = i32([0 if b in refused else n for b, n in enumerate(lens)])
        table, kw, freq = s.table.cpu().numpy(), f64(s.weights[1]), f64(s.freq)
        for layer, (q, out, lse) in enumerate(outs):
            for b, L in enumerate(lens):
                if L == 0:
                    continue
                raw = f64(history[b][layer]).reshape(L, 2, HKV, D)
                ref, size = paged.norm_rope(raw[:, 0], kw, 1e-6, np.arange(L)[None], freq)
                assert_within(paged.gather(f64(s.kp[layer]), table[b], L).transpose(1, 0, 2), ref,
                              rope_bound(ref, size, torch.bfloat16), f"step {step}: keys of request {b}")
                assert np.array_equal(paged.gather(f64(s.vp[layer]), table[b], L).transpose(1, 0, 2), raw[:, 1])
            x = dict(q=q, kp=s.kp[layer], vp=s.vp[layer], table=s.table, starts=starts, lens=seen,
                     few=few_rows(4, H, HKV, s.max_new, WIDTH * PAGE))
            check_attn(x, out, lse, window, sinks, rows=[0, 1, 40, 63, -2, -1])
            for b in refused:
                assert (out[at[b]:at[b + 1]] == 0).all() and torch.isneginf(lse[at[b]:at[b + 1]]).all()
    assert rf.rf_device_error() == 0
