"""Page tables against the definition, request by request: every output is a whole number and equal."""

import random

import numpy as np
import pytest
import torch

import cascaded_reductions_gb300 as rf
from oracle import paged
from paged_helpers import i32, tables

pytestmark = pytest.mark.gpu


def check(lens, news, page, width, free, tokens=None, seed=0, in_place=False):
    B = len(lens)
    held = [min(paged.pages(max(0, n), page), width) for n in lens]
    table, stack, P = tables(B, page, held, width, free, seed)
    total = sum(max(0, n) for n in news)
    tokens = max(1, total) if tokens is None else tokens
    ref = paged.page_tables(lens, news, table, stack, free, page, tokens)
    dev = dict(lens=i32(lens), news=i32(news), table=i32(table), stack=i32(stack), n_free=i32([free]))
    out = dict(lens_out=dev["lens"], n_free_out=dev["n_free"]) if in_place else {}
    starts, positions, slots, lens_out, n_free_out = rf.page_tables(
        dev["lens"], dev["news"], dev["table"], dev["stack"], dev["n_free"], page, tokens, **out)
    got = (starts, positions, slots, lens_out, n_free_out[0], dev["table"], dev["stack"])
    names = ("starts", "positions", "slots", "lens", "n_free", "table", "stack")
    for name, g, r in zip(names, got, ref):
        assert np.array_equal(g.cpu().numpy(), r), name
    if not in_place:
        assert dev["lens"].tolist() == list(lens) and dev["n_free"].tolist() == [free]
    return got


@pytest.mark.parametrize("page", [1, 16, 24, 256])
@pytest.mark.parametrize("B", [1, 2, 31, 33, 300, 1025])
def test_mixed_batches(B, page):
    rng = random.Random(B * 1000 + page)
    lens = [rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, 900)]) for _ in range(B)]
    news = [rng.choice([-1, 0, 1, 1, 1, 2, page, rng.randint(1, 40)]) for _ in range(B)]
    width = paged.pages(1000, page) + 1
    need = sum(paged.pages(n + k, page) - paged.pages(n, page) for n, k in zip(lens, news) if k > 0)
    for free in {need, need + 3, need // 2, 0}:
        check(lens, news, page, width, free, seed=B)


def test_first_that_does_not_fit_stops_those_behind_it():
    # pages needed: 1, 3, 0 (inside its last page), 1; two are free
    got = check([16, 16, 17, 32], [1, 40, 3, 1], 16, 8, 2)
    assert got[3].tolist() == [17, 16, 20, 32] and got[4].item() == 1
    assert (got[2].cpu() >= 0).tolist() == [True] + [False] * 40 + [True] * 3 + [False]


def test_pages_given_back_are_taken_in_the_same_step():
    got = check([48, 16, 5], [-1, 33, -1], 16, 4, 0)
    assert got[4].item() == 1 and got[3].tolist() == [0, 49, 0]


def test_more_than_the_table_holds():
    got = check([64, 60, 0], [1, 4, 65], 16, 4, 50)
    assert got[3].tolist() == [64, 64, 0]


@pytest.mark.parametrize("tokens", [1, 5, 1030, 5000])
def test_rows_past_the_total_and_tokens_past_the_rows(tokens):
    check([3, 900, 17], [2, 1023, 0], 16, 200, 100, tokens=tokens)


def test_long_prompts_in_place():
    lens, news = [0, 5000, 31, 0], [40000, 25001, 8192, 3]
    check(lens, news, 64, 700, 1300, in_place=True)


def test_negative_lengths_and_counts():
    check([-5, 7, 0], [3, -9, -1], 16, 3, 4)


def test_large_batch_and_refusal():
    rng = random.Random(3)
    check([rng.randint(0, 60) for _ in range(8192)], [rng.choice([-1, 0, 1, 5]) for _ in range(8192)],
          16, 5, 6000)
    z = i32(np.zeros(8193))
    with pytest.raises(rf.RFError):
        rf.page_tables(z, z, z.view(-1, 1), i32(np.zeros(4)), i32([4]), 16, 8)


def test_captured_steps_in_place():
    """One token per step, replayed: lengths and the stack go on from replay to replay."""
    B, page, width = 5, 16, 20
    lens, free = [0, 15, 16, 31, 7], 40
    table, stack, _ = tables(B, page, [paged.pages(n, page) for n in lens], width, free, 1)
    d = [i32(lens), i32([1] * B), i32(table), i32(stack), i32([free])]
    step = lambda: rf.page_tables(*d, page, B, lens_out=d[0], n_free_out=d[4])      # noqa: E731
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = step()
    for _ in range(40):
        ref = paged.page_tables(lens, [1] * B, table, stack, free, page, B)
        g.replay()
        torch.cuda.synchronize()
        lens, free, table, stack = ref[3], ref[4], ref[5], ref[6]
        assert out[2].tolist() == ref[2].tolist()
        assert d[0].tolist() == list(lens) and d[4].item() == free
        assert np.array_equal(d[2].cpu().numpy(), table)


def test_outputs_are_tensors_of_their_own():
    """They may share memory behind them, but no element, and each can be sliced, viewed and written."""
    lens, news, stack = i32([3, 0, 17]), i32([2, 1, 0]), i32(list(range(8)))
    table = i32(np.full((3, 4), -1))
    table[0, 0], table[2, :2] = 6, i32([5, 7])
    outs = rf.page_tables(lens, news, table, stack, i32([5]), 16, 5)
    want = [t.clone() for t in outs]
    assert [tuple(t.shape) for t in outs] == [(4,), (5,), (5,), (3,), (1,)]
    for i, t in enumerate(outs):
        assert t.is_contiguous() and t.dtype == torch.int32 and t.data_ptr() % 16 == 0
        t.view(-1, 1).fill_(-7)
        for j, other in enumerate(outs):
            if j > i:
                assert torch.equal(other, want[j])
    assert outs[1][1:3].tolist() == [-7, -7]


def filled(n, x=7):
    return torch.full((n,), x, dtype=torch.int32, device="cuda")


def test_as_many_rows_as_an_int_counts():
    """T = 2^31 - 1, near which a thread's next row passes the largest int."""
    lens, news, page, width, free, T = [0, 33], [20000, 5], 16, 1260, 1260, 2 ** 31 - 1
    table, stack, _ = tables(2, page, [0, 3], width, free, 4)
    total = sum(news)
    ref = paged.page_tables(lens, news, table, stack, free, page, total)
    positions, slots = filled(T), filled(T)
    starts, lens_out, n_free_out, dev_table = filled(3), filled(2), filled(1), i32(table)
    rf.rf_page_tables(i32(lens), i32(news), dev_table, i32(stack), i32([free]), page, starts, positions, slots, lens_out,
                      n_free_out)
    for got, want in zip((starts, positions[:total], slots[:total], lens_out, n_free_out[0], dev_table), ref):
        assert np.array_equal(got.cpu().numpy(), want)
    for at in range(total, T, 1 << 28):
        assert (positions[at:at + (1 << 28)] == 0).all() and (slots[at:at + (1 << 28)] == -1).all(), at


def test_as_many_pages_as_an_int_counts():
    """A stack of 2^31 - 1 pages, whose top the pages given back reach and are taken from."""
    P, given, taken = 2 ** 31 - 1, 20000, 9000
    table = filled(2 * given).view(2, given)
    table[0] = torch.arange(given, dtype=torch.int32, device="cuda") + 5
    stack = filled(P, -3)
    starts, positions, slots, lens_out, n_free_out = rf.page_tables(
        i32([given, 0]), i32([-1, taken]), table, stack, i32([P - given]), 1, taken)
    assert n_free_out.item() == P - taken and lens_out.tolist() == [0, taken]
    assert torch.equal(stack[P - given:], table[0])
    assert torch.equal(table[1, :taken], table[0].flip(0)[:taken]) and (table[1, taken:] == 7).all()
    assert torch.equal(slots, table[1, :taken]) and torch.equal(positions, torch.arange(taken, device="cuda").int())
    assert (stack[:P - given][-(1 << 20):] == -3).all() and (stack[:1 << 20] == -3).all()


def test_requests_that_only_end():
    """A step without new tokens."""
    table, stack, _ = tables(3, 16, [2, 0, 3], 4, 5, 6)
    ref = paged.page_tables([20, 0, 48], [-1, 0, -1], table, stack, 5, 16, 0)
    dev_table, dev_stack = i32(table), i32(stack)
    got = rf.page_tables(i32([20, 0, 48]), i32([-1, 0, -1]), dev_table, dev_stack, i32([5]), 16, 0)
    for g, r in zip((*got[:4], got[4][0], dev_table, dev_stack), ref):
        assert tuple(g.shape) == np.shape(r) and np.array_equal(g.cpu().numpy(), r)
    with pytest.raises((ValueError, RuntimeError)):
        rf.page_tables(i32([20]), i32([1]), i32([[0, 1]]), i32([3, 2]), i32([2]), 16, -1)
