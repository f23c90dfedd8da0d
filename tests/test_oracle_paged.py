"""Pins of the paged-cache definitions to closed forms, library routines and brute force."""

import numpy as np
import pytest
import torch

from oracle import cache, paged


def test_tables_by_hand():
    # two pages held by the first, none by the second; the stack's top is its end
    starts, pos, slots, lens, n, table, stack = paged.page_tables(
        [5, 0], [4, 3], [[7, 2, -1], [-1, -1, -1]], [9, 4, 1], 3, 4, 9)
    assert starts.tolist() == [0, 4, 7] and lens.tolist() == [9, 3] and n == 1
    assert table.tolist() == [[7, 2, 1], [4, -1, -1]]
    assert pos.tolist() == [5, 6, 7, 8, 0, 1, 2, 0, 0]
    assert slots.tolist() == [2 * 4 + 1, 2 * 4 + 2, 2 * 4 + 3, 4, 16, 17, 18, -1, -1]


def test_tables_no_page_has_two_owners():
    rng = np.random.default_rng(0)
    B, page, width = 12, 3, 9
    table, stack, n = np.full((B, width), -1), np.arange(40), 40
    lens = [0] * B
    for step in range(60):
        news = rng.choice([-1, 0, 1, 2, 7], B, p=[.1, .2, .4, .2, .1]).tolist()
        _, _, slots, lens, n, table, stack = paged.page_tables(lens, news, table, stack, n, page, 200)
        owned = [p for b in range(B) for p in table[b, :paged.pages(lens[b], page)]]
        assert sorted(owned + stack[:n].tolist()) == list(range(40)), step
        written = slots[slots >= 0]
        assert len(set(written.tolist())) == len(written)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x, f = rng.standard_normal((5, 2, 16)), rng.standard_normal(6)
    pos = rng.integers(0, 1000, (1, 5))
    y, size = paged.norm_rope(x, None, 0.0, pos, f, interleaved=interleaved)
    pairs = (lambda z: z[..., 0:12:2] + 1j * z[..., 1:12:2]) if interleaved else (lambda z: z[..., :6] + 1j * z[..., 6:12])
    assert np.allclose(pairs(y), pairs(x) * np.exp(1j * pos[0][:, None, None] * f))
    assert np.array_equal(y[..., 12:], x[..., 12:])
    assert np.all(np.abs(y) <= size + 1e-12)


def test_scores_depend_on_distance_and_axes_are_apart():
    rng = np.random.default_rng(2)
    q, k, f = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8)), np.array([1.0, .3, .1, .03])
    at = lambda x, *p: paged.norm_rope(x, None, 0.0, np.array(p)[:, None], f, axis=[0, 1, 0, 1])[0]   # noqa: E731
    s = lambda p, r: float((at(q, *p) * at(k, *r)).sum())                                       # noqa: E731
    assert np.isclose(s((5, 9), (2, 4)), s((105, 59), (102, 54)))
    assert not np.isclose(s((5, 9), (2, 4)), s((5, 9), (3, 4)))


def test_norm_against_torch():
    x, w = torch.randn(3, 2, 16, dtype=torch.float64), torch.randn(16, dtype=torch.float64)
    y, _ = paged.norm_rope(x.numpy(), w.numpy(), 1e-3, np.zeros((1, 3), int), np.zeros(8))
    assert np.allclose(y, torch.nn.functional.rms_norm(x, (16,), w, 1e-3).numpy())


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 2)])
def test_attention_equals_the_dense_cache(window, sinks):
    """Rows of a chunk, pages shuffled, against the dense definition row by row and torch."""
    rng = np.random.default_rng(3)
    lens, news, page, Hkv, G, D = [11, 4, 9], [3, 4, 1], 4, 2, 2, 8
    dense = rng.standard_normal((2, 3, Hkv, 12, D))
    kp, vp = np.full((20, Hkv, page, D), np.nan), np.full((20, Hkv, page, D), np.nan)
    ids = rng.permutation(20)[:9].reshape(3, 3)
    for b, n in enumerate(lens):
        for t in range(n):
            for x, d in ((kp, dense[0]), (vp, dense[1])):
                x[ids[b, t // page], :, t % page] = d[b, :, t]
    q = rng.standard_normal((9, Hkv * G, D))
    out, lse = paged.attend(q, kp, vp, ids, [0, 3, 7, 8], lens, .4, window, sinks)
    assert np.isnan(out[8]).all()
    t = 0
    for b, (n, new) in enumerate(zip(lens, news)):
        for p in range(n - new, n):
            for h in range(Hkv * G):
                o, z = cache.prefill_row(q[t, h], dense[0][b, h // G], dense[1][b, h // G], p, .4, window, sinks)
                assert np.allclose(out[t, h], o) and np.isclose(lse[t, h], z)
            t += 1
    if not window:
        mask = torch.ones(3, 11, dtype=torch.bool).tril(8)
        ref = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q[:3]).transpose(0, 1),
            torch.from_numpy(dense[0, 0, :, :11]).repeat_interleave(G, 0),
            torch.from_numpy(dense[1, 0, :, :11]).repeat_interleave(G, 0), attn_mask=mask, scale=.4)
        assert np.allclose(out[:3], ref.transpose(0, 1).numpy())


def test_pages_outside_read_as_zeros_and_rows_without_keys():
    kp = np.ones((2, 1, 4, 3))
    out, lse = paged.attend(np.ones((2, 1, 3)), kp, kp * 5, [[1, 7]], [0, 2], [8], 1.0)
    e = np.exp(3)
    assert np.allclose(out[1, 0], 20 * e / (4 * e + 4)) and np.isclose(lse[1, 0], np.log(4 * e + 4))
    out, lse = paged.attend(np.ones((2, 1, 3)), kp, kp, [[1, 7]], [0, 2], [1], 1.0)
    assert np.array_equal(out[0, 0], np.zeros(3)) and lse[0, 0] == -np.inf and lse[1, 0] == 3.0
