"""Pins of oracle/cache.py to something other than itself: torch's float64
softmax attention with an explicit mask, closed forms, the invariance of a
split and merged softmax, and brute force for the eviction."""

import itertools

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import cache as C


def rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (3, 0), (3, 2), (2, 5), (40, 3), (7, 40)])
def test_visible_keys_are_the_mask(window, sinks):
    for p in range(20):
        mask = [j <= p and (window == 0 or j > p - window or j < sinks) for j in range(20)]
        assert np.array_equal(C.visible(p, window, sinks), np.flatnonzero(mask))
    assert len(C.visible(-1, window, sinks)) == 0


@pytest.mark.parametrize("window,sinks", [(0, 0), (5, 0), (5, 2), (30, 4)])
def test_rows_against_torch_attention_with_a_mask(window, sinks):
    g = rng(1)
    q, k, v = g.normal(size=(23, 16)), g.normal(size=(23, 16)), g.normal(size=(23, 8))
    i, j = np.arange(23)[:, None], np.arange(23)[None]
    mask = (j <= i) & ((window == 0) | (j > i - window) | (j < sinks))
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q)[None], torch.from_numpy(k)[None], torch.from_numpy(v)[None],
        attn_mask=torch.from_numpy(mask)[None], scale=0.3)[0].numpy()
    lse = torch.logsumexp(torch.from_numpy(np.where(mask, 0.3 * q @ k.T, -np.inf)), -1).numpy()
    for p in range(23):
        out, z = C.prefill_row(q[p], k, v, p, 0.3, window, sinks)
        assert np.allclose(out, ref[p], rtol=1e-12, atol=1e-13)
        assert np.isclose(z, lse[p], rtol=1e-12)


def test_no_window_is_the_causal_prefill():
    g = rng(2)
    q, k, v = (g.normal(size=(17, 8)) for _ in range(3))
    ref, lse = A.causal_attention(q, k, v, 0.25)
    for p in range(17):
        out, z = C.prefill_row(q[p], k, v, p, 0.25, 0, 0)
        assert np.allclose(out, ref[p], rtol=1e-12) and np.isclose(z, lse[p], rtol=1e-12)


def test_grouped_heads_read_their_key_head():
    g = rng(3)
    q, k, v = g.normal(size=(2, 6, 8)), g.normal(size=(2, 2, 9, 8)), g.normal(size=(2, 2, 9, 8))
    out, lse, weight = C.decode(q, k, v, [9, 4], 0.4)
    for b, n in ((0, 9), (1, 4)):
        for h in range(6):
            ref = torch.softmax(torch.from_numpy(0.4 * k[b, h // 3, :n] @ q[b, h]), 0).numpy()
            assert np.allclose(out[b, h], ref @ v[b, h // 3, :n], rtol=1e-12)
    # every head's weights sum to one: three heads to a key head
    assert np.allclose(weight.sum(-1), 3.0, rtol=1e-12)
    assert np.all(weight[1, :, 4:] == 0)


def test_prefix_is_the_same_as_keys_in_front():
    g = rng(4)
    q, k, v = g.normal(size=(3, 4, 8)), g.normal(size=(3, 2, 5, 8)), g.normal(size=(3, 2, 5, 8))
    kp, vp = g.normal(size=(2, 7, 8)), g.normal(size=(2, 7, 8))
    out, lse, weight = C.decode(q, k, v, [5, 0, 2], 0.5, kp=kp, vp=vp)
    whole_k = np.concatenate([np.broadcast_to(kp, (3, 2, 7, 8)), k], 2)
    whole_v = np.concatenate([np.broadcast_to(vp, (3, 2, 7, 8)), v], 2)
    ref, rl, rw = C.decode(q, whole_k, whole_v, [12, 7, 9], 0.5)
    assert np.allclose(out, ref, rtol=1e-12) and np.allclose(lse, rl, rtol=1e-12)
    assert np.allclose(weight, rw[:, :, 7:], rtol=1e-12)


def test_empty_sequence():
    out, lse, weight = C.decode(np.ones((1, 1, 4)), np.ones((1, 1, 3, 4)), np.ones((1, 1, 3, 4)), [0], 1.0)
    assert np.all(out == 0) and np.all(np.isneginf(lse)) and np.all(weight == 0)


def test_equal_scores_weigh_the_same():
    out, lse, weight = C.decode(np.zeros((1, 1, 4)), np.ones((1, 1, 5, 4)), np.arange(20.0).reshape(1, 1, 5, 4),
                                [5], 1.0)
    assert np.allclose(weight, 0.2) and np.allclose(lse, np.log(5)) and np.allclose(out, [[8, 9, 10, 11]])


def test_kept_rows_by_brute_force():
    """The best sum of weights among all choices, and among those the lexicographically first."""
    for seed in range(30):
        g = rng(seed)
        n, sinks, recent = 9, int(g.integers(0, 3)), int(g.integers(0, 3))
        keep = int(g.integers(max(1, sinks + recent), 9))
        w = np.floor(g.random(n) * 4)                       # ties
        must = set(range(sinks)) | set(range(n - recent, n))
        best = max((sum(w[list(c)]), [-i for i in c]) for c in itertools.combinations(range(n), keep)
                   if must <= set(c))
        assert np.array_equal(C.kept_rows(w, n, keep, sinks, recent), [-i for i in best[1]])


def test_kept_rows_of_short_sequences_and_nan():
    assert np.array_equal(C.kept_rows(np.ones(5), 3, 4, 1, 1), [0, 1, 2])
    w = np.array([1.0, np.nan, -np.inf, 0.0, np.nan])
    assert np.array_equal(C.kept_rows(w, 5, 3, 0, 0), [0, 2, 3])    # NaN below every number
    assert np.array_equal(C.kept_rows(w, 5, 4, 0, 0), [0, 1, 2, 3])


def test_score_error_covers_fp32_sums():
    g = rng(5)
    q = g.normal(size=(4, 128)).astype(np.float32)
    k = g.normal(size=(50, 128)).astype(np.float32)
    exact = q.astype(np.float64) @ k.astype(np.float64).T * 0.1
    run = np.zeros((4, 50), np.float32)
    for d in range(128):                                    # one addition at a time
        run = run + q[:, d:d + 1] * k[:, d]
    assert np.abs(run * np.float32(0.1) - exact).max() <= C.score_error(q.astype(np.float64), k.astype(np.float64), 0.1)
