"""Eviction by accumulated weight (rf_cache_evict) against the definition: every
output is a copy or an index, so all comparisons are exact."""

import numpy as np
import pytest
import torch

from cache_helpers import DT, normal
from oracle import cache as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def check(rf, k, v, weight, lens, keep, sinks, recent, cap_out=None, full=False):
    B, Hkv, cap, D = k.shape
    rows = cap_out or keep
    mark = lambda t, *s: torch.full(s, 7.0, dtype=t.dtype, device="cuda")       # noqa: E731
    k_out, w_out = mark(k, B, Hkv, rows, D), mark(weight, B, Hkv, rows)
    v_out = None if v is None else mark(v, B, Hkv, rows, D)
    n = None if full else torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = rf.cache_evict(k, v, weight, n, keep, sinks, recent, out=(k_out, v_out, w_out))
    assert got[0] is k_out and got[1] is v_out and got[2] is w_out
    new, kept = got[3].cpu().numpy(), got[4].cpu().numpy()
    wh = weight.cpu().numpy()
    assert np.array_equal(new, np.minimum(lens, keep))
    for b in range(B):
        for h in range(Hkv):
            ref = C.kept_rows(wh[b, h], int(lens[b]), keep, sinks, recent)
            c = len(ref)
            assert np.array_equal(kept[b, h, :c], ref), (b, h)
            assert np.all(kept[b, h, c:] == -1)
            for src, dst in ((k, k_out), (v, v_out), (weight, w_out)):
                if src is not None:
                    assert np.array_equal(bits(dst[b, h, :c]), bits(src[b, h, torch.from_numpy(ref).cuda()]))
                    assert torch.all(dst[b, h, c:] == 7.0)           # behind the sequence: untouched


def make(seed, B, Hkv, cap, D=128, dtype=torch.bfloat16, levels=None):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(B, Hkv, cap, generator=g) ** 6
    if levels:                                       # few distinct weights: ties everywhere
        w = torch.floor(w * levels) / levels
    k, v = normal(seed + 1, B, Hkv, cap, D, dtype=dtype), normal(seed + 2, B, Hkv, cap, D, dtype=dtype)
    return k.cuda(), v.cuda(), w.cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("cap,keep,sinks,recent", [(1, 1, 0, 0), (2, 1, 0, 0), (2, 1, 1, 0), (2, 1, 0, 1),
                                                   (33, 32, 4, 8), (100, 37, 0, 0), (100, 37, 4, 33),
                                                   (1025, 1000, 1, 999), (3001, 500, 4, 100)])
def test_sizes(rf, cap, keep, sinks, recent, dtype):
    k, v, w = make(cap, 2, 3, cap, dtype=DT[dtype])
    check(rf, k, v, w, [cap, cap], keep, sinks, recent)


@pytest.mark.parametrize("levels", [1, 3, 50])
def test_ties_go_to_the_lower_index(rf, levels):
    k, v, w = make(levels, 3, 2, 999, levels=levels)
    check(rf, k, v, w, [999, 500, 301], 300, 4, 64)


@pytest.mark.parametrize("levels", [None, 7])
@pytest.mark.parametrize("close", [1, 3, 4, 127, 128, 129, 131])
def test_weights_close_to_the_threshold(rf, close, levels):
    # `close` weights share their leading bits with the threshold; 100 are far above
    k, v, w = make(10, 4, 1, 500)
    g = torch.Generator().manual_seed(close)
    near = 1 + torch.rand(4, close, generator=g) * 0.24
    if levels is not None:
        near = 1 + (near * 100).floor() % levels / 32
    w[:] = 0.01
    for b in range(4):
        at = torch.randperm(500, generator=g)
        w[b, 0, at[:close].cuda()] = near[b].cuda()
        w[b, 0, at[close:close + 100].cuda()] = 8.0
    for need in sorted({1, (close + 1) // 2, close}):
        check(rf, k, v, w, [500] * 4, 100 + need, 0, 0)


def test_ragged_and_short_sequences(rf):
    lens = [0, 1, 99, 100, 101, 640]
    k, v, w = make(4, len(lens), 2, 640)
    check(rf, k, v, w, lens, 100, 4, 30, cap_out=170)


def test_no_lengths(rf):
    k, v, w = make(5, 2, 2, 300)
    check(rf, k, v, w, [300, 300], 77, 2, 9, full=True)


def test_special_weights(rf):
    # infinities, NaN (below every number), both zeros, subnormals and negative values
    k, v, w = make(6, 1, 4, 400)
    w[0, 0, ::3] = float("nan")
    w[0, 1, ::2] = float("inf")
    w[0, 1, 1::4] = float("-inf")
    w[0, 2, :] = torch.tensor([0.0, -0.0], device="cuda").repeat(200)
    w[0, 2, 50:90] = 1e-42
    w[0, 3, :] = -w[0, 3]
    check(rf, k, v, w, [400], 150, 0, 0)
    w[0, 0, :] = float("nan")
    check(rf, k, v, w, [400], 150, 3, 7)


def test_longer_than_shared_memory(rf):
    # 60000 weights do not fit; rows of 16 bytes keep the case small
    k, v, w = make(7, 2, 1, 60000, D=8, levels=1000)
    check(rf, k, v, w, [60000, 50001], 20000, 4, 1000)


def test_one_tensor_of_fp32_rows(rf):
    k, _, w = make(8, 2, 1, 500, D=64, dtype=torch.float32)
    check(rf, k, None, w, [500, 30], 100, 4, 10)


def test_rows_behind_the_end_may_weigh_anything(rf):
    k, v, w = make(9, 1, 1, 500)
    w[0, 0, 300:] = float("inf")
    check(rf, k, v, w, [300], 100, 4, 10)


def test_decode_total_evict_decode(rf):
    """As a serving loop uses them: decode steps total the weights, the cache is evicted, and the
    next token attends to what was kept, at the kept rows' own values."""
    B, H, Hkv, cap, keep = 2, 8, 2, 400, 150
    lens = [400, 90]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k, v = normal(60, B, Hkv, cap, 128).cuda(), normal(61, B, Hkv, cap, 128).cuda()
    total = torch.zeros(B, Hkv, cap, device="cuda")
    work = rf.decode_workspace(B, H, Hkv, cap, weights=True)
    for step in range(3):
        q = normal(70 + step, B, H, 128).cuda()
        rf.attn_decode_weights(q, k, v, n, weight=total, weight_out=total, work=work)
    # three tokens, each head's weights sum to one: 3 G in all (fp32 sums)
    assert np.allclose(total.double().sum(-1).cpu().numpy(), 3 * H / Hkv, rtol=1e-5)
    k2, v2, w2, n2, kept = rf.cache_evict(k, v, total, n, keep, sinks=4, recent=32)
    q = normal(80, B, H, 128).cuda()
    out, lse = rf.attn_decode_window(q, k2, v2, n2)
    from cache_helpers import check_decode
    kz, vz = torch.zeros_like(k2), torch.zeros_like(v2)
    for b in range(B):
        for h in range(Hkv):
            rows = kept[b, h][kept[b, h] >= 0].long()
            kz[b, h, :len(rows)], vz[b, h, :len(rows)] = k[b, h, rows], v[b, h, rows]
    check_decode(out, lse, q, kz, vz, n2.cpu().numpy(), 128 ** -0.5)


def test_captured_and_replayed(rf):
    k, v, w = make(10, 2, 2, 300)
    n = torch.tensor([300, 300], dtype=torch.int32, device="cuda")
    out = (torch.zeros(2, 2, 100, 128, dtype=torch.bfloat16, device="cuda"),
           torch.zeros(2, 2, 100, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 2, 100, device="cuda"))
    rf.cache_evict(k, v, w, n, 100, 4, 10, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        *_, n_out, kept = rf.cache_evict(k, v, w, n, 100, 4, 10, out=out)
    w.copy_(torch.rand(2, 2, 300, generator=torch.Generator().manual_seed(3)))
    n.copy_(torch.tensor([250, 60], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert n_out.tolist() == [100, 60]
    for b, m in enumerate((250, 60)):
        for h in range(2):
            ref = C.kept_rows(w[b, h].cpu().numpy(), m, 100, 4, 10)
            assert np.array_equal(kept[b, h, :len(ref)].cpu().numpy(), ref)
            assert torch.equal(out[0][b, h, :len(ref)], k[b, h, torch.from_numpy(ref).cuda()])


@pytest.mark.parametrize("D", [8, 24, 576, 1160, 4104, 32768])
def test_row_sizes(rf, D):
    # rows of 16 bytes up to 64 KiB, whole and odd parts of a block's 256 columns
    cap, keep = (300, 131) if D < 4000 else (40, 17)
    k, v, w = make(D, 2, 1, cap, D=D)
    check(rf, k, v, w, [cap, cap // 2], keep, 1, 5)
