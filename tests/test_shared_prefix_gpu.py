"""Decode of a batch that shares a prefix (rf_attn_decode_shared) against the
definition in float64: softmax over the prefix and each sequence's own keys.

The prefix's weights are rounded to 16 bits for the tensor cores (half a step
each), which the output bound counts; rows behind a sequence's end hold NaN.
"""

import pytest
import torch

from cache_helpers import DT, HALF_STEP, check_decode, normal

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def make(seed, B, H, Hkv, prefix, cap, lens, dtype):
    q = normal(seed, B, H, 128, dtype=dtype)
    kp, vp = normal(seed + 1, Hkv, prefix, 128, dtype=dtype), normal(seed + 2, Hkv, prefix, 128, dtype=dtype)
    k, v = normal(seed + 3, B, Hkv, cap, 128, dtype=dtype), normal(seed + 4, B, Hkv, cap, 128, dtype=dtype)
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = float("nan"), float("nan")
    return [t.cuda() for t in (q, kp, vp, k, v)] + [torch.tensor(lens, dtype=torch.int32, device="cuda")]


def check(rf, args, lens, work=None, **kw):
    q, kp, vp, k, v, n = args
    out, lse = rf.attn_decode_shared(q, kp, vp, k, v, n, scale=SCALE, work=work, **kw)
    torch.cuda.synchronize()
    assert rf.rf_device_error() == 0
    check_decode(out, lse, q, k, v, lens, SCALE, kp=kp, vp=vp, p_step=HALF_STEP[q.dtype])
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("prefix", [1, 2, 127, 128, 255, 256, 257, 1000])
def test_prefix_lengths(rf, prefix, dtype):
    lens = [0, 1, 40, 33]
    check(rf, make(prefix, 4, 8, 2, prefix, 40, lens, DT[dtype]), lens)


# group sizes that do and do not divide a tile of 128 rows; batches that end inside a tile
@pytest.mark.parametrize("B,H,Hkv", [(1, 1, 1), (1, 16, 1), (5, 4, 4), (43, 6, 2), (37, 7, 1), (130, 2, 1),
                                     (3, 128, 1), (9, 40, 1), (257, 1, 1), (70, 8, 2)])
def test_batches_and_head_groups(rf, B, H, Hkv):
    lens = [(7 * b) % 21 for b in range(B)]
    check(rf, make(B, B, H, Hkv, 700, 20, lens, torch.bfloat16), lens)


@pytest.mark.parametrize("Sp,S", [(2, 1), (3, 5), (40, 2)])
def test_segment_counts(rf, Sp, S):
    lens = [300, 0, 77]
    args = make(Sp, 3, 8, 2, 5000, 300, lens, torch.bfloat16)
    q, kp, vp, k, v, n = args
    # whatever the scratch held before must not show
    f32 = dict(device="cuda", dtype=torch.float32)
    m, l = (torch.full((24, Sp + S), float("nan"), **f32) for _ in range(2))
    acc = torch.full((24, Sp + S, 128), float("nan"), **f32)
    counters = torch.zeros(6, device="cuda", dtype=torch.int32)
    for _ in range(2):
        out, lse = torch.empty_like(q), torch.empty(3, 8, **f32)
        rf.rf_attn_decode_shared(q, kp, vp, k, v, n, Sp, S, SCALE, m, l, acc, counters, out, lse)
        check_decode(out, lse, q, k, v, lens, SCALE, kp=kp, vp=vp, p_step=2.0 ** -8)
    assert torch.all(counters == 0)


def test_long_prefix_and_fp32_output(rf):
    lens = [100] * 40
    check(rf, make(3, 40, 32, 8, 9001, 100, lens, torch.bfloat16), lens, out_dtype=torch.float32)


def test_empty_own_caches(rf):
    lens = [0, 0]
    check(rf, make(4, 2, 8, 2, 300, 16, lens, torch.float16), lens)


def test_equals_one_long_cache(rf):
    # the prefix copied in front of every sequence's own keys gives the same attention
    lens = [50, 9]
    q, kp, vp, k, v, n = make(5, 2, 8, 2, 600, 50, lens, torch.bfloat16)
    out, lse = rf.attn_decode_shared(q, kp, vp, k, v, n, scale=SCALE)
    kk = torch.cat([kp.expand(2, -1, -1, -1), k], 2).contiguous()
    vv = torch.cat([vp.expand(2, -1, -1, -1), v], 2).contiguous()
    ref, rl = rf.attn_decode_window(q, kk, vv, n + 600, scale=SCALE)
    # the prefix's weights are rounded to bf16 (2^-8 each) and both outputs once
    assert torch.all((out.double() - ref.double()).abs() <= 2 ** -7 * ref.double().abs() + 2 ** -7 * vp.abs().max())
    assert torch.all((lse - rl).abs() <= 1e-4)


def test_the_same_bits_every_time(rf):
    lens = [64 - b for b in range(30)]
    args = make(6, 30, 32, 8, 3000, 64, lens, torch.bfloat16)
    first = check(rf, args, lens)
    for _ in range(4):
        again = check(rf, args, lens)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_captured_and_replayed(rf):
    lens = [30, 12, 0]
    args = make(7, 3, 8, 2, 500, 30, lens, torch.bfloat16)
    q, kp, vp, k, v, n = args
    work = rf.decode_workspace(3, 8, 2, 30, prefix=500)
    check(rf, args, lens, work)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = rf.attn_decode_shared(q, kp, vp, k, v, n, scale=SCALE, work=work)
    for seed, lens in ((8, [1, 30, 5]), (9, [0, 0, 17])):
        for dst, src in zip(args, make(seed, 3, 8, 2, 500, 30, lens, torch.bfloat16)):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        check_decode(out, lse, q, k, v, lens, SCALE, kp=kp, vp=vp, p_step=2.0 ** -8)


# Above, most calls are small enough to read the prefix once per sequence.  Below, more row
# groups than that allows: the prefix kernel, then the merge.
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("prefix", [1, 2, 127, 128, 129, 255, 256, 257, 513, 1000])
def test_many_sequences_prefix_lengths(rf, prefix, dtype):
    lens = [(5 * b) % 9 for b in range(40)]
    check(rf, make(prefix, 40, 16, 8, prefix, 8, lens, DT[dtype]), lens)


@pytest.mark.parametrize("B,H,Hkv", [(310, 1, 1), (160, 16, 2), (110, 21, 3), (40, 128, 8), (26, 160, 4),
                                     (20, 256, 2), (313, 3, 1)])
def test_many_sequences_head_groups(rf, B, H, Hkv):
    lens = [(7 * b) % 21 for b in range(B)]
    check(rf, make(B, B, H, Hkv, 300, 20, lens, torch.bfloat16), lens)


@pytest.mark.parametrize("Sp,S", [(2, 1), (3, 2), (40, 1)])
def test_many_sequences_segment_counts(rf, Sp, S):
    lens = [(37 * b) % 90 for b in range(40)]
    args = make(Sp, 40, 16, 8, 2000, 90, lens, torch.bfloat16)
    q, kp, vp, k, v, n = args
    f32 = dict(device="cuda", dtype=torch.float32)
    m, l = (torch.full((640, Sp + S), float("nan"), **f32) for _ in range(2))
    acc = torch.full((640, Sp + S, 128), float("nan"), **f32)
    counters = torch.zeros(320, device="cuda", dtype=torch.int32)
    for _ in range(2):
        out, lse = torch.empty_like(q), torch.empty(40, 16, **f32)
        rf.rf_attn_decode_shared(q, kp, vp, k, v, n, Sp, S, SCALE, m, l, acc, counters, out, lse)
        check_decode(out, lse, q, k, v, lens, SCALE, kp=kp, vp=vp, p_step=2.0 ** -8)
    assert torch.all(counters == 0)


@pytest.mark.parametrize("B", [6, 40])
def test_nan_in_the_prefix_and_behind_it(rf, B):
    # a NaN value row of the prefix reaches its key head's rows alone, one behind a sequence none
    lens = [3] * B
    q, kp, vp, k, v, n = make(10, B, 16, 8, 100, 8, lens, torch.bfloat16)
    vp[2, 99] = float("nan")
    out, lse = rf.attn_decode_shared(q, kp, vp, k, v, n, scale=SCALE)
    bad = out.isnan().all(-1)
    assert torch.equal(bad, torch.arange(16, device="cuda").expand(B, 16) // 2 == 2)
    assert torch.equal(out.isnan().any(-1), bad) and lse.isfinite().all()


def test_many_sequences_captured_and_replayed(rf):
    lens = [b % 30 for b in range(40)]
    args = make(11, 40, 16, 8, 500, 30, lens, torch.bfloat16)
    q, kp, vp, k, v, n = args
    work = rf.decode_workspace(40, 16, 8, 30, prefix=500)
    check(rf, args, lens, work)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = rf.attn_decode_shared(q, kp, vp, k, v, n, scale=SCALE, work=work)
    for seed, lens in ((12, [30] * 40), (13, [0] * 40)):
        for dst, src in zip(args, make(seed, 40, 16, 8, 500, 30, lens, torch.bfloat16)):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        check_decode(out, lse, q, k, v, lens, SCALE, kp=kp, vp=vp, p_step=2.0 ** -8)
