"""Small softmax weights in fp16: one key that outweighs all others, with a value of zero, so that
the output is made of weights far below the largest.

Key 0 (or the last) has the score ``gap`` (in log2 units), the others 0, so a weight is 2^-gap of the
largest.  Scores have one nonzero product, which is exact, and lose 2^-23 of gap to the scale: at most
2^-17 of a weight for gap <= 64.
"""

import math

import numpy as np
import pytest
import torch

from helpers import f64
from oracle import cache as C

pytestmark = pytest.mark.gpu

F16 = torch.float16


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def scale_for(gap):
    return float(np.float32(gap * math.log(2)))


def peaked(n, at):
    """k, v [n, 128]: a score of 1 x scale at key ``at`` alone for a query of 1, 0, 0 ..."""
    k, v = torch.zeros(n, 128, dtype=F16), torch.zeros(n, 128, dtype=F16)
    k[at, 0] = 1
    v += torch.linspace(0.5, 2, 128).to(F16)
    v[at] = 0
    return k.cuda(), v.cuda()


def query(*shape):
    q = torch.zeros(*shape, 128, dtype=F16)
    q[..., 0] = 1
    return q.cuda()


def one_term_bound(ref, n):
    """Weights as one fp16 number: half a step of it, or of the smallest one, 2^-25, in units of 2^-7
    of the largest weight.  The sum of n such products in fp32, 16 at a time, truncated at worst."""
    return np.abs(ref) * (2.0 ** -11 + n / 16 * 2.0 ** -23 + 2.0 ** -17) + n * 2.0 ** -32 * 2


@pytest.mark.parametrize("gap", [20.3, 26.0, 28.0])
def test_prefix(rf, gap):
    n, B, H = 32769, 2 * torch.cuda.get_device_properties(0).multi_processor_count + 1, 1
    kp, vp = peaked(n, 0)
    q, k = query(B, H), torch.zeros(B, H, 1, 128, dtype=F16, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    f32 = dict(device="cuda", dtype=torch.float32)
    out, lse = torch.empty(B, H, 128, **f32), torch.empty(B, H, **f32)
    # two slots: one cluster goes through the whole prefix, the largest weight first
    rf.rf_attn_decode_shared(q, kp[None], vp[None], k, k, lens, 2, 1, scale_for(gap), torch.empty(B, 3, **f32),
                             torch.empty(B, 3, **f32), torch.empty(B, 3, 128, **f32),
                             torch.zeros(B, dtype=torch.int32, device="cuda"), out, lse)
    ref, rl, _ = C.attend(f64(q[0, 0]), f64(kp), f64(vp), scale_for(gap))
    assert np.all(np.abs(f64(out) - ref) <= one_term_bound(ref, n))
    assert np.all(np.abs(f64(lse) - rl) <= 2.0 ** -17 * abs(rl))


@pytest.mark.parametrize("gap", [20.3, 26.0, 28.0])
def test_prefill(rf, gap):
    # blocks are visited from the last on, which holds the largest weight of the last row
    n, N = 32769, 4
    k, v = peaked(n, n - 1)
    out, lse = rf.attn_prefill_window(query(1, 1, N), k[None, None], v[None, None], scale=scale_for(gap))
    ref, rl, _ = C.attend(f64(query(1)[0]), f64(k), f64(v), scale_for(gap))
    bound = one_term_bound(ref, n) + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
    assert np.all(np.abs(f64(out[0, 0, -1]) - ref) <= bound)
    assert abs(f64(lse[0, 0, -1]) - rl) <= 2.0 ** -17 * abs(rl)


@pytest.mark.parametrize("gap", [13.3, 18.3, 24.3])
@pytest.mark.parametrize("S", [1, 4])
def test_decode(rf, gap, S):
    # two terms: the second is exact to 2^-25 in units of 2^-15 of the largest weight
    n = 512
    k, v = peaked(n, 0)
    work = rf.decode_workspace(1, 1, 1, n, S=S)
    out, lse = rf.attn_decode_window(query(1, 1), k[None, None], v[None, None], scale=scale_for(gap), work=work,
                                     out_dtype=torch.float32)
    ref, rl, _ = C.attend(f64(query(1)[0]), f64(k), f64(v), scale_for(gap))
    assert np.all(np.abs(f64(out[0, 0]) - ref) <= np.abs(ref) * 2.0 ** -16 + n * 2.0 ** -40 * 2)
    assert abs(f64(lse[0, 0]) - rl) <= 2.0 ** -17 * abs(rl)
