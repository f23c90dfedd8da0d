"""Inputs and derived tolerances for the tests of the calls over a serving cache."""

import numpy as np
import torch

from oracle import cache as C
from helpers import f64

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def normal(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype)


def out_bound(ref, delta, vmax, out_dtype, p_step):
    """|out - ref| allowed.  A score error of at most ``delta`` moves every weight by at most
    exp(2 delta) - 1 of itself (numerator and normaliser); exp2 and the sums add 2^-19; a weight
    rounded to ``p_step`` moves it by that share; the weights sum to 1, so the output moves by at
    most that share of the largest |v|.  Rounding the output adds half a step of the result."""
    moved = (np.expm1(2 * delta) + 2.0 ** -19 + p_step) * vmax
    return HALF_STEP[out_dtype] * (np.abs(ref) + moved) + moved + 2.0 ** -25


def assert_within(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    bound = np.broadcast_to(bound, ref.shape)
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - ref) <= bound))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first at {i}: "
                             f"got {got[i]!r}, ref {ref[i]!r}, bound {bound[i]!r}")


def check_decode(out, lse, q, k, v, lens, scale, window=0, sinks=0, kp=None, vp=None,
                 p_step=2.0 ** -16):
    """out and lse of a decode call against the definition; returns the oracle's weights and the
    score error bound.  NaN rows that the call must not read are zeroed for the oracle."""
    qd, kd, vd = f64(q), np.nan_to_num(f64(k)), np.nan_to_num(f64(v))
    kpd, vpd = (None, None) if kp is None else (f64(kp), f64(vp))
    ref, rl, w = C.decode(qd, kd, vd, lens, scale, window, sinks, kpd, vpd)
    delta = max(C.score_error(qd[b], kd[b].reshape(-1, qd.shape[-1]), scale) for b in range(qd.shape[0]))
    vmax = float(np.abs(vd).max())
    if kp is not None:
        delta = max(delta, C.score_error(qd.reshape(-1, qd.shape[-1]), kpd.reshape(-1, qd.shape[-1]), scale))
        vmax = max(vmax, float(np.abs(vpd).max()))
    assert_within(f64(out), ref, out_bound(ref, delta, vmax, out.dtype, p_step), "out")
    live = ~np.isneginf(rl)
    assert np.array_equal(np.isneginf(f64(lse)), ~live), "rows without keys"
    # the logarithm's argument is off by the weights' share, its value rounded to fp32
    assert_within(f64(lse)[live], rl[live], delta + 2.0 ** -19 + 2.0 ** -22 * np.abs(rl[live]), "lse")
    return w, delta
