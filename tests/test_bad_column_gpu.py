"""The windowed prefill's second look at rows that hold a NaN costs little where the row rightly
does: a value row that many see, with a NaN in one column or a NaN key."""

import pytest
import torch

from cache_helpers import normal

pytestmark = pytest.mark.gpu

N, H, HKV = 2048, 8, 2


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def ms(call):
    call()
    best = []
    for _ in range(3):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        b.synchronize()
        best.append(a.elapsed_time(b))
    return min(best)


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("where", ["first key", "sink", "middle", "each block", "key", "every key"])
def test_time_and_values(rf, where, window, record_property):
    q = normal(1, 1, H, N, 128).cuda()
    k, v = (normal(s, 1, HKV, N, 128).cuda() for s in (2, 3))

    def call():
        return rf.attn_prefill_window(q, k, v, window=window, sinks=4)
    out, lse = call()
    clean = ms(call)
    nan = float("nan")
    rows = {"first key": [0], "sink": [3], "middle": [N // 2], "each block": range(100, N, 256),
            "key": [N // 2], "every key": range(N)}[where]
    for j in rows:
        if where == "key":
            k[0, 0, j, 7] = nan
        else:
            v[0, 0, j, 3] = nan
    bad, lse2 = call()
    torch.cuda.synchronize()
    i = torch.arange(N, device="cuda")
    seen = torch.zeros(N, dtype=torch.bool, device="cuda")
    for j in rows:
        seen |= (i >= j) & ((i - j < window) if window and j >= 4 else True)
    want, want_lse = out.clone(), lse.clone()
    if where == "key":
        want[0, :4, seen] = nan
        want_lse[0, :4, seen] = nan
    else:
        want[0, :4, seen, 3] = nan
    spent = ms(call)
    record_property("clean_ms", clean)
    record_property("bad_ms", spent)
    print(f"{where}, window {window}: {clean:.3f} -> {spent:.3f} ms")
    assert torch.equal(bad.isnan(), want.isnan()) and torch.equal(lse2.nan_to_num(), want_lse.nan_to_num())
    # what was right is kept, and a row that is computed again agrees to its rounding
    assert torch.all((bad.nan_to_num().double() - want.nan_to_num().double()).abs() <= 0.02)
    # Nearly every row is NaN by right.  Some before a bad key share a block with it (an item has 64
    # positions, and where its window begins a block may end up to 192 keys behind them) and are
    # computed again: a warp's 32 rows, one behind the other, over the window, or over the keys before
    # the first bad one, at most 0.4 us for each.
    limit = 40 * clean + 32 * {"middle": window, "each block": 128}.get(where, 0) * 0.4e-3
    assert spent <= limit
