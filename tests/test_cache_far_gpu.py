"""Calls over a serving cache whose offsets pass 32 bits, and two threads that call at once."""

import threading

import pytest
import torch

from cache_helpers import normal

pytestmark = pytest.mark.gpu

HEADS, L = 34, 1 << 19                   # 2^31 elements lie before the last key head's rows


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


@pytest.fixture(scope="module")
def far():
    """k, v [1, HEADS, L, 128]: zeros but for the first 8 and last 600 rows of the last head."""
    k, v = (torch.zeros(1, HEADS, L, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t, s in ((k, 1), (v, 3)):
        t[0, -1, :8], t[0, -1, -600:] = normal(s, 8, 128).cuda(), normal(s + 1, 600, 128).cuda()
    yield k, v
    del k, v
    torch.cuda.empty_cache()


def near(k, v):
    """What the last head's rows see, as a cache of its own."""
    return (torch.cat([t[:, -1:, :8], t[:, -1:, -600:]], 2).contiguous() for t in (k, v))


# the same arithmetic on the same keys: the same bits, where the blocks are the same
@pytest.mark.parametrize("N", [3, 300])
def test_prefill(rf, far, N):
    k, v = far
    q = normal(5, 1, HEADS, N, 128).cuda()
    out, lse = rf.attn_prefill_window(q, k, v, window=250, sinks=8)
    ref, rl = rf.attn_prefill_window(q[:, -1:].contiguous(), *near(k, v), window=250, sinks=8)
    # each within half a step of the weights and of the output of the definition
    bound = 2.0 ** -7 * ref.double().abs() + 2.0 ** -8 * v.abs().max().double()
    assert torch.all((out[:, -1:].double() - ref.double()).abs() <= bound)
    assert torch.all((lse[:, -1:] - rl).abs() <= 1e-4) and torch.all(out[:, :-1] == 0)
    kept = v[0, -1, -3, 5].clone()
    v[0, -1, -3, 5] = float("nan")       # seen by the last three rows, beside others of their block
    bad, _ = rf.attn_prefill_window(q, k, v, window=250, sinks=8)
    v[0, -1, -3, 5] = kept
    assert bad.isnan().nonzero().tolist() == [[0, HEADS - 1, i, 5] for i in range(N - 3, N)]


def test_shared_prefix(rf, far):
    kp, vp = far[0][0], far[1][0]
    B, cap = 10, 20
    q = normal(6, B, HEADS, 128).cuda()
    k, v = normal(7, B, HEADS, cap, 128).cuda(), normal(8, B, HEADS, cap, 128).cuda()
    out, lse = rf.attn_decode_shared(q, kp, vp, k, v)
    kk = torch.cat([kp[-1:].expand(B, 1, L, 128), k[:, -1:]], 2)
    vv = torch.cat([vp[-1:].expand(B, 1, L, 128), v[:, -1:]], 2)
    ref, rl = rf.attn_decode_window(q[:, -1:].contiguous(), kk, vv)
    # the prefix's weights are rounded to bf16 and both outputs once
    p = torch.exp(torch.einsum("bd,bkd->bk", q[:, -1].double(), kk[:, 0].double()) * 128 ** -0.5 - rl.double())
    moved = 2.0 ** -8 * torch.einsum("bk,bkd->bd", p, vv[:, 0].double().abs())
    assert torch.all((out[:, -1].double() - ref[:, 0].double()).abs() <= 2.0 ** -7 * ref[:, 0].double().abs() + moved)
    assert torch.all((lse[:, -1:] - rl).abs() <= 1e-4)


def test_eviction(rf, far):
    k, v = far
    w = torch.rand(1, HEADS, L, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    k_out, v_out, w_out, lens, kept = rf.cache_evict(k, v, w, None, 1000, sinks=8, recent=600)
    at = kept[0, -1].long()
    middle = torch.sort(w[0, -1, 8:L - 600], descending=True, stable=True).indices[:392].sort().values + 8
    assert torch.equal(at[8:400], middle) and lens.item() == 1000
    for got, src in ((k_out, k), (v_out, v), (w_out, w)):
        assert torch.equal(got[0, -1], src[0, -1, at])


def test_two_threads(rf):
    def make(seed):
        B, H, Hkv, cap = 24, 32, 8, 2000
        d = {n: normal(seed + i, *s).cuda() for i, (n, s) in enumerate(dict(
            q=(B, H, 128), k=(B, Hkv, cap, 128), v=(B, Hkv, cap, 128), kp=(Hkv, 900, 128), vp=(Hkv, 900, 128),
            qs=(1, H, 900, 128), ks=(1, Hkv, 900, 128), vs=(1, Hkv, 900, 128)).items())}
        d["lens"] = torch.tensor([cap - 71 * b for b in range(B)], dtype=torch.int32, device="cuda")
        d["work"] = rf.decode_workspace(B, H, Hkv, cap, prefix=900, weights=True)
        return d

    def steps(d):
        a, _ = rf.attn_decode_window(d["q"], d["k"], d["v"], d["lens"], window=700, sinks=4, work=d["work"])
        b, _ = rf.attn_decode_shared(a, d["kp"], d["vp"], d["k"], d["v"], d["lens"], work=d["work"])
        c, _, t = rf.attn_decode_weights(b, d["k"], d["v"], d["lens"], work=d["work"])
        e = rf.cache_evict(d["k"], d["v"], t, d["lens"], 500, sinks=4, recent=50)
        f, _ = rf.attn_prefill_window(d["qs"], d["ks"], d["vs"], window=300, sinks=4)
        return [a, b, c, t, *e, f]

    data = [make(20), make(40)]
    want = [[x.clone() for x in steps(d)] for d in data]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(5):
                    for _ in range(10):
                        got = steps(data[i])
                    stream.synchronize()
                    wrong.extend((i, j) for j, (x, y) in enumerate(zip(got, want[i])) if not torch.equal(x, y))
        except Exception as e:           # noqa: BLE001  (told by the assertion below)
            wrong.append(repr(e))
    threads = [threading.Thread(target=run, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and rf.rf_device_error() == 0
