"""The calls over a serving cache give the same outputs, bit for bit, and the same refusals with
the extension of csrc/calls.cpp as marshalled in Python."""

import pytest
import torch

from cache_helpers import DT, normal

pytestmark = pytest.mark.gpu

B, H, HKV, CAP, D, PREFIX = 3, 8, 2, 200, 128, 300


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def inputs(dt):
    t = dict(q=normal(1, B, H, D, dtype=dt), k=normal(2, B, HKV, CAP, D, dtype=dt),
             v=normal(3, B, HKV, CAP, D, dtype=dt), kp=normal(4, HKV, PREFIX, D, dtype=dt),
             vp=normal(5, HKV, PREFIX, D, dtype=dt), lens=torch.tensor([1, 200, 77], dtype=torch.int32),
             weight=normal(6, B, HKV, CAP, dtype=torch.float32).abs(),
             qs=normal(7, B, H, 70, D, dtype=dt))
    return {n: x.cuda() for n, x in t.items()}


def calls(rf, t):
    """Name -> a call whose keyword arguments replace the named inputs."""
    wide = rf.decode_workspace(B, H, HKV, CAP, window=50, sinks=4)
    shared = rf.decode_workspace(B, H, HKV, CAP, prefix=PREFIX)
    totals = rf.decode_workspace(B, H, HKV, CAP, weights=True)

    def window(**o):
        a = {**t, "window": 50, "sinks": 4, "scale": None, "work": wide, **o}
        return rf.attn_decode_window(a["q"], a["k"], a["v"], a["lens"], a["window"], a["sinks"],
                                     a["scale"], a["work"])

    def prefix(**o):
        a = {**t, "scale": 0.07, "work": shared, **o}
        return rf.attn_decode_shared(a["q"], a["kp"], a["vp"], a["k"], a["v"], a["lens"], a["scale"],
                                     a["work"])

    def weights(**o):
        a = {**t, "scale": 0.07, "work": totals, **o}
        return rf.attn_decode_weights(a["q"], a["k"], a["v"], a["lens"], a["weight"], a["scale"], a["work"])

    def prefill(**o):
        a = {**t, "window": 50, "sinks": 4, "scale": None, **o}
        return rf.attn_prefill_window(a["qs"], a["k"], a["v"], a["window"], a["sinks"], a["scale"])

    def evict(**o):
        a = {**t, "keep": 60, "sinks": 4, "recent": 8, **o}
        out = o.get("out", [torch.zeros_like(t["k"][:, :, :60]), torch.zeros_like(t["k"][:, :, :60]),
                            torch.zeros_like(t["weight"][:, :, :60])])
        return rf.cache_evict(a["k"], a["v"], a["weight"], a["lens"], a["keep"], a["sinks"], a["recent"],
                              out=out)
    return dict(window=window, prefix=prefix, weights=weights, prefill=prefill, evict=evict)


NAMES = ("window", "prefix", "weights", "prefill", "evict")


def counted(rf, monkeypatch):
    """Puts a proxy before the extension; gives the list of its calls' results."""
    seen, real = [], rf._calls

    class Proxy:
        def __getattr__(self, name):
            def f(*args):
                seen.append(getattr(real, name)(*args))
                return seen[-1]
            return f
    monkeypatch.setattr(rf, "_calls", Proxy())
    return seen


def same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and x.device == y.device
        assert x.is_contiguous() and not x.requires_grad
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("name", NAMES)
def test_same_outputs(rf, monkeypatch, name, dtype):
    assert rf._calls is not None, "csrc/calls.cpp was not built"
    call = calls(rf, inputs(DT[dtype]))[name]
    variants = [{}, {"lens": None}] if name != "prefill" else [{}, {"window": 0, "sinks": 0}]
    if name in ("window", "prefill"):
        variants += [{"window": 1 << 40}, {"sinks": 1 << 40, "scale": 0.3}]
    if name == "weights":
        variants.append({"weight": None})
    seen = counted(rf, monkeypatch)
    quick = [call(**o) for o in variants]
    assert len(seen) == len(variants) and all(type(r) is tuple for r in seen)
    monkeypatch.setattr(rf, "_calls", None)
    for o, got in zip(variants, quick):
        same(got, call(**o))


@pytest.mark.parametrize("name", NAMES)
def test_same_refusals(rf, monkeypatch, name):
    t = inputs(torch.bfloat16)
    call = calls(rf, t)[name]
    other = rf.decode_workspace(B + 1, H, HKV, CAP, prefix=PREFIX, weights=True)
    longer = rf.decode_workspace(B, H, HKV, CAP + 1, prefix=PREFIX, weights=True)
    ways = [{"k": t["k"].cpu()}, {"k": t["k"].float()}, {"k": t["k"][:, :, ::2]}, {"v": t["v"][:, :, 1:]}]
    if name != "prefill":
        ways += [{"lens": t["lens"].long()}, {"lens": t["lens"][:2]}]
    if name in ("window", "prefix", "weights"):
        ways += [{"q": t["q"][..., :64]}, {"q": t["q"].transpose(0, 1)}, {"work": other},
                 {"scale": float("nan")}, {"q": t["q"].float(), "k": t["k"].float(), "v": t["v"].float(),
                                           "kp": t["kp"].float(), "vp": t["vp"].float()}]
    if name in ("window", "prefill"):
        ways += [{"window": -1}, {"sinks": -3}]
    if name == "prefill":
        ways += [{"qs": t["qs"][0]}, {"scale": float("inf")}]
    if name == "prefix":
        ways += [{"kp": t["kp"][0]}, {"vp": t["vp"][:, 1:]}]
    if name == "weights":
        ways += [{"weight": t["weight"].half()}, {"work": longer}]
    if name == "evict":
        ways += [{"keep": 0}, {"keep": 5}, {"keep": 61}, {"sinks": -1}, {"recent": -2}, {"v": None},
                 {"weight": t["weight"][..., 1:]}, {"out": [t["k"], t["v"], t["weight"]]},
                 {"out": [t["k"][:, :, :60], t["v"][:, :, :60], t["weight"][..., :60]]}]
    for o in ways:
        told = []
        for extension in (True, False):
            with monkeypatch.context() as m:
                if not extension:
                    m.setattr(rf, "_calls", None)
                with pytest.raises((ValueError, TypeError, RuntimeError)) as e:
                    call(**o)
                told.append((type(e.value), str(e.value)))
        assert told[0] == told[1], list(o)


def test_numbers_of_other_types(rf):
    """What the extension does not take (numpy's integers, an int as the scale) still works."""
    np = pytest.importorskip("numpy")
    t = inputs(torch.bfloat16)
    c = calls(rf, t)
    same(c["window"](window=np.int64(50), scale=1), c["window"](scale=1.0))


def test_leaves_that_require_gradients_are_not_recorded(rf):
    t = inputs(torch.bfloat16)
    q = t["q"].clone().requires_grad_()
    same(calls(rf, t)["window"](q=q), calls(rf, t)["window"]())


def test_captured(rf, monkeypatch):
    t = inputs(torch.bfloat16)
    c = calls(rf, t)
    seen = counted(rf, monkeypatch)
    want = [c[n]() for n in NAMES]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = [c[n]() for n in NAMES]
    assert len(seen) == 2 * len(NAMES) and all(type(r) is tuple for r in seen)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        same(a, b)
