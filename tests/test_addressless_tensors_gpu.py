"""Tensors that have a shape but no address (their memory was given back, or they stand for a batch
of tensors inside a transform) are refused with a Python error by every call over a serving cache,
as marshalled by the extension and in Python."""

import pytest
import torch

from cache_helpers import normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


def calls(rf):
    t = dict(q=normal(1, 2, 8, 128), qs=normal(2, 2, 8, 70, 128), k=normal(3, 2, 2, 90, 128),
             v=normal(4, 2, 2, 90, 128), kp=normal(5, 2, 60, 128), vp=normal(6, 2, 60, 128),
             lens=torch.tensor([90, 5], dtype=torch.int32), weight=normal(7, 2, 2, 90, dtype=torch.float32),
             k_out=torch.zeros(2, 2, 20, 128, dtype=torch.bfloat16), w_out=torch.zeros(2, 2, 20))
    t = {n: x.cuda() for n, x in t.items()}
    work = rf.decode_workspace(2, 8, 2, 90, prefix=60, weights=True)
    return {
        "window": (lambda a: rf.attn_decode_window(a["q"], a["k"], a["v"], a["lens"], work=work),
                   ("q", "k", "v", "lens")),
        "shared": (lambda a: rf.attn_decode_shared(a["q"], a["kp"], a["vp"], a["k"], a["v"], a["lens"], work=work),
                   ("q", "kp", "vp", "k", "v", "lens")),
        "weights": (lambda a: rf.attn_decode_weights(a["q"], a["k"], a["v"], a["lens"], a["weight"], work=work),
                    ("q", "k", "v", "lens", "weight")),
        "prefill": (lambda a: rf.attn_prefill_window(a["qs"], a["k"], a["v"]), ("qs", "k", "v")),
        "evict": (lambda a: rf.cache_evict(a["k"], None, a["weight"], a["lens"], 20, out=(a["k_out"], None, a["w_out"])),
                  ("k", "weight", "lens", "k_out", "w_out")),
    }, t


NAMES = ("window", "shared", "weights", "prefill", "evict")


@pytest.mark.parametrize("extension", [True, False])
@pytest.mark.parametrize("name", NAMES)
def test_memory_given_back(rf, monkeypatch, name, extension):
    if not extension:
        monkeypatch.setattr(rf, "_calls", None)
    every, t = calls(rf)
    call, names = every[name]
    call(t)
    for n in names:
        gone = t[n].clone()
        gone.untyped_storage().resize_(0)
        with pytest.raises((RuntimeError, ValueError)):
            call({**t, n: gone})
    call(t)
    torch.cuda.synchronize()


@pytest.mark.parametrize("extension", [True, False])
@pytest.mark.parametrize("name", NAMES)
def test_inside_a_batched_transform(rf, monkeypatch, name, extension):
    if not extension:
        monkeypatch.setattr(rf, "_calls", None)
    every, t = calls(rf)
    call, names = every[name]
    for n in names:
        with pytest.raises((RuntimeError, ValueError, TypeError)):
            torch.func.vmap(lambda x: call({**t, n: x}), randomness="different")(torch.stack([t[n]] * 3))
    call(t)
    torch.cuda.synchronize()
