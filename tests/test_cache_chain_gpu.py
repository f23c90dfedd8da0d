"""Calls over a serving cache, one behind the other on a stream, each reading what the one before
wrote: kernels that are set up beside their predecessor's end must not read ahead of it."""

import pytest
import torch

from cache_helpers import normal

pytestmark = pytest.mark.gpu

B, H, HKV, CAP, D, PREFIX, KEEP = 2, 8, 2, 700, 128, 600, 256


@pytest.fixture(scope="module")
def rf():
    import cascaded_reductions_gb300 as m
    return m


class Loop:
    """A decode loop: window decode -> shared-prefix decode -> weight totals -> eviction -> decode of
    what was kept -> windowed prefill over it, every call's output the next one's input."""

    def __init__(self, rf, large=False):
        self.rf, self.B = rf, 24 if large else B
        b, cap = self.B, 6000 if large else CAP
        self.q = normal(1, b, H, D).cuda()
        self.k0, self.v0 = normal(2, b, HKV, cap, D).cuda(), normal(3, b, HKV, cap, D).cuda()
        self.k, self.v = torch.empty_like(self.k0), torch.empty_like(self.v0)
        self.kp, self.vp = normal(4, HKV, PREFIX, D).cuda(), normal(5, HKV, PREFIX, D).cuda()
        self.lens0 = torch.tensor([cap - 37 * i % cap for i in range(b)], dtype=torch.int32).cuda()
        self.lens = torch.empty_like(self.lens0)
        self.works = [rf.decode_workspace(b, H, HKV, cap, window=200, sinks=4),
                      rf.decode_workspace(b, H, HKV, cap, prefix=PREFIX),
                      rf.decode_workspace(b, H, HKV, cap, weights=True),
                      rf.decode_workspace(b, H, HKV, KEEP)]
        self.kept = [torch.zeros(b, HKV, KEEP, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.kept.append(torch.zeros(b, HKV, KEEP, device="cuda"))

    def fill(self):
        """The cache and its lengths, written just before the first call reads them."""
        self.k.copy_(self.k0)
        self.v.copy_(self.v0)
        self.lens.copy_(self.lens0)

    def steps(self, q, pause):
        rf, w = self.rf, self.works
        outs = []
        for _ in range(3):
            a, _ = rf.attn_decode_window(q, self.k, self.v, self.lens, window=200, sinks=4, work=w[0])
            pause()
            b, _ = rf.attn_decode_shared(a, self.kp, self.vp, self.k, self.v, self.lens, work=w[1])
            pause()
            c, lse, total = rf.attn_decode_weights(b, self.k, self.v, self.lens, work=w[2])
            pause()
            *_, lens, kept = rf.cache_evict(self.k, self.v, total, self.lens, KEEP, sinks=4, recent=32,
                                            out=self.kept)
            pause()
            d, _ = rf.attn_decode_window(c, self.kept[0], self.kept[1], lens, work=w[3])
            pause()
            e, _ = rf.attn_prefill_window(d.view(self.B, H, 1, D), self.kept[0], self.kept[1], window=100)
            pause()
            q = e.view(self.B, H, D)
            outs += [a, b, c, lse, total, lens, kept, d, q]
        return outs


def same(got, want):
    for i, (a, b) in enumerate(zip(got, want, strict=True)):
        assert torch.equal(a.nan_to_num(), b.nan_to_num()), i


@pytest.mark.parametrize("large", [False, True])
def test_back_to_back(rf, large):
    loop = Loop(rf, large)
    loop.fill()
    want = [x.clone() for x in loop.steps(loop.q, torch.cuda.synchronize)]
    for _ in range(5):
        loop.k.zero_()
        loop.v.zero_()
        loop.lens.zero_()
        torch.cuda.synchronize()
        loop.fill()
        got = loop.steps(loop.q, lambda: None)
        torch.cuda.synchronize()
        same(got, want)


@pytest.mark.parametrize("before", ["kernel", "copy", "joined stream", "memset"])
def test_captured_behind_other_work(rf, before):
    """The first call of a graph behind a kernel, a copy between tensors, work of another stream
    that joins, or an allocation's zeroing."""
    loop = Loop(rf)
    loop.fill()
    want = [x.clone() for x in loop.steps(loop.q, torch.cuda.synchronize)]
    loop.k.zero_()
    loop.v.zero_()
    loop.lens.zero_()
    torch.cuda.synchronize()
    graph, side, other = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        if before == "joined stream":
            other.wait_stream(side)
            with torch.cuda.stream(other):
                loop.k.copy_(loop.k0)
                loop.lens.copy_(loop.lens0)
            loop.v.copy_(loop.v0)
            side.wait_stream(other)
        else:
            loop.fill()
            if before == "kernel":
                loop.k.mul_(1)
            if before == "memset":
                loop.kept[0].zero_()
        got = loop.steps(loop.q, lambda: None)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        same(got, want)


@pytest.mark.parametrize("call", ["decode", "prefix", "evict", "prefill"])
def test_first_call_of_a_graph_and_of_a_stream(rf, call):
    """A call with nothing before it, and one that another stream's work precedes."""
    loop = Loop(rf)
    loop.fill()
    weight = normal(9, B, HKV, CAP, dtype=torch.float32).cuda()

    def run():
        if call == "decode":
            return list(rf.attn_decode_window(loop.q, loop.k, loop.v, loop.lens, work=loop.works[0]))
        if call == "prefix":
            return list(rf.attn_decode_shared(loop.q, loop.kp, loop.vp, loop.k, loop.v, loop.lens,
                                              work=loop.works[1]))
        if call == "evict":
            return list(rf.cache_evict(loop.k, loop.v, weight, loop.lens, KEEP, out=loop.kept))
        return list(rf.attn_prefill_window(loop.q.view(B, H, 1, D), loop.k, loop.v, window=50))
    torch.cuda.synchronize()
    want = [x.clone() for x in run()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    graph.replay()
    torch.cuda.synchronize()
    same(got, want)
    loop.k.zero_()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        loop.k.copy_(loop.k0)
    b.wait_stream(a)
    with torch.cuda.stream(b):
        got = run()
    torch.cuda.synchronize()
    same(got, want)
