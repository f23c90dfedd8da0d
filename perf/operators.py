"""Measured cases of the cache-attention operators.

Five operators on a serving cache of grouped heads, 16-bit, head dimension 128:

* prefill of N query rows at the end of L positions with a sliding window and
  a few first tokens (sinks) that stay visible;
* the single-token form of the same mask over a ragged batch of caches;
* single-token decode of a batch that shares one long prefix;
* single-token decode that also adds each key's attention weight to a running
  total per key;
* eviction from the cache by that total.

``own`` selects between the plain torch form of each operator and the
library's kernels.  Sizes follow the library's own workloads (32 heads of 128,
32768 cached keys, 8192-row prompts) and smaller or odd ones around them.
"""

import math

import numpy as np
import torch

own = False

D = 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one user's chat turn on a windowed model: latency of a single token
        {"name": "window-decode-one", "op": "decode_window", "B": 1, "H": 32, "Hkv": 8,
         "cap": 4096, "window": 1024, "sinks": 4, "dtype": "bf16"},
        # a full serving batch of long ragged conversations on a windowed model
        {"name": "window-decode-batch", "op": "decode_window", "B": 64, "H": 32, "Hkv": 8,
         "cap": 16384, "window": 4096, "sinks": 4, "dtype": "bf16"},
        # a short prompt of odd length
        {"name": "window-prefill-short", "op": "prefill_window", "B": 1, "H": 32, "Hkv": 8,
         "N": 777, "L": 777, "window": 256, "sinks": 4, "dtype": "fp16"},
        # one chunk of a long document, appended to an existing cache
        {"name": "window-prefill-chunk", "op": "prefill_window", "B": 1, "H": 32, "Hkv": 8,
         "N": 512, "L": 12345, "window": 4096, "sinks": 4, "dtype": "bf16"},
        # a batch of long prompts
        {"name": "window-prefill-long", "op": "prefill_window", "B": 4, "H": 32, "Hkv": 8,
         "N": 8192, "L": 8192, "window": 1024, "sinks": 16, "dtype": "bf16"},
        # four samples of one short prompt
        {"name": "shared-few", "op": "decode_shared", "B": 4, "H": 32, "Hkv": 8, "prefix": 1000,
         "cap": 64, "dtype": "bf16"},
        # a large batch behind one long document
        {"name": "shared-batch", "op": "decode_shared", "B": 128, "H": 32, "Hkv": 8,
         "prefix": 32768, "cap": 512, "dtype": "bf16"},
        # the same with a key head for every query head, behind a system prompt
        {"name": "shared-mha", "op": "decode_shared", "B": 32, "H": 32, "Hkv": 32, "prefix": 8192,
         "cap": 1024, "dtype": "fp16"},
        # a single sequence that keeps count of its keys' weights
        {"name": "weights-one", "op": "decode_weights", "B": 1, "H": 32, "Hkv": 8, "cap": 2048,
         "dtype": "bf16"},
        # a serving batch that does
        {"name": "weights-batch", "op": "decode_weights", "B": 32, "H": 32, "Hkv": 8,
         "cap": 16384, "dtype": "bf16"},
        # one sequence's cache halved
        {"name": "evict-one", "op": "evict", "B": 1, "Hkv": 8, "cap": 2048, "keep": 1024,
         "sinks": 4, "recent": 256, "dtype": "bf16"},
        # a serving batch's caches brought down to a budget; some are within it already
        {"name": "evict-batch", "op": "evict", "B": 32, "Hkv": 8, "cap": 16384, "keep": 4096,
         "sinks": 4, "recent": 1024, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges, no more work than the largest of its operator."""
    op = rng.choice(["decode_window", "prefill_window", "decode_shared", "decode_weights", "evict"])
    top = [work(c) for c in listed() if c["op"] == op]
    while True:
        Hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
        H = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        c = {"op": op, "dtype": rng.choice(["bf16", "fp16"])}
        if op == "prefill_window":
            N = _log_int(rng, 1, 8192)
            c.update(B=_log_int(rng, 1, 4), H=H, Hkv=Hkv, N=N,
                     L=N + (0 if rng.random() < 0.5 else _log_int(rng, 1, 16384)),
                     window=_log_int(rng, 16, 4096), sinks=rng.choice([0, 1, 4, 16, 64]))
        elif op == "decode_window":
            c.update(B=_log_int(rng, 1, 64), H=H, Hkv=Hkv, cap=_log_int(rng, 16, 32768),
                     window=_log_int(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 16, 64]))
        elif op == "decode_shared":
            c.update(B=_log_int(rng, 1, 128), H=H, Hkv=Hkv, prefix=_log_int(rng, 16, 32768),
                     cap=_log_int(rng, 1, 1024))
        elif op == "decode_weights":
            c.update(B=_log_int(rng, 1, 32), H=H, Hkv=Hkv, cap=_log_int(rng, 16, 32768))
        else:
            cap = _log_int(rng, 64, 32768)
            keep = max(32, int(cap * rng.uniform(0.1, 0.9)))
            c.update(B=_log_int(rng, 1, 32), Hkv=Hkv, cap=cap, keep=keep,
                     sinks=rng.choice([0, 1, 4, 16]),
                     recent=_log_int(rng, 1, max(1, keep // 2)))
        w = work(c)
        if (H <= 64 and w["bytes"] <= max(t["bytes"] for t in top)
                and w["flops"] <= max(t["flops"] for t in top)):
            return c


def _spread(B, cap):
    """Ragged lengths from cap down to a quarter of it, cap among them."""
    return [max(1, cap - (3 * cap * b) // (4 * B)) for b in range(B)]


def _visible(length, window, sinks):
    lo = max(0, length - window)
    return min(sinks, lo) + length - lo


def work(case):
    c, op = case, case["op"]
    if op == "evict":
        lens = _spread(c["B"], c["cap"])
        kept = sum(min(n, c["keep"]) for n in lens) * c["Hkv"]
        # the weights are read whole; K, V and weight of the kept keys move; their
        # indices and the new lengths are written
        return {"bytes": 4 * sum(lens) * c["Hkv"] + kept * 2 * (2 * 2 * D)
                + kept * 4 + 4 * c["B"] * c["Hkv"] * c["keep"] + 8 * c["B"],
                "flops": sum(lens) * c["Hkv"]}
    B, H, Hkv = c["B"], c["H"], c["Hkv"]
    if op == "prefill_window":
        N, L = c["N"], c["L"]
        pairs = sum(_visible(p + 1, c["window"], c["sinks"]) for p in range(L - N, L))
        lo = max(0, L - N + 1 - c["window"])
        keys = L - lo + min(c["sinks"], lo)
        return {"bytes": B * (2 * H * N * 2 * D + 4 * H * N + 2 * Hkv * keys * 2 * D),
                "flops": B * H * pairs * 4 * D}
    rows = B * H
    io = rows * (2 * 2 * D + 4) + 4 * B
    if op == "decode_window":
        keys = sum(_visible(n, c["window"], c["sinks"]) for n in _spread(B, c["cap"]))
        return {"bytes": io + Hkv * keys * 2 * 2 * D, "flops": H * keys * 4 * D}
    keys = sum(_spread(B, c["cap"]))
    if op == "decode_shared":
        return {"bytes": io + Hkv * (keys + c["prefix"]) * 2 * 2 * D,
                "flops": H * (keys + B * c["prefix"]) * 4 * D}
    return {"bytes": io + Hkv * keys * (2 * 2 * D + 8), "flops": H * keys * 4 * D}


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    """Normal queries, keys and values; lengths spread over the batch; weights as
    decode steps leave them: a few large, most small, new keys at zero."""
    c = dict(case)
    dt = DTYPES[c["dtype"]]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)

    st = {"case": c, "scale": D ** -0.5}
    B, Hkv = c["B"], c["Hkv"]
    if c["op"] == "prefill_window":
        st.update(q=normal(B, c["H"], c["N"], D), k=normal(B, Hkv, c["L"], D),
                  v=normal(B, Hkv, c["L"], D))
        return st
    order = torch.randperm(B, generator=g, device="cuda")
    st["lens"] = torch.tensor(_spread(B, c["cap"]), dtype=torch.int32, device="cuda")[order]
    st["k"], st["v"] = normal(B, Hkv, c["cap"], D), normal(B, Hkv, c["cap"], D)
    if c["op"] in ("decode_weights", "evict"):
        w = torch.rand(B, Hkv, c["cap"], generator=g, device="cuda") ** 6 * 4
        st["weight"] = w * (torch.rand(w.shape, generator=g, device="cuda") > 0.05)
    if c["op"] == "evict":
        # the destination cache; rows behind a short sequence stay as they are
        st.update(k_out=torch.zeros(B, Hkv, c["keep"], D, dtype=dt, device="cuda"),
                  v_out=torch.zeros(B, Hkv, c["keep"], D, dtype=dt, device="cuda"),
                  weight_out=torch.zeros(B, Hkv, c["keep"], device="cuda"))
        return st
    st["q"] = normal(B, c["H"], D)
    if c["op"] == "decode_shared":
        st["kp"], st["vp"] = normal(Hkv, c["prefix"], D), normal(Hkv, c["prefix"], D)
    if own:
        # the segment states and counters that a serving loop allocates once
        import cascaded_reductions_gb300 as rf
        st["work"] = rf.decode_workspace(B, c["H"], Hkv, c["cap"], prefix=c.get("prefix", 0),
                                         window=c.get("window", 0), sinks=c.get("sinks", 0),
                                         weights=c["op"] == "decode_weights")
    return st


# -------------------------------------------------------------- plain form --

def _softmax_parts(s):
    """exp(s - max), its sum and the max of each row; a row of -inf gives zeros."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return p, p.sum(-1, keepdim=True), m


def _finish(acc, l, m, dt):
    out = torch.where(l > 0, acc / l, torch.zeros_like(acc))
    return out.to(dt), (m + torch.log(l)).squeeze(-1)


def _plain_decode(q, k, v, lens, window, sinks, scale):
    B, H, _ = q.shape
    Hkv, cap = k.shape[1], k.shape[2]
    lens = lens.long()[:, None]
    window = window or cap
    lo = (lens - window).clamp(min=0)
    ns = lo.clamp(max=sinks)
    t = torch.arange(min(cap, window + sinks), device=q.device)[None]
    idx = torch.where(t < ns, t, t - ns + lo)                   # visible keys, in order
    live = t < ns + lens - lo
    idx = idx.clamp(max=cap - 1)
    b = torch.arange(B, device=q.device)[:, None, None]
    h = torch.arange(Hkv, device=q.device)[None, :, None]
    kf, vf = k[b, h, idx[:, None]].float(), v[b, h, idx[:, None]].float()
    s = torch.matmul(q.float().view(B, Hkv, H // Hkv, D), kf.transpose(-1, -2)) * scale
    s = s.masked_fill(~live[:, None, None], -math.inf)
    p, l, m = _softmax_parts(s)
    out, lse = _finish(torch.matmul(p, vf), l, m, q.dtype)
    return out.view(B, H, D), lse.view(B, H), p / l


def _plain_prefill(q, k, v, window, sinks, scale):
    B, H, N, _ = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    G = H // Hkv
    C = min(N, 512)                                             # query rows of a block
    nb = (N + C - 1) // C
    qf = torch.nn.functional.pad(q.float(), (0, 0, 0, nb * C - N)).view(B, Hkv, G, nb, C, D)
    first = L - N + C * torch.arange(nb, device=q.device)       # position of each block's first row
    span = min(L, window - 1) + C
    idx = first[:, None] - (span - C) + torch.arange(span, device=q.device)[None]
    idx = torch.cat([torch.arange(sinks, device=q.device).expand(nb, sinks), idx], 1)
    pos = (first[:, None] + torch.arange(C, device=q.device)[None])[:, :, None]
    j = idx[:, None]
    near = (j > pos - window) & (j <= pos) & (j >= 0)
    is_sink = torch.arange(sinks + span, device=q.device)[None, None] < sinks
    seen = torch.where(is_sink, (j <= pos - window), near)      # sinks inside the window count once
    at = idx.clamp(0, L - 1)
    kf, vf = k[:, :, at].float().unsqueeze(2), v[:, :, at].float().unsqueeze(2)
    s = torch.matmul(qf, kf.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    p, l, m = _softmax_parts(s)
    out, lse = _finish(torch.matmul(p, vf), l, m, q.dtype)
    return out.reshape(B, H, nb * C, D)[:, :, :N], lse.reshape(B, H, nb * C)[:, :, :N]


def _plain_shared(q, kp, vp, k, v, lens, scale):
    B, H, _ = q.shape
    Hkv, P, cap = k.shape[1], kp.shape[1], k.shape[2]
    qf = q.float().view(B, Hkv, H // Hkv, D)
    s1 = torch.einsum("bhgd,hld->bhgl", qf, kp.float()) * scale
    s2 = torch.matmul(qf, k.float().transpose(-1, -2)) * scale
    live = torch.arange(cap, device=q.device)[None] < lens[:, None]
    s2 = s2.masked_fill(~live[:, None, None], -math.inf)
    p, l, m = _softmax_parts(torch.cat([s1, s2], -1))
    acc = torch.einsum("bhgl,hld->bhgd", p[..., :P], vp.float()) + torch.matmul(p[..., P:], v.float())
    out, lse = _finish(acc, l, m, q.dtype)
    return out.view(B, H, D), lse.view(B, H)


def _plain_evict(k, v, weight, lens, keep, sinks, recent, k_out, v_out, weight_out):
    B, Hkv, cap = weight.shape
    j = torch.arange(cap, device=k.device)
    n = lens.long()[:, None, None]
    rank = torch.where((j < sinks) | (j >= n - recent), 0, 1)    # protected keys first
    rank = torch.where(j < n, rank, 2).expand(B, Hkv, cap)       # then by weight; behind the end last
    by_weight = torch.sort(weight, dim=-1, descending=True, stable=True).indices
    order = by_weight.gather(-1, torch.sort(rank.gather(-1, by_weight), dim=-1, stable=True).indices)
    count = n.clamp(max=keep)
    slot = torch.arange(keep, device=k.device)
    full = order if cap >= keep else torch.nn.functional.pad(order, (0, keep - cap), value=cap)
    kept = torch.where(slot < count, full[..., :keep], cap).sort(-1).values
    live = slot < count
    at = kept.clamp(max=cap - 1)
    rows = at[..., None].expand(B, Hkv, keep, D)
    return (torch.where(live[..., None], k.gather(2, rows), k_out),
            torch.where(live[..., None], v.gather(2, rows), v_out),
            torch.where(live, weight.gather(2, at), weight_out),
            count[:, 0, 0].int(), torch.where(live, kept, -1).int())


def run(state):
    c = state["case"]
    op, scale = c["op"], state["scale"]
    if own:
        import cascaded_reductions_gb300 as rf
        if op == "decode_window":
            return rf.attn_decode_window(state["q"], state["k"], state["v"], state["lens"],
                                         window=c["window"], sinks=c["sinks"], scale=scale,
                                         work=state["work"])
        if op == "prefill_window":
            return rf.attn_prefill_window(state["q"], state["k"], state["v"], window=c["window"],
                                          sinks=c["sinks"], scale=scale)
        if op == "decode_shared":
            return rf.attn_decode_shared(state["q"], state["kp"], state["vp"], state["k"],
                                         state["v"], state["lens"], scale=scale,
                                         work=state["work"])
        if op == "decode_weights":
            return rf.attn_decode_weights(state["q"], state["k"], state["v"], state["lens"],
                                          weight=state["weight"], scale=scale, work=state["work"])
        return rf.cache_evict(state["k"], state["v"], state["weight"], state["lens"], c["keep"],
                              sinks=c["sinks"], recent=c["recent"],
                              out=(state["k_out"], state["v_out"], state["weight_out"]))
    if op == "decode_window":
        return _plain_decode(state["q"], state["k"], state["v"], state["lens"], c["window"],
                             c["sinks"], scale)[:2]
    if op == "prefill_window":
        return _plain_prefill(state["q"], state["k"], state["v"], c["window"], c["sinks"], scale)
    if op == "decode_shared":
        return _plain_shared(state["q"], state["kp"], state["vp"], state["k"], state["v"],
                             state["lens"], scale)
    if op == "decode_weights":
        out, lse, p = _plain_decode(state["q"], state["k"], state["v"], state["lens"], 0, 0, scale)
        return out, lse, _add_weights(state["weight"], p, state["lens"])
    return _plain_evict(state["k"], state["v"], state["weight"], state["lens"], c["keep"],
                        c["sinks"], c["recent"], state["k_out"], state["v_out"],
                        state["weight_out"])


def _add_weights(weight, p, lens):
    """Each key's total over the query heads of its group; behind the end nothing is added."""
    return weight + torch.nan_to_num(p, nan=0.0).sum(2)


# ------------------------------------------------------------- 64-bit form --

def _exact_rows(q, k, v, scale):
    """Softmax attention of rows q [..., D] over keys k [n, D], from the definition."""
    logits = (q.double() @ k.double().T) * scale
    lse = torch.logsumexp(logits, -1)
    w = torch.exp(logits - lse[..., None])
    return w @ v.double(), lse, w


def exact(case, seed):
    st = prepare(case, seed)
    c, op, scale = st["case"], st["case"]["op"], st["scale"]
    k, v = st["k"], st["v"]
    if op == "evict":
        return _exact_evict(st, c)
    q = st["q"]
    G = c["H"] // c["Hkv"]
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(q.shape[:-1], dtype=torch.float64, device="cuda")
    if op == "prefill_window":
        step = 256
        for b in range(c["B"]):
            for h in range(c["H"]):
                for i in range(0, c["N"], step):
                    pos = torch.arange(c["L"] - c["N"] + i,
                                       c["L"] - c["N"] + min(i + step, c["N"]), device="cuda")
                    lo = max(0, int(c["L"] - c["N"] + i) - c["window"] + 1)
                    keys = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"),
                                      torch.arange(lo, c["L"] - c["N"] + min(i + step, c["N"]),
                                                   device="cuda")])
                    s = (q[b, h, i:i + step].double() @ k[b, h // G, keys].double().T) * scale
                    hidden = (keys > pos[:, None]) | ((keys <= pos[:, None] - c["window"])
                                                      & (keys >= c["sinks"]))
                    s[hidden] = -math.inf
                    z = torch.logsumexp(s, -1)
                    lse[b, h, i:i + step] = z
                    out[b, h, i:i + step] = torch.exp(s - z[:, None]) @ v[b, h // G, keys].double()
        return out, lse
    if op == "decode_weights":
        total = st["weight"].double()
    for b, n in enumerate(st["lens"].tolist()):
        if op == "decode_window":
            lo = max(0, n - c["window"])
            keys = list(range(min(c["sinks"], lo))) + list(range(lo, n))
            keys = torch.tensor(keys, device="cuda")
        for h in range(c["Hkv"]):
            if op == "decode_window":
                kk, vv = k[b, h, keys], v[b, h, keys]
            elif op == "decode_shared":
                kk, vv = torch.cat([st["kp"][h], k[b, h, :n]]), torch.cat([st["vp"][h], v[b, h, :n]])
            else:
                kk, vv = k[b, h, :n], v[b, h, :n]
            g = slice(h * G, (h + 1) * G)
            out[b, g], lse[b, g], w = _exact_rows(q[b, g], kk, vv, scale)
            if op == "decode_weights":
                total[b, h, :n] += w.sum(0)
    return (out, lse, total) if op == "decode_weights" else (out, lse)


def _exact_evict(st, c):
    weight = st["weight"].cpu().numpy()
    lens = st["lens"].tolist()
    k_out, v_out = st["k_out"].double(), st["v_out"].double()
    w_out = st["weight_out"].double()
    kept = np.full((c["B"], c["Hkv"], c["keep"]), -1, np.int32)
    for b, n in enumerate(lens):
        count = min(n, c["keep"])
        first = min(c["sinks"], n)
        last = max(first, n - c["recent"])
        if n <= c["keep"]:
            rows = [np.arange(n)] * c["Hkv"]
        else:
            middle = np.arange(first, last)
            rows = [np.sort(np.concatenate([
                np.arange(first), np.arange(last, n),
                middle[np.lexsort((middle, -weight[b, h, first:last]))][:count - first - (n - last)]]))
                for h in range(c["Hkv"])]
        for h, r in enumerate(rows):
            kept[b, h, :count] = r
            at = torch.from_numpy(r).to("cuda")
            k_out[b, h, :count] = st["k"][b, h, at].double()
            v_out[b, h, :count] = st["v"][b, h, at].double()
            w_out[b, h, :count] = st["weight"][b, h, at].double()
    new = torch.tensor([min(n, c["keep"]) for n in lens], dtype=torch.int32, device="cuda")
    return k_out, v_out, w_out, new, torch.from_numpy(kept).to("cuda")
