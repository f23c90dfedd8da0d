"""Measured cases of the operators of a serving step over a paged cache.

Three operators, in the order of a step:

* page tables: pages for the new tokens of a ragged batch of requests, taken from
  a stack of free ones, and each new token's position and slot in the cache;
* norm and rotation: the norm of each query and key head, the rotation by a
  position of one or several axes, and the write of keys and values into the
  cache's pages, in one pass;
* attention of the new tokens over the pages: single tokens, a few drafted ones,
  chunks of prompts, and batches that mix them.

``own`` selects between the plain torch form of each operator and the library's
kernels.  Sizes follow the library's own workloads (32 heads of 128 over 8 key
heads, 32768 cached keys, 8192-row prompts) and smaller or odd ones around them.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
D = 128                                # attention's head dimension


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one user's next token: latency of the smallest step
        {"name": "tables-one", "op": "tables", "B": 1, "longest": 1500, "page": 16, "ended": 0,
         "prompts": 0, "chunk": 1, "spare": 1.0},
        # a large server's step: many decodes, some prompt chunks, some requests that ended
        {"name": "tables-batch", "op": "tables", "B": 256, "longest": 32768, "page": 16,
         "ended": 9, "prompts": 25, "chunk": 4096, "spare": 1.2},
        # one token of one user, written to the cache
        {"name": "rope-one", "op": "rope", "T": 1, "H": 32, "Hkv": 8, "D": 128, "R": 128, "axes": 1,
         "interleaved": False, "norm": True, "page": 16, "far": 4096, "dtype": "bf16"},
        # a batch of single tokens at far positions, half of each head rotated
        {"name": "rope-batch", "op": "rope", "T": 193, "H": 32, "Hkv": 8, "D": 128, "R": 64,
         "axes": 1, "interleaved": True, "norm": True, "page": 64, "far": 1000000, "dtype": "fp16"},
        # a chunk of prompts, written to the cache
        {"name": "rope-prompt", "op": "rope", "T": 8192, "H": 32, "Hkv": 8, "D": 128, "R": 128,
         "axes": 1, "interleaved": False, "norm": True, "page": 64, "far": 32768, "dtype": "bf16"},
        # frames of a video between text, three axes (time, height, width), outside a cache
        {"name": "rope-video", "op": "rope", "T": 14007, "H": 16, "Hkv": 16, "D": 128, "R": 128,
         "axes": 3, "interleaved": False, "norm": True, "page": 0, "far": 20000, "dtype": "bf16"},
        # one user's next token behind a conversation
        {"name": "paged-one", "op": "attn", "B": 1, "longest": 4097, "prompts": 0, "chunk": 1,
         "H": 32, "Hkv": 8, "page": 16, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a full batch of single tokens behind long ragged contexts
        {"name": "paged-batch", "op": "attn", "B": 64, "longest": 16384, "prompts": 0, "chunk": 1,
         "H": 32, "Hkv": 8, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # four drafted tokens each, checked at once
        {"name": "paged-draft", "op": "attn", "B": 17, "longest": 8191, "prompts": 17, "chunk": 4,
         "H": 32, "Hkv": 8, "page": 32, "window": 0, "sinks": 0, "dtype": "fp16"},
        # one chunk of a long document behind what the cache holds
        {"name": "paged-chunk", "op": "attn", "B": 1, "longest": 32768, "prompts": 1, "chunk": 512,
         "H": 32, "Hkv": 8, "page": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # decodes beside two prompt chunks on a windowed model
        {"name": "paged-mixed", "op": "attn", "B": 34, "longest": 12345, "prompts": 2,
         "chunk": 2048, "H": 32, "Hkv": 8, "page": 16, "window": 4096, "sinks": 4, "dtype": "bf16"},
        # a batch of long prompts, whole
        {"name": "paged-prompts", "op": "attn", "B": 4, "longest": 8192, "prompts": 4,
         "chunk": 8192, "H": 32, "Hkv": 8, "page": 128, "window": 0, "sinks": 0, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges, no more work than the largest of its operator."""
    op = rng.choice(["tables", "rope", "attn", "attn"])
    top = [work(c) for c in listed() if c["op"] == op]
    while True:
        Hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
        H = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        page = rng.choice([16, 32, 64, 128, 256])
        dtype = rng.choice(["bf16", "fp16"])
        if op == "rope":
            d = rng.choice([64, 128, 128, 256])
            c = {"T": _log_int(rng, 1, 16384), "H": H, "Hkv": Hkv, "D": d,
                 "R": rng.choice([d, d, d // 2, 48]), "axes": rng.choice([1, 1, 2, 3]),
                 "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.8,
                 "page": rng.choice([0, page]), "far": _log_int(rng, 64, 1000000), "dtype": dtype}
        else:
            B = _log_int(rng, 1, 512 if op == "tables" else 64)
            longest = _log_int(rng, 1, 32768)
            kind = rng.choice(["single", "few", "mixed", "prompts"])
            chunk = 1 if kind == "single" else rng.randint(2, 9) if kind == "few" else _log_int(rng, 10, 8192)
            prompts = {"single": 0, "few": B, "mixed": max(1, B // 8), "prompts": B}[kind]
            c = {"B": B, "longest": longest, "page": page, "prompts": prompts,
                 "chunk": min(chunk, longest)}
            if op == "tables":
                c.update(ended=rng.randint(0, B // 4), spare=rng.choice([0.5, 1.0, 1.5]))
                c["prompts"] = min(c["prompts"], B - c["ended"])
            else:
                c.update(H=H, Hkv=Hkv, dtype=dtype, window=rng.choice([0, 0, _log_int(rng, 16, 8192)]),
                         sinks=rng.choice([0, 4, 64]))
        c["op"] = op
        w = work(c)
        if (H <= 64 and w["bytes"] <= max(t["bytes"] for t in top)
                and w["flops"] <= max(t["flops"] for t in top)
                and (op != "attn" or sum(_news(c)) * H <= 32 * 32768)
                and (op != "tables" or sum(max(0, n) for n in _news(c)) <= 131072)):
            return c


def _lens(c):
    """Keys of each request after the step, from the longest down to a quarter of it."""
    B, top = c["B"], c["longest"]
    return [max(1, top - (3 * top * b) // (4 * B)) for b in range(B)]


def _news(c):
    """New tokens of each request: the first ones have a chunk, the last ones ended (-1),
    the others have one token."""
    lens, ended = _lens(c), c.get("ended", 0)
    news = [min(c["chunk"], n) if b < c["prompts"] else 1 for b, n in enumerate(lens)]
    return [-1 if b >= c["B"] - ended else n for b, n in enumerate(news)]


def _pages(n, page):
    return (n + page - 1) // page


def _visible(p, window, sinks):
    lo = max(0, p + 1 - window) if window else 0
    return min(sinks, lo) + p + 1 - lo


def work(case):
    c, op = case, case["op"]
    if op == "tables":
        T = sum(n for n in _news(c) if n > 0)
        lens, news = _lens(c), _news(c)
        moved = sum(_pages(n, c["page"]) if k < 0 else _pages(n, c["page"]) - _pages(n - k, c["page"])
                    for n, k in zip(lens, news))
        # lengths and new counts in, starts and lengths out, each page moved once from where
        # it is listed to where it goes, a position and a slot per token
        return {"bytes": 16 * c["B"] + 8 * moved + 8 * T, "flops": T + c["B"]}
    if op == "rope":
        heads = c["H"] + c["Hkv"] * (2 if c["page"] else 1)
        return {"bytes": c["T"] * (heads * c["D"] * 4 + 4 * c["axes"] + (4 if c["page"] else 0)),
                "flops": c["T"] * (c["H"] + c["Hkv"]) * c["D"] * 7}
    H, Hkv, window, sinks = c["H"], c["Hkv"], c["window"], c["sinks"]
    rows = pairs = keys = pages = 0
    for n, k in zip(_lens(c), _news(c)):
        lo = max(0, n - k + 1 - window) if window else 0
        rows += k
        keys += n - lo + min(sinks, lo)
        pages += _pages(n - lo + min(sinks, lo), c["page"])
        if window == 0:
            pairs += k * (n - k) + k * (k + 1) // 2
        else:
            pairs += sum(_visible(p, window, sinks) for p in range(n - k, n))
    return {"bytes": rows * H * (4 * D + 4) + Hkv * keys * 4 * D + 4 * pages + 8 * c["B"],
            "flops": pairs * H * 4 * D}


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"tables": _prepare_tables, "rope": _prepare_rope, "attn": _prepare_attn}[c["op"]](c, g, seed)


def _prepare_tables(c, g, seed):
    """Requests that hold pages scattered over the pool, and a stack of the free ones."""
    rng = random.Random(seed)
    B, page = c["B"], c["page"]
    order = rng.sample(range(B), B)
    news = [_news(c)[b] for b in order]
    lens = [_lens(c)[b] - max(0, n) for b, n in zip(order, news)]
    held = [_pages(n, page) for n in lens]
    need = sum(_pages(n + k, page) - h for n, k, h in zip(lens, news, held) if k > 0)
    width = max(_pages(c["longest"], page), 1)
    free = max(1, int(need * c["spare"]))
    P = sum(held) + free
    ids = torch.randperm(P, generator=g, device="cuda", dtype=torch.int32)
    row = torch.repeat_interleave(torch.arange(B), torch.tensor(held))
    col = torch.cat([torch.arange(h) for h in held]) if B else torch.empty(0)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[row.cuda(), col.cuda()] = ids[:sum(held)]
    stack = torch.full((P,), -1, dtype=torch.int32, device="cuda")
    stack[:free] = ids[sum(held):]
    as_int = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")       # noqa: E731
    return {"case": c, "lens": as_int(lens), "news": as_int(news), "table": table, "stack": stack,
            "n_free": as_int([free]), "tokens": max(1, sum(max(0, n) for n in news))}


def _prepare_rope(c, g, seed):
    """Rows of a projection of q, k and v; weights near 1; frequencies of base 10000."""
    T, H, Hkv, d, R, dt = c["T"], c["H"], c["Hkv"], c["D"], c["R"], DTYPES[c["dtype"]]
    rows = torch.randn(T, (H + 2 * Hkv) * d, generator=g, device="cuda", dtype=dt)
    q, k, v = rows.split([H * d, Hkv * d, Hkv * d], 1)
    st = {"case": c, "q": q.view(T, H, d), "k": k.view(T, Hkv, d), "v": v.view(T, Hkv, d),
          "eps": 1e-6}
    weight = lambda: (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt)   # noqa: E731
    st["qw"], st["kw"] = (weight(), weight()) if c["norm"] else (None, None)
    st["freq"] = (10000.0 ** (-torch.arange(R // 2, device="cuda", dtype=torch.float64) * 2 / R)).float()
    # text counts on by one on every axis; frames of 24 x 40 patches lie between
    rng = random.Random(seed)
    first = rng.randint(0, max(0, c["far"] - T))
    pos = (first + torch.arange(T, device="cuda", dtype=torch.int32)).expand(c["axes"], T).clone()
    if c["axes"] > 1:
        t = torch.arange(T, device="cuda")
        frame, patch = t // 960, t % 960
        grid = [frame, patch // 40, patch % 40][:c["axes"]]
        text = t % 1920 >= 1500
        for a, x in enumerate(grid):
            pos[a] = torch.where(text, pos[a], first + x)
    st["positions"] = pos
    if c["axes"] > 1:                    # time, height and width share the pairs in turn
        st["axis"] = (torch.arange(R // 2, device="cuda", dtype=torch.int32) * c["axes"]) // (R // 2)
    else:
        st["axis"] = None
    if c["page"]:
        P = _pages(T, c["page"]) + 5
        st["kp"] = torch.zeros(P, Hkv, c["page"], d, dtype=dt, device="cuda")
        st["vp"] = torch.zeros_like(st["kp"])
        st["slots"] = torch.randperm(P * c["page"], generator=g, device="cuda", dtype=torch.int32)[:T].contiguous()
        if T > 8:
            st["slots"][::97] = -1       # rows of padding, or of a request that got no pages
    return st


def _prepare_attn(c, g, seed):
    dt, H, Hkv, page = DTYPES[c["dtype"]], c["H"], c["Hkv"], c["page"]
    rng = random.Random(seed)
    order = rng.sample(range(c["B"]), c["B"])
    lens, news = [_lens(c)[b] for b in order], [_news(c)[b] for b in order]
    held = [_pages(n, page) for n in lens]
    P = sum(held) + 3
    ids = torch.randperm(P, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((c["B"], max(held)), -1, dtype=torch.int32, device="cuda")
    row = torch.repeat_interleave(torch.arange(c["B"]), torch.tensor(held))
    col = torch.cat([torch.arange(h) for h in held])
    table[row.cuda(), col.cuda()] = ids[:sum(held)]
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=dt)   # noqa: E731
    T = sum(news)
    starts = torch.tensor([0] + news, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    st = {"case": c, "q": normal(T, H, D), "kp": normal(P, Hkv, page, D),
          "vp": normal(P, Hkv, page, D), "table": table, "starts": starts,
          "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "scale": D ** -0.5,
          "host": (lens, news)}
    if own:
        # a step's plan serves all layers, and a loop keeps its buffers from step to step
        import cascaded_reductions_gb300 as rf
        st["plan"] = rf.paged_plan(st["starts"], st["lens"], T, H, Hkv, max_new=max(news),
                                   max_len=max(held) * page, window=c["window"], sinks=c["sinks"])
    return st


# -------------------------------------------------------------- plain form --

def _plain_tables(st):
    page, T = st["case"]["page"], st["tokens"]
    lens, news = st["lens"].long(), st["news"].long()
    n_free = st["n_free"].long()
    table, stack = st["table"].clone(), st["stack"].clone()
    width = table.shape[1]
    held = (lens + page - 1) // page
    # pages of ended requests go onto the stack, in order
    given = torch.where(news < 0, held, 0)
    at = n_free + given.cumsum(0) - given
    col = torch.arange(width, device=lens.device)
    gives = col < given[:, None]
    stack[(at[:, None] + col)[gives]] = table[gives]
    top = n_free + given.sum()
    # a request gets its pages if those of all up to it are there
    new = news.clamp(min=0)
    total = (lens + new + page - 1) // page
    need = torch.where(total <= width, total - held, 0)
    upto = need.cumsum(0)
    ok = (total <= width) & ((upto <= top) | (need == 0))
    took = torch.where(ok, need, 0)
    gets = (col >= held[:, None]) & (col < (held + took)[:, None])
    index = top - 1 - ((upto - need)[:, None] + col - held[:, None])
    table[gets] = stack[index[gets]]
    lens_out = torch.where(news < 0, 0, torch.where(ok, lens + new, lens))
    starts = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(T, device=lens.device)
    row = (t[:, None] >= starts[None, 1:]).sum(1)
    live = row < lens.shape[0]
    row = row.clamp(max=lens.shape[0] - 1)
    pos = torch.where(live, lens[row] + t - starts[row], 0)
    inside = live & ok[row]
    entry = table[row, (pos // page).clamp(max=width - 1)].long()
    slots = torch.where(inside, entry * page + pos % page, -1)
    return (starts.int(), pos.int(), slots.int(), lens_out.int(), (top - took.sum()).int(), table, stack)


def _plain_rope(st):
    c = st["case"]
    R, half = c["R"], c["R"] // 2
    pos = st["positions"]
    p = pos[0][:, None] if st["axis"] is None else pos[st["axis"].long()].T
    angle = p.double() * st["freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = []
    for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + st["eps"]) * w.float()
        if c["interleaved"]:
            a, b = y[..., 0:R:2], y[..., 1:R:2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = y[..., :half], y[..., half:R]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        out.append(torch.cat([r, y[..., R:]], -1).to(x.dtype))
    if not c["page"]:
        return out[0], out[1]
    keep = st["slots"] >= 0
    page, off = st["slots"][keep].long() // c["page"], st["slots"][keep].long() % c["page"]
    st["kp"][page, :, off] = out[1][keep]
    st["vp"][page, :, off] = st["v"][keep]
    return out[0], st["kp"], st["vp"]


def _hidden(first, rows, L, window, sinks, device):
    """True where key j of L is hidden from position first + i."""
    p = first + torch.arange(rows, device=device)[:, None]
    j = torch.arange(L, device=device)[None]
    hide = j > p
    if window:
        hide |= (j <= p - window) & (j >= sinks)
    return hide


def _plain_attn(st):
    c = st["case"]
    H, Hkv, page = c["H"], c["Hkv"], c["page"]
    G = H // Hkv
    T = st["q"].shape[0]
    out = torch.empty_like(st["q"])
    lse = torch.empty(T, H, device="cuda")
    t0 = 0
    for b, (L, N) in enumerate(zip(*st["host"])):
        ids = st["table"][b, :_pages(L, page)].long()
        k = st["kp"][ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :L].float()
        v = st["vp"][ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :L].float()
        step = max(1, min(N, (1 << 28) // (H * L)))
        for i in range(0, N, step):
            n = min(step, N - i)
            q = st["q"][t0 + i:t0 + i + n].float().view(n, Hkv, G, D).permute(1, 2, 0, 3)
            s = torch.matmul(q.reshape(Hkv, G * n, D), k.transpose(1, 2)).view(Hkv, G, n, L)
            s.mul_(st["scale"]).masked_fill_(_hidden(L - N + i, n, L, c["window"], c["sinks"], s.device),
                                             -math.inf)
            m = s.amax(-1, keepdim=True)
            p = s.sub_(m).exp_()
            z = p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(Hkv, G * n, L), v).view(Hkv, G, n, D) / z
            out[t0 + i:t0 + i + n] = o.permute(2, 0, 1, 3).reshape(n, H, D).to(out.dtype)
            lse[t0 + i:t0 + i + n] = (m + z.log()).squeeze(-1).permute(2, 0, 1).reshape(n, H)
        t0 += N
    return out, lse


def run(state):
    st, c = state, state["case"]
    if own:
        import cascaded_reductions_gb300 as rf
        if c["op"] == "tables":
            starts, positions, slots, lens, n_free = rf.page_tables(
                st["lens"], st["news"], st["table"], st["stack"], st["n_free"], c["page"], st["tokens"])
            return starts, positions, slots, lens, n_free, st["table"], st["stack"]
        if c["op"] == "rope":
            if c["page"]:
                q = rf.qk_norm_rope(st["q"], st["k"], st["positions"], st["freq"], st["qw"], st["kw"],
                                    axis=st["axis"], interleaved=c["interleaved"], eps=st["eps"],
                                    v=st["v"], slots=st["slots"], kp=st["kp"], vp=st["vp"])
                return q, st["kp"], st["vp"]
            return rf.qk_norm_rope(st["q"], st["k"], st["positions"], st["freq"], st["qw"], st["kw"],
                                   axis=st["axis"], interleaved=c["interleaved"], eps=st["eps"])
        return rf.attn_paged(st["q"], st["kp"], st["vp"], st["table"], st["plan"], scale=st["scale"])
    return {"tables": _plain_tables, "rope": _plain_rope, "attn": _plain_attn}[c["op"]](st)


# ------------------------------------------------------------- 64-bit form --

def exact(case, seed):
    st = prepare(case, seed)
    return {"tables": _exact_tables, "rope": _exact_rope, "attn": _exact_attn}[case["op"]](st)


def _exact_tables(st):
    """Request by request, as the definition reads."""
    page, T = st["case"]["page"], st["tokens"]
    lens, news = st["lens"].tolist(), st["news"].tolist()
    table, stack = st["table"].tolist(), st["stack"].tolist()
    n = int(st["n_free"])
    width = len(table[0])
    for b, (length, new) in enumerate(zip(lens, news)):
        if new < 0:
            for i in range(_pages(length, page)):
                stack[n] = table[b][i]
                n += 1
    starts, pos, slots, lens_out, dry = [0], [], [], [], False
    for b, (length, new) in enumerate(zip(lens, news)):
        if new < 0:
            lens_out.append(0)
            starts.append(starts[-1])
            continue
        held, total = _pages(length, page), _pages(length + new, page)
        fits = total <= width
        if fits and total > held and (dry or total - held > n):
            fits, dry = False, True
        if fits:
            for i in range(held, total):
                n -= 1
                table[b][i] = stack[n]
        lens_out.append(length + new if fits else length)
        starts.append(starts[-1] + new)
        for p in range(length, length + new):
            pos.append(p)
            slots.append(table[b][p // page] * page + p % page if fits else -1)
    pos += [0] * (T - len(pos))
    slots += [-1] * (T - len(slots))
    as_int = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")       # noqa: E731
    return (as_int(starts), as_int(pos), as_int(slots), as_int(lens_out),
            torch.tensor(n, dtype=torch.int32, device="cuda"), as_int(table), as_int(stack))


def _exact_rope(st):
    c = st["case"]
    R, d = c["R"], c["D"]
    # the pair and the sign of each rotated column, then one product per column
    col = torch.arange(R, device="cuda")
    if c["interleaved"]:
        pair, other, sign = col // 2, col ^ 1, torch.where(col % 2 == 0, -1.0, 1.0)
    else:
        pair, other = col % (R // 2), (col + R // 2) % R
        sign = torch.where(col < R // 2, -1.0, 1.0)
    axis = torch.zeros(R // 2, dtype=torch.long, device="cuda") if st["axis"] is None else st["axis"].long()
    turn = st["positions"].double()[axis[pair]].T * st["freq"].double()[pair]
    cos, sin = turn.cos()[:, None], (turn.sin() * sign.double())[:, None]
    res = []
    for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        y = x.double()
        if w is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / d + st["eps"]).sqrt() * w.double()
        z = y.clone()
        z[..., :R] = y[..., :R] * cos + y[..., other] * sin
        res.append(z)
    if not c["page"]:
        return res[0], res[1]
    kp, vp = st["kp"].double(), st["vp"].double()
    rows = torch.nonzero(st["slots"] >= 0).flatten()
    flat = st["slots"][rows].long()
    at = (flat // c["page"], slice(None), flat % c["page"])
    kp[at] = res[1][rows]
    vp[at] = st["v"][rows].double()
    return res[0], kp, vp


def _exact_attn(st):
    c = st["case"]
    H, Hkv, page, window, sinks = c["H"], c["Hkv"], c["page"], c["window"], c["sinks"]
    if work(c)["flops"] > 6e12:
        return None
    T = st["q"].shape[0]
    out = torch.empty(T, H, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(T, H, dtype=torch.float64, device="cuda")
    lens, starts = st["lens"].tolist(), st["starts"].tolist()
    for b, L in enumerate(lens):
        t0, t1 = starts[b], starts[b + 1]
        flat = torch.arange(L, device="cuda")
        ids = st["table"][b][flat // page].long()
        for h in range(Hkv):
            k, v = st["kp"][ids, h, flat % page].double(), st["vp"][ids, h, flat % page].double()
            heads = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
            step = 1024
            for i in range(t0, t1, step):
                e = min(i + step, t1)
                p1 = L - (t1 - e)                      # one past the last position of these rows
                p = torch.arange(L - (t1 - i), p1, device="cuda")
                lo = max(0, int(p[0]) - window + 1) if window else 0
                keys = torch.cat([flat[:min(sinks, lo)], flat[lo:p1]])
                s = torch.einsum("thd,ld->htl", st["q"][i:e, heads].double(), k[keys]) * st["scale"]
                seen = keys <= p[:, None]
                if window:
                    seen &= (keys > p[:, None] - window) | (keys < sinks)
                s = torch.where(seen, s, -math.inf)
                z = torch.logsumexp(s, -1)
                lse[i:e, heads] = z.T
                out[i:e, heads] = torch.einsum("htl,ld->thd", torch.exp(s - z[..., None]), v[keys])
    return out, lse
