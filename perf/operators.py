"""The operators around a paged BF16 KV cache, as measured cases.

Three operators: attention of new tokens over the pages (``attend``), the
append of new tokens' keys and values with norm and rotation (``append``),
and the norm and rotation of queries and keys on their own (``rope``).
``run`` computes each in plain torch, or through the package's entry points
where ``own`` is true.
"""
import math
import random

import torch

own = False


# ---- cases ------------------------------------------------------------------

def _attend(name, heads, kv_heads, dim, page, spread, news, longest, shortest, **more):
    case = {"op": "attend", "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "spread": spread, "news": news, "longest": longest, "shortest": shortest,
            "tokens_first": True, "window": 0, "softcap": 0.0}
    case.update(more)
    return dict(case, name=name) if name else case


def _append(name, heads, kv_heads, dim, page, spread, news, longest, shortest, **more):
    case = {"op": "append", "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "spread": spread, "news": news, "longest": longest, "shortest": shortest,
            "tokens_first": True, "rotary": dim, "interleaved": False, "norm": False,
            "stretch": 1.0, "wide": False}
    case.update(more)
    return dict(case, name=name) if name else case


def _rope(name, heads, kv_heads, dim, tokens, first, **more):
    case = {"op": "rope", "heads": heads, "kv_heads": kv_heads, "dim": dim, "tokens": tokens,
            "first": first, "rotary": dim, "interleaved": False, "norm": False, "stretch": 1.0,
            "wide": False}
    case.update(more)
    return dict(case, name=name) if name else case


# "news" says how many new tokens each sequence has, as text: "1x48" is 48
# sequences of one token, parts are joined by "+".  Cached lengths (after the
# call) are spread between "shortest" and "longest" by the case's own "spread".

def listed():
    return [
        # one user, one new token, a short conversation: pure latency
        _attend("attend_token_short", 32, 8, 128, 16, 1, "1x1", 777, 777),
        # a decode server's step: a full batch of requests of every length up to 8K
        _attend("attend_tokens_batch", 32, 8, 128, 64, 2, "1x48", 8192, 130),
        # two long contexts, one token each: the cache does not fit any on-chip memory,
        # and there are few rows to spread over the chip
        _attend("attend_tokens_long", 64, 8, 128, 32, 3, "1x2", 32768, 31111),
        # a few drafted tokens a request, checked at once, under a sliding window, small heads
        _attend("attend_drafts_window", 24, 8, 64, 32, 4, "5x9", 6001, 40, window=1024,
                tokens_first=False),
        # one chunk of a long prompt over what is already cached
        _attend("attend_chunk_long", 64, 8, 128, 64, 5, "2048x1", 32768, 32768),
        # a whole 8K prompt at once
        _attend("attend_prompt", 32, 8, 128, 64, 6, "8192x1", 8192, 8192),
        # requests that decode next to two prompts that are being read; wide heads, capped scores
        _attend("attend_mixed_capped", 16, 4, 256, 16, 7, "1x24+500x1+333x1", 4096, 350,
                softcap=30.0),
        # the append of one decoded token
        _append("append_token", 32, 8, 128, 16, 8, "1x1", 777, 777),
        # a decode server's step for many requests, normed heads, stretched frequencies
        _append("append_tokens_batch", 64, 8, 128, 64, 9, "1x192", 32768, 2, norm=True,
                stretch=4.0),
        # a whole prompt goes into the cache
        _append("append_prompt", 32, 8, 128, 64, 10, "8192x1", 8192, 8192),
        # four tokens' queries and keys, far into a long context, a part of the head interleaved
        _rope("rope_tokens_far", 16, 4, 96, 4, 900001, rotary=64, interleaved=True),
        # a prompt's queries and keys from 32-bit projections, normed
        _rope("rope_prompt", 64, 8, 128, 8192, 0, norm=True, wide=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    dim = rng.choice([64, 96, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    spread = rng.randrange(1, 1 << 20)
    first = rng.random() < 0.6
    kind = rng.choice(["attend", "attend", "append", "rope"])
    half = dim // 2 if rng.random() < 0.3 else dim
    turned = {"rotary": half, "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.5,
              "stretch": rng.choice([1.0, 4.0]), "wide": rng.random() < 0.3}
    if kind == "rope":
        return _rope(None, heads, kv_heads, dim, _log(rng, 1, 4096), _log(rng, 1, 1 << 20),
                     **turned)
    shape = rng.choice(["tokens", "drafts", "chunk", "mixed"])
    if shape == "tokens":
        news, longest = "1x%d" % _log(rng, 1, 48), _log(rng, 2, 8192)
    elif shape == "drafts":
        news = "%dx%d" % (rng.randrange(2, 9), _log(rng, 1, 16))
        longest = _log(rng, 16, 8192)
    elif shape == "chunk":
        n = _log(rng, 16, 2048)
        news, longest = "%dx1" % n, max(n, _log(rng, 16, 8192))
    else:
        n = _log(rng, 16, 600)
        news, longest = "1x%d+%dx1" % (_log(rng, 1, 16), n), max(n, _log(rng, 256, 4096))
    most = max(int(p.split("x")[0]) for p in news.split("+"))
    shortest = max(most, longest // rng.choice([1, 2, 10]))
    if kind == "append":
        return _append(None, heads, kv_heads, dim, page, spread, news, longest, shortest,
                       tokens_first=first, **turned)
    return _attend(None, heads, kv_heads, dim, page, spread, news, longest, shortest,
                   tokens_first=first, window=rng.choice([0, 0, 0, _log(rng, 8, 4096)]),
                   softcap=rng.choice([0.0, 0.0, 0.0, 50.0]))


def _lengths(case):
    """(new tokens, cached tokens after the call) of each sequence."""
    rng = random.Random(case["spread"])
    got = []
    for part in case["news"].split("+"):
        new, times = (int(x) for x in part.split("x"))
        for _ in range(times):
            got.append((new, max(new, rng.randint(case["shortest"], case["longest"]))))
    if len(got) > 1 or case["shortest"] == case["longest"]:
        got[-1] = (got[-1][0], case["longest"])      # the longest is always there
    rng.shuffle(got)
    return got


def _frequencies(case):
    """Angle per position of each pair; with a stretch, the slow pairs (fewer than one turn
    in 4096 positions) go slower by it and the fast ones (more than 32 turns) stay."""
    r = case["rotary"]
    out = []
    for i in range(r // 2):
        f = 500000.0 ** (-2.0 * i / r)
        turns = 4096 * f / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1.0) / 31.0))
        out.append(f * (keep + (1.0 - keep) / case["stretch"]))
    return out


def _magnitude(case):
    return 0.1 * math.log(case["stretch"]) + 1.0


# ---- inputs -----------------------------------------------------------------

def _paged(case, lens, g, touched_from=None):
    """A pool of pages handed out in shuffled order and each sequence's row of page numbers.
    With touched_from, pages that end at or before that position are one shared page (a common
    prefix that nobody writes)."""
    T, width = case["page"], case["kv_heads"] * case["dim"]
    rows = [-(-n // T) for n in lens]
    shared = [0] * len(lens) if touched_from is None else [f // T for f in touched_from]
    count = sum(r - s for r, s in zip(rows, shared)) + 3
    order = torch.randperm(count - 1, generator=g, device="cuda") + 1
    ids = torch.zeros(len(lens), max(rows), dtype=torch.int64, device="cuda")
    at = 0
    for s, (r, skip) in enumerate(zip(rows, shared)):
        ids[s, skip:r] = order[at:at + r - skip]
        at += r - skip
    return ids, count, T * width


def _channels(case, g):
    """Per-channel sizes of a key: a KV cache's channels differ by factors of a few."""
    return torch.exp(0.5 * torch.randn(case["kv_heads"], case["dim"], generator=g, device="cuda"))


def _table(pool, ids):
    return pool.data_ptr() + ids * (pool.shape[1] * pool.element_size())


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    H, KH, D = case["heads"], case["kv_heads"], case["dim"]
    state = {"case": case}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] != "attend":
        kind = torch.float32 if case["wide"] else torch.bfloat16
        state["freq"] = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
        state["q_weight"] = 1 + 0.2 * randn(D) if case["norm"] else None
        state["k_weight"] = 1 + 0.2 * randn(D) if case["norm"] else None
    if case["op"] == "rope":
        n = case["tokens"]
        state["q"], state["k"] = randn(n, H, D).to(kind), randn(n, KH, D).to(kind)
        state["positions"] = torch.arange(n, dtype=torch.int32, device="cuda") + case["first"]
        state["q_out"] = torch.zeros(n, H, D, dtype=torch.bfloat16, device="cuda")
        state["k_out"] = torch.zeros(n, KH, D, dtype=torch.bfloat16, device="cuda")
        if own:
            state["plan"] = _plan_rope(state)
        return state

    pairs = _lengths(case)
    news, lens = [p[0] for p in pairs], [p[1] for p in pairs]
    n = sum(news)
    starts = [0]
    for x in news:
        starts.append(starts[-1] + x)
    state["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    state["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    begin = [b - a for a, b in pairs] if case["op"] == "append" else None
    state["ids"], count, words = _paged(case, lens, g, begin)
    shape = (case["page"], KH, D) if case["tokens_first"] else (KH, case["page"], D)
    size = _channels(case, g)
    size = size if case["tokens_first"] else size.unsqueeze(1)
    state["k_pool"] = torch.empty(count, words, dtype=torch.bfloat16, device="cuda")
    state["v_pool"] = torch.empty(count, words, dtype=torch.bfloat16, device="cuda")
    for at in range(0, count, 4096):
        m = min(4096, count - at)
        state["k_pool"][at:at + m] = (randn(m, *shape) * size).view(m, words).bfloat16()
        state["v_pool"][at:at + m] = randn(m, *shape).view(m, words).bfloat16()
    state["k_table"] = _table(state["k_pool"], state["ids"])
    state["v_table"] = _table(state["v_pool"], state["ids"])
    if case["op"] == "attend":
        state["q"] = randn(n, H, D).bfloat16()
        state["out"] = torch.zeros(n, H, D, dtype=torch.bfloat16, device="cuda")
        state["lse"] = torch.zeros(n, H, dtype=torch.float32, device="cuda")
        if own:
            state["plan"] = _plan_attend(state)
    else:
        state["q"], state["k"] = randn(n, H, D).to(kind), randn(n, KH, D).to(kind)
        state["v"] = randn(n, KH, D).to(kind)
        state["q_out"] = torch.zeros(n, H, D, dtype=torch.bfloat16, device="cuda")
        if own:
            state["plan"] = _plan_append(state)
    return state


# ---- the package's operators -------------------------------------------------
# The descriptions of tensors, pages and batch, and the workspace: what a
# serving loop makes once and keeps.

def _plan_cache(state):
    import lossless_bf16_kv_split_amd as sz
    case = state["case"]
    T, KH, D = case["page"], case["kv_heads"], case["dim"]
    strides = (KH * D, D) if case["tokens_first"] else (D, T * D)
    cache = sz.KVCache(state["k_table"], state["v_table"], KH, D, T, *strides)
    return cache, sz.Batch(state["starts"], state["lens"], state["q"].shape[0])


def _plan_attend(state):
    import lossless_bf16_kv_split_amd as sz
    cache, batch = _plan_cache(state)
    heads, longest = state["case"]["heads"], state["case"]["longest"]
    size = sz.sz_attend_workspace_size(heads, cache, batch, longest)
    return {"cache": cache, "batch": batch, "q": sz.Heads(state["q"]),
            "out": sz.Heads(state["out"]), "size": size,
            "workspace": torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")}


def _plan_turn(state):
    import lossless_bf16_kv_split_amd as sz
    case = state["case"]
    return sz.Rope(sz.rope_phases(_frequencies(case)).cuda(), interleaved=case["interleaved"],
                   magnitude=_magnitude(case))


def _plan_append(state):
    import lossless_bf16_kv_split_amd as sz
    cache, batch = _plan_cache(state)
    return {"cache": cache, "batch": batch, "rope": _plan_turn(state),
            **{x: sz.Heads(state[x]) for x in ("q", "k", "v", "q_out")}}


def _plan_rope(state):
    import lossless_bf16_kv_split_amd as sz
    return {"rope": _plan_turn(state),
            **{x: sz.Heads(state[x]) for x in ("q", "k", "q_out", "k_out")}}


def _run_own(state):
    import lossless_bf16_kv_split_amd as sz
    case, plan = state["case"], state["plan"]
    if case["op"] == "attend":
        sz.sz_attend_pages(plan["q"], plan["out"], state["lse"], plan["cache"], plan["batch"],
                           case["longest"], case["dim"] ** -0.5, case["softcap"], True,
                           case["window"], plan["workspace"], plan["size"])
        return {"out": state["out"], "lse": state["lse"]}
    if case["op"] == "append":
        sz.sz_kv_append(plan["k"], plan["v"], state["k_weight"], plan["q"], plan["q_out"],
                        state["q_weight"], 1e-6, plan["rope"], None, plan["cache"],
                        plan["batch"])
        return {"k": state["k_pool"], "v": state["v_pool"], "q": state["q_out"]}
    sz.sz_qk_norm_rope(plan["q"], plan["q_out"], state["q_weight"], plan["k"], plan["k_out"],
                       state["k_weight"], case["dim"], case["tokens"], state["positions"], 1e-6,
                       plan["rope"])
    return {"q": state["q_out"], "k": state["k_out"]}


# ---- the plain form -----------------------------------------------------------

def _tokens(state):
    """Sequence, index within its new tokens and cache position of every token."""
    n = state["q"].shape[0]
    t = torch.arange(n, device="cuda")
    starts = state["starts"].long()
    seq = torch.searchsorted(starts[1:], t, right=True)
    i = t - starts[seq]
    return seq, i, (state["lens"].long() - starts[1:] + starts[:-1])[seq] + i


def _gathered(state, pool):
    """The pages of each sequence as [sequence, head, position, dim] in 32 bits."""
    case = state["case"]
    T, KH, D = case["page"], case["kv_heads"], case["dim"]
    x = pool[state["ids"]]
    S, P = state["ids"].shape
    if case["tokens_first"]:
        x = x.view(S, P, T, KH, D).permute(0, 3, 1, 2, 4)
    else:
        x = x.view(S, P, KH, T, D).permute(0, 2, 1, 3, 4)
    return x.reshape(S, KH, P * T, D).float()


def _plain_attend(state):
    case = state["case"]
    H, KH, D = case["heads"], case["kv_heads"], case["dim"]
    G = H // KH
    most = max(int(p.split("x")[0]) for p in case["news"].split("+"))
    starts, lens = state["starts"].long(), state["lens"].long()
    K, V = _gathered(state, state["k_pool"]), _gathered(state, state["v_pool"])
    S, L = K.shape[0], K.shape[2]
    at = torch.arange(most, device="cuda")
    rows = (starts[:-1, None] + at).clamp(max=state["q"].shape[0] - 1)
    q = state["q"][rows].float().view(S, most, KH, G, D).permute(0, 2, 3, 1, 4)
    s = torch.matmul(q.reshape(S, KH, G * most, D), K.transpose(2, 3)) * D ** -0.5
    s = s.view(S, KH, G, most, L)
    if case["softcap"]:
        s = case["softcap"] * torch.tanh(s / case["softcap"])
    pos = (lens - starts[1:] + starts[:-1])[:, None] + at
    j = torch.arange(L, device="cuda")
    seen = (j < lens[:, None, None]) & (j <= pos[:, :, None])
    if case["window"]:
        seen = seen & (j > pos[:, :, None] - case["window"])
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.max(-1, keepdim=True).values.clamp(min=-3e38)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul((p / total.clamp(min=1e-38)).view(S, KH, G * most, L), V)
    o = o.view(S, KH, G, most, D)
    lse = (torch.log(total) + top)[..., 0]
    seq, i, _ = _tokens(state)
    return {"out": o[seq, :, :, i].reshape(-1, H, D).bfloat16(),
            "lse": lse[seq, :, :, i].reshape(-1, H)}


def _plain_turn(state, x, weight, positions):
    case = state["case"]
    R = case["rotary"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight
    angle = positions.double()[:, None, None] * state["freq"]
    cos, sin = (angle.cos() * _magnitude(case)).float(), (angle.sin() * _magnitude(case)).float()
    if case["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., R:]], -1).bfloat16()


def _plain_append(state):
    case = state["case"]
    T, KH, D = case["page"], case["kv_heads"], case["dim"]
    seq, _, pos = _tokens(state)
    page, slot = state["ids"][seq, pos // T], pos % T
    h = torch.arange(KH, device="cuda")
    step = (KH * D, D) if case["tokens_first"] else (D, T * D)
    at = (page * (T * KH * D) + slot * step[0])[:, None] + h * step[1]
    at = at[:, :, None] + torch.arange(D, device="cuda")
    state["k_pool"].view(-1)[at] = _plain_turn(state, state["k"], state["k_weight"], pos)
    state["v_pool"].view(-1)[at] = state["v"].bfloat16()
    return {"k": state["k_pool"], "v": state["v_pool"],
            "q": _plain_turn(state, state["q"], state["q_weight"], pos)}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "attend":
        return _plain_attend(state)
    if op == "append":
        return _plain_append(state)
    return {"q": _plain_turn(state, state["q"], state["q_weight"], state["positions"]),
            "k": _plain_turn(state, state["k"], state["k_weight"], state["positions"])}


# ---- bytes and operations -------------------------------------------------------

def work(case):
    H, KH, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        return {"bytes": case["tokens"] * (H + KH) * D * (6 if case["wide"] else 4),
                "flops": case["tokens"] * (H + KH) * D * (7 if case["norm"] else 3)}
    n = sum(new for new, _ in _lengths(case))
    if case["op"] == "append":
        wide = 6 if case["wide"] else 4
        return {"bytes": n * (H + 2 * KH) * D * wide,
                "flops": n * (H + KH) * D * (7 if case["norm"] else 3)}
    seen = keys = 0
    for new, length in _lengths(case):
        W = case["window"] or length + 1
        first = length - new                       # position of the first new token
        keys += length - max(0, first + 1 - W)
        below = max(0, min(new, W - first - 1))    # rows that the window does not cut
        seen += below * first + below * (below + 1) // 2 + (new - below) * W
    return {"bytes": 4 * KH * D * keys + n * H * (4 * D + 4), "flops": 4 * D * H * seen}


# ---- the definition, in 64 bits --------------------------------------------------

def _exact_attend(case, state):
    H, KH, D, T = case["heads"], case["kv_heads"], case["dim"], case["page"]
    n = state["q"].shape[0]
    out = torch.zeros(n, H, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(n, H, dtype=torch.float64, device="cuda")
    starts, lens = state["starts"].tolist(), state["lens"].tolist()
    for s, length in enumerate(lens):
        pages = state["ids"][s, :-(-length // T)].tolist()
        rows = {}
        for which in ("k_pool", "v_pool"):
            parts = []
            for page in pages:
                w = state[which][page].double()
                parts.append(w.view(T, KH, D) if case["tokens_first"]
                             else w.view(KH, T, D).transpose(0, 1))
            rows[which] = torch.cat(parts)[:length]
        for a in range(starts[s], starts[s + 1], 512):
            b = min(a + 512, starts[s + 1])
            where = torch.arange(a, b, device="cuda") - starts[s + 1] + length
            j = torch.arange(length, device="cuda")
            hidden = j[None] > where[:, None]
            if case["window"]:
                hidden |= where[:, None] - j[None] >= case["window"]
            for h in range(H):
                kv = h * KH // H
                z = state["q"][a:b, h].double() @ rows["k_pool"][:, kv].t() / math.sqrt(D)
                if case["softcap"]:
                    z = torch.tanh(z / case["softcap"]) * case["softcap"]
                z[hidden] = -math.inf
                lse[a:b, h] = torch.logsumexp(z, 1)
                out[a:b, h] = torch.softmax(z, 1) @ rows["v_pool"][:, kv]
    return {"out": out, "lse": lse}


def _exact_turn(case, x, weight, positions):
    R, m = case["rotary"], _magnitude(case)
    x = x.double().clone()
    if weight is not None:
        x /= torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6)
        x *= weight.double()
    for i, f in enumerate(_frequencies(case)):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)
        angle = positions.double() * f
        turn = torch.polar(torch.full_like(angle, m), angle)[:, None]
        z = torch.complex(x[..., a], x[..., b]) * turn
        x[..., a], x[..., b] = z.real, z.imag
    return x


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, state)
    if case["op"] == "rope":
        return {"q": _exact_turn(case, state["q"], state["q_weight"], state["positions"]),
                "k": _exact_turn(case, state["k"], state["k_weight"], state["positions"])}
    T, KH, D = case["page"], case["kv_heads"], case["dim"]
    k_pool, v_pool = state["k_pool"].double(), state["v_pool"].double()
    starts, lens = state["starts"].tolist(), state["lens"].tolist()
    where = torch.cat([torch.arange(n - (b - a), n, device="cuda")
                       for a, b, n in zip(starts, starts[1:], lens)])
    k = _exact_turn(case, state["k"], state["k_weight"], where)
    ids = state["ids"].tolist()
    for s, n in enumerate(lens):
        new = starts[s + 1] - starts[s]
        c = n - new
        while c < n:                                # one page at a time
            upto = min(n, (c // T + 1) * T)
            t = starts[s] + c - (n - new)
            page = ids[s][c // T]
            for pool, rows in ((k_pool, k), (v_pool, state["v"].double())):
                to = pool[page].view(T, KH, D) if case["tokens_first"] \
                    else pool[page].view(KH, T, D).transpose(0, 1)
                to[c % T:c % T + upto - c] = rows[t:t + upto - c]
            c = upto
    return {"k": k_pool, "v": v_pool,
            "q": _exact_turn(case, state["q"], state["q_weight"], where)}
