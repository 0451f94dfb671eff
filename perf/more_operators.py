"""Latent attention and eviction on a paged BF16 cache, as measured cases.

Five operators: the append of new tokens to a cache of latents (``append``), attention over it
in the absorbed form (``absorbed``) and over keys and values expanded from it (``expanded``);
the attention weight that each cached token has received (``weigh``) and the eviction of the
tokens with the least (``evict``).  ``run`` computes each in plain torch, or through the
package's entry points where ``own`` is true.
"""
import math
import random

import numpy as np
import torch

own = False


# ---- cases ------------------------------------------------------------------
# "news" says how many new tokens each sequence has, as text: "1x48" is 48 sequences of one
# token, parts are joined by "+".  Cached lengths (after the call) are spread between
# "shortest" and "longest" by the case's own "spread".

def _case(op, name, page, spread, news, longest, shortest, **more):
    case = {"op": op, "page": page, "spread": spread, "news": news, "longest": longest,
            "shortest": shortest}
    case.update(more)
    return dict(case, name=name) if name else case


def _append(name, heads, latent, rotary, *batch, **more):
    return _case("append", name, *batch, **dict({"heads": heads, "latent": latent,
                 "rotary": rotary, "interleaved": True, "wide": False}, **more))


def _absorbed(name, heads, latent, rotary, *batch):
    return _case("absorbed", name, *batch, heads=heads, latent=latent, rotary=rotary)


def _expanded(name, heads, dim, rotary, value, *batch):
    return _case("expanded", name, *batch, heads=heads, dim=dim, rotary=rotary, value=value)


def _weigh(name, heads, kv_heads, dim, *batch, **more):
    return _case("weigh", name, *batch, **dict({"heads": heads, "kv_heads": kv_heads, "dim": dim,
                 "window": 0, "softcap": 0.0, "keep": 1.0}, **more))


def _evict(name, kv_heads, dim, shared, budget, first, recent, *batch, **more):
    return _case("evict", name, *batch, **dict({"kv_heads": kv_heads, "dim": dim,
                 "shared": shared, "budget": budget, "first": first, "recent": recent,
                 "ties": False}, **more))


def listed():
    return [
        # a decode server's step: 40 requests' latents go into the cache, their queries turn
        _append("append_tokens", 128, 512, 64, 64, 1, "1x40", 32768, 2),
        # a prompt of 8K tokens goes into the cache, from 32-bit projections
        _append("append_prompt", 32, 512, 64, 64, 2, "8192x1", 8192, 8192, wide=True),
        # one user, one new token, a short conversation, few heads: pure latency
        _absorbed("absorbed_token_short", 16, 512, 64, 16, 3, "1x1", 901, 901),
        # a decode server's step: a batch of requests of every length up to 8K, many heads
        _absorbed("absorbed_tokens_batch", 128, 512, 64, 64, 4, "1x48", 8192, 100),
        # drafted tokens checked at once, smaller latents
        _absorbed("absorbed_drafts", 64, 384, 32, 32, 5, "3x7", 5001, 60),
        # a whole prompt of 8K tokens
        _expanded("expanded_prompt", 32, 128, 64, 128, 64, 6, "8192x1", 8192, 8192),
        # chunks of several requests' prompts behind what they have cached
        _expanded("expanded_chunks", 20, 128, 64, 128, 64, 7, "500x1+77x2+1300x1", 4099, 700),
        # one new token's weights on a short cache: latency
        _weigh("weigh_token", 32, 8, 128, 16, 8, "1x1", 777, 777),
        # a decode server's step, weights fading from step to step
        _weigh("weigh_tokens_batch", 32, 8, 128, 64, 9, "1x48", 8192, 130, keep=0.98),
        # the weights of a whole prompt, as it has been read
        _weigh("weigh_prompt", 32, 8, 128, 64, 10, "4096x1", 4096, 4096),
        # a batch of requests over their budget, each head keeping its own tokens
        _evict("evict_batch", 8, 128, False, 1024, 4, 64, 64, 11, "1x24", 8192, 1100),
        # one long context cut to a quarter, the same tokens for all heads
        _evict("evict_long", 8, 128, True, 8192, 4, 1024, 64, 12, "1x1", 32768, 32768),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    page = rng.choice([16, 32, 64, 128])
    spread = rng.randrange(1, 1 << 20)
    op = rng.choice(["append", "absorbed", "absorbed", "expanded", "weigh", "weigh", "evict"])

    def batch(most_tokens, most_len, most_seqs, shapes):
        shape = rng.choice(shapes)
        if shape == "tokens":
            news, longest = "1x%d" % _log(rng, 1, most_seqs), _log(rng, 2, most_len)
        elif shape == "drafts":
            news = "%dx%d" % (rng.randrange(2, 7), _log(rng, 1, 16))
            longest = _log(rng, 16, most_len)
        elif shape == "chunk":
            n = _log(rng, 16, most_tokens)
            news, longest = "%dx1" % n, max(n, _log(rng, 16, most_len))
        else:
            n = _log(rng, 16, 600)
            news, longest = "1x%d+%dx1" % (_log(rng, 1, 16), n), max(n, _log(rng, 256, 4096))
        most = max(int(p.split("x")[0]) for p in news.split("+"))
        shortest = max(most, longest // rng.choice([1, 2, 10]))
        return page, spread, news, longest, shortest

    every = ["tokens", "drafts", "chunk", "mixed"]
    if op in ("append", "absorbed"):
        heads = rng.choice([8, 16, 20, 32, 64, 128])
        latent, rotary = rng.choice([(512, 64), (512, 64), (384, 32), (256, 64)])
        if op == "append":
            return _append(None, heads, latent, rotary, *batch(4096, 8192, 48, every),
                           interleaved=rng.random() < 0.5, wide=rng.random() < 0.3)
        return _absorbed(None, heads, latent, rotary,
                         *batch(max(16, 4096 // heads), 8192, 48, every))
    if op == "expanded":
        dim, rotary, value = rng.choice([(128, 64, 128), (128, 64, 128), (96, 32, 96),
                                         (64, 64, 128)])
        return _expanded(None, rng.choice([4, 5, 16, 20]), dim, rotary, value,
                         *batch(2048, 8192, 4, ["chunk", "chunk", "mixed"]))
    dim = rng.choice([64, 96, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "weigh":
        return _weigh(None, kv_heads * rng.choice([1, 3, 4, 8]), kv_heads, dim,
                      *batch(1024, 8192, 48, every),
                      window=rng.choice([0, 0, 0, _log(rng, 8, 4096)]),
                      softcap=rng.choice([0.0, 0.0, 0.0, 50.0]), keep=rng.choice([0.0, 0.9, 1.0]))
    page, spread, news, longest, shortest = batch(16, 8192, 24, ["tokens"])
    budget = max(1, min(longest, _log(rng, 16, 4096)))
    first, recent = rng.choice([0, 4]), rng.choice([0, 1, 32, 128])
    first = min(first, budget)
    return _evict(None, kv_heads, dim, rng.random() < 0.4, budget, first,
                  min(recent, budget - first), page, spread, news, longest, shortest,
                  ties=rng.random() < 0.4)


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
    return [10000.0 ** (-2.0 * i / case["rotary"]) for i in range(case["rotary"] // 2)]


# ---- inputs -----------------------------------------------------------------

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pages(lens, page, g, skip=None):
    """Each sequence's row of page numbers, handed out in shuffled order (the pages before
    position skip[s] are one shared page), and the number of pages."""
    rows = [-(-n // page) for n in lens]
    shared = [0] * len(lens) if skip is None else [f // page for f in skip]
    count = sum(r - s for r, s in zip(rows, shared)) + 3
    order = torch.randperm(count - 1, generator=g, device="cuda") + 1
    ids = torch.zeros(len(lens), max(rows + [1]), dtype=torch.int64, device="cuda")
    at = 0
    for s, (r, k) in enumerate(zip(rows, shared)):
        ids[s, k:r] = order[at:at + r - k]
        at += r - k
    return ids, count


def _pool(count, width, g, size=None):
    """Pages of random words, each channel of its own size."""
    pool = torch.empty(count, width, dtype=torch.bfloat16, device="cuda")
    for at in range(0, count, 4096):
        x = torch.randn(min(4096, count - at), width, generator=g, device="cuda")
        if size is not None:
            x = (x.view(x.shape[0], -1, size.numel()) * size.reshape(-1)).view(x.shape)
        pool[at:at + x.shape[0]] = x.bfloat16()
    return pool


def _table(pool, ids):
    return pool.data_ptr() + ids * (pool.shape[1] * pool.element_size())


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    pairs = _lengths(case)
    news, lens = [p[0] for p in pairs], [p[1] for p in pairs]
    n, T = sum(news), case["page"]
    starts = [0]
    for x in news:
        starts.append(starts[-1] + x)
    most = max(lens)
    state = {"case": case, "starts": _i32(starts), "lens": _i32(lens), "most": most}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if op == "append":
        H, L, R = case["heads"], case["latent"], case["rotary"]
        kind = torch.float32 if case["wide"] else torch.bfloat16
        state["ids"], count = _pages(lens, T, g, [b - a for a, b in pairs])
        state["pool"] = _pool(count, T * (L + R), g)
        state["freq"] = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
        state["weight"] = 1 + 0.2 * randn(L)
        state["kv"] = randn(n, 1, L + R).to(kind)        # one projection gives both parts
        # the queries as the attention takes them: behind their latent part
        state["q"] = randn(n, H, R).to(kind)
        state["q_out"] = torch.zeros(n, H, R, dtype=torch.bfloat16, device="cuda")
    elif op == "absorbed":
        H, L, R = case["heads"], case["latent"], case["rotary"]
        state["ids"], count = _pages(lens, T, g)
        state["pool"] = _pool(count, T * (L + R), g)
        state["q"] = randn(n, H, L + R).bfloat16()
        state["out"] = torch.zeros(n, H, L, dtype=torch.bfloat16, device="cuda")
        state["lse"] = torch.zeros(n, H, device="cuda")
    elif op == "expanded":
        H, D, R, V = case["heads"], case["dim"], case["rotary"], case["value"]
        at = [0]
        for x in lens:
            at.append(at[-1] + x)
        state["key_starts"] = _i32(at[:-1])
        state["q"] = randn(n, H, D + R).bfloat16()
        # keys and values as one projection leaves them, beside each other in every head; the
        # rotary part at the end of the latent rows
        kv = randn(at[-1], H, D + V).bfloat16()
        rows = randn(at[-1], 1, 4 * D + R).bfloat16()
        state["k"], state["v"], state["r"] = kv[..., :D], kv[..., D:], rows[..., 4 * D:]
        state["out"] = torch.zeros(n, H, V, dtype=torch.bfloat16, device="cuda")
        state["lse"] = torch.zeros(n, H, device="cuda")
    elif op == "weigh":
        H, KH, D = case["heads"], case["kv_heads"], case["dim"]
        state["ids"], count = _pages(lens, T, g)
        size = torch.exp(0.5 * randn(KH * D))            # a cache's channels differ in size
        state["k_pool"] = _pool(count, T * KH * D, g, size)
        state["q"] = randn(n, H, D).bfloat16()
        state["before"] = -torch.log(torch.rand(len(lens), KH, most, generator=g,
                                                device="cuda").clamp(min=1e-6))
        state["weights"] = torch.zeros_like(state["before"])
        # the log-sums that attention left
        state["lse"] = torch.empty(n, H, device="cuda")
        for s, rows, kv, z in _scores(state):
            state["lse"][rows, kv * (H // KH):(kv + 1) * (H // KH)] = torch.logsumexp(z, -1).t()
    else:
        KH, D, B = case["kv_heads"], case["dim"], case["budget"]
        WH = 1 if case["shared"] else KH
        kept = [min(x, B) for x in lens]
        state["ids"], count = _pages(lens, T, g)
        state["to_ids"], to_count = _pages(kept, T, g)
        state["k_pool"] = _pool(count, T * KH * D, g)
        state["v_pool"] = _pool(count, T * KH * D, g)
        state["k_to"] = torch.zeros(to_count, T * KH * D, dtype=torch.bfloat16, device="cuda")
        state["v_to"] = torch.zeros_like(state["k_to"])
        # few tokens hold most of the weight; some have received none
        w = torch.rand(len(lens), WH, most, generator=g, device="cuda")
        w = (0.05 / w.clamp(min=1e-4)) * (w < 0.95)
        state["weights"] = (w * 16).round() / 16 if case["ties"] else w
        state["weights_to"] = torch.zeros(len(lens), WH, B, device="cuda")
        state["kept"] = torch.zeros(len(lens), WH, B, dtype=torch.int32, device="cuda")
        state["lens_to"] = torch.zeros_like(state["lens"])
    if own:
        state["plan"] = _plan(state)
    return state


# ---- the package's operators -------------------------------------------------
# The descriptions of tensors, pages and batch, and the workspace: what a serving loop makes
# once and keeps.

def _plan(state):
    import lossless_bf16_kv_split_amd as sz
    case, plan = state["case"], {}
    op, T = case["op"], case["page"]
    if op == "evict":
        def cache(k, v, ids):
            return sz.KVCache(_table(k, ids), _table(v, ids), case["kv_heads"], case["dim"], T,
                              keep=(k, v))
        return {"from": cache(state["k_pool"], state["v_pool"], state["ids"]),
                "to": cache(state["k_to"], state["v_to"], state["to_ids"])}
    n, most = state["q"].shape[0], state["most"]
    plan["batch"] = sz.Batch(state["starts"], state["lens"], n)
    plan["q"] = sz.Heads(state["q"])
    size = 0
    if op in ("append", "absorbed"):
        plan["cache"] = sz.LatentCache(_table(state["pool"], state["ids"]), case["latent"],
                                       case["rotary"], T, keep=state["pool"])
    if op == "append":
        plan["rope"] = sz.Rope(sz.rope_phases(_frequencies(case)).cuda(),
                               interleaved=case["interleaved"])
        plan["latent"] = sz.Heads(state["kv"][..., :case["latent"]])
        plan["k"] = sz.Heads(state["kv"][..., case["latent"]:])
        plan["q_out"] = sz.Heads(state["q_out"])
    elif op == "absorbed":
        plan["out"] = sz.Heads(state["out"])
        size = sz.sz_attend_latent_workspace_size(case["heads"], plan["cache"], plan["batch"],
                                                  most)
    elif op == "expanded":
        for x in ("k", "r", "v", "out"):
            plan[x] = sz.Heads(state[x])
        size = sz.sz_attend_expanded_workspace_size(case["heads"], case["value"], plan["batch"],
                                                    most)
    else:
        table = _table(state["k_pool"], state["ids"])
        plan["cache"] = sz.KVCache(table, table, case["kv_heads"], case["dim"], T,
                                   keep=state["k_pool"])
        size = sz.sz_weigh_workspace_size(case["heads"], plan["cache"], plan["batch"], most)
    plan["size"] = size
    plan["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    return plan


def _run_own(state):
    import lossless_bf16_kv_split_amd as sz
    case, plan = state["case"], state["plan"]
    op = case["op"]
    if op == "append":
        sz.sz_latent_append(plan["latent"], state["weight"], 1e-6, plan["k"], plan["q"],
                            plan["q_out"], plan["rope"], None, plan["cache"], plan["batch"])
        return {"pool": state["pool"], "q": state["q_out"]}
    if op == "absorbed":
        sz.sz_attend_latent(plan["q"], plan["out"], state["lse"], plan["cache"], plan["batch"],
                            state["most"], _scale(case), True, plan["workspace"], plan["size"])
        return {"out": state["out"], "lse": state["lse"]}
    if op == "expanded":
        sz.sz_attend_expanded(plan["q"], plan["out"], state["lse"], plan["k"], plan["r"],
                              plan["v"], state["key_starts"], plan["batch"], state["most"],
                              _scale(case), True, plan["workspace"], plan["size"])
        return {"out": state["out"], "lse": state["lse"]}
    if op == "weigh":
        sz.sz_weigh_pages(plan["q"], state["lse"], state["before"], state["weights"],
                          state["most"], case["keep"], plan["cache"], plan["batch"],
                          state["most"], _scale(case), case["softcap"], True, case["window"],
                          plan["workspace"], plan["size"])
        return state["weights"]
    sz.sz_evict_pages(state["weights"], state["weights_to"], plan["from"], plan["to"],
                      state["lens"], state["lens_to"], state["most"], case["budget"],
                      case["first"], case["recent"], state["kept"])
    return {x: state[x] for x in ("k_to", "v_to", "weights_to", "kept", "lens_to")}


# ---- the plain form -----------------------------------------------------------

def _scale(case):
    if case["op"] == "weigh":
        return case["dim"] ** -0.5
    return (128 + case["rotary"]) ** -0.5                # of the heads before they are absorbed


def _tokens(state):
    """Sequence, index within its new tokens and cache position of every token."""
    starts = state["starts"].long()
    t = torch.arange(state["q"].shape[0], device="cuda")
    seq = torch.searchsorted(starts[1:], t, right=True)
    i = t - starts[seq]
    return seq, i, (state["lens"].long() - starts[1:] + starts[:-1])[seq] + i


def _turned(case, x, freq, positions):
    angle = positions.double()[:, None, None] * freq
    cos, sin = angle.cos().float(), angle.sin().float()
    x, R = x.float(), case["rotary"]
    if case["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :R // 2], x[..., R // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(state):
    case = state["case"]
    T, L, W = case["page"], case["latent"], case["latent"] + case["rotary"]
    seq, _, pos = _tokens(state)
    c = state["kv"][..., :L].float()
    c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + 1e-6) * state["weight"]
    r = _turned(case, state["kv"][..., L:], state["freq"], pos)
    pool = state["pool"].view(-1, W)
    pool[state["ids"][seq, pos // T] * T + pos % T] = torch.cat([c, r], -1)[:, 0].bfloat16()
    return {"pool": state["pool"],
            "q": _turned(case, state["q"], state["freq"], pos).bfloat16()}


def _attention(q, K, V, first, scale):
    """q [heads, rows, D], K [heads or 1, keys, D], V likewise; row i sees keys up to first + i."""
    s = torch.matmul(q, K.transpose(1, 2)) * scale
    j = torch.arange(K.shape[1], device="cuda")
    i = torch.arange(q.shape[1], device="cuda") + first
    s.masked_fill_(j > i[:, None], -math.inf)
    top = s.max(-1, keepdim=True).values
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p / total, V), (torch.log(total) + top)[..., 0]


def _plain_rows(state, K, V):
    """Attention sequence by sequence, where the keys of one are a tensor of their own."""
    starts, lens = state["starts"].tolist(), state["lens"].tolist()
    outs, lses = [], []
    for s, length in enumerate(lens):
        q = state["q"][starts[s]:starts[s + 1]].float().transpose(0, 1)
        heads = max(1, (1 << 29) // max(1, q.shape[1] * length))
        k, v, first = K(s), V(s), length - q.shape[1]
        parts = [_attention(q[h:h + heads], k if k.shape[0] == 1 else k[h:h + heads],
                            v if v.shape[0] == 1 else v[h:h + heads], first, _scale(state["case"]))
                 for h in range(0, q.shape[0], heads)]
        outs.append(torch.cat([p[0] for p in parts]).transpose(0, 1))
        lses.append(torch.cat([p[1] for p in parts]).t())
    return {"out": torch.cat(outs).bfloat16(), "lse": torch.cat(lses)}


def _plain_absorbed(state):
    case = state["case"]
    T, W, L = case["page"], case["latent"] + case["rotary"], case["latent"]
    lens = state["lens"].tolist()
    if case["news"].split("+")[0].startswith("1x") and "+" not in case["news"]:
        # one token each: all sequences at once
        c = state["pool"][state["ids"]].view(len(lens), -1, W).float()
        s = torch.matmul(state["q"].float(), c.transpose(1, 2)) * _scale(case)
        j = torch.arange(c.shape[1], device="cuda")
        s.masked_fill_(j >= state["lens"][:, None, None], -math.inf)
        top = s.max(-1, keepdim=True).values
        p = torch.exp(s - top)
        total = p.sum(-1, keepdim=True)
        return {"out": torch.matmul(p / total, c[..., :L]).bfloat16(),
                "lse": (torch.log(total) + top)[..., 0]}

    rows = {}

    def keys(s):
        pages = state["ids"][s, :-(-lens[s] // T)]
        rows[s] = state["pool"][pages].view(1, -1, W)[:, :lens[s]].float()
        return rows[s]
    return _plain_rows(state, keys, lambda s: rows.pop(s)[..., :L])


def _plain_expanded(state):
    lens, at = state["lens"].tolist(), state["key_starts"].tolist()
    H = state["case"]["heads"]

    def keys(s):
        k, r = (state[x][at[s]:at[s] + lens[s]].float() for x in ("k", "r"))
        return torch.cat([k, r.expand(-1, H, -1)], -1).transpose(0, 1)
    return _plain_rows(state, keys,
                       lambda s: state["v"][at[s]:at[s] + lens[s]].float().transpose(0, 1))


def _scores(state):
    """(sequence, its tokens' rows, KV head, scores [heads of the group, rows, keys]), hidden
    ones at -infinity, in pieces of bounded size."""
    case = state["case"]
    T, H, KH, D = case["page"], case["heads"], case["kv_heads"], case["dim"]
    G = H // KH
    starts, lens = state["starts"].tolist(), state["lens"].tolist()
    for s, length in enumerate(lens):
        pages = state["ids"][s, :-(-length // T)]
        K = state["k_pool"][pages].view(-1, KH, D)[:length].float().transpose(0, 1)
        j = torch.arange(length, device="cuda")
        step = max(1, (1 << 28) // (G * length))
        for a in range(starts[s], starts[s + 1], step):
            b = min(a + step, starts[s + 1])
            i = torch.arange(a, b, device="cuda")[:, None] - starts[s + 1] + length
            hidden = j > i
            if case["window"]:
                hidden = hidden | (j <= i - case["window"])
            for kv in range(KH):
                q = state["q"][a:b, kv * G:(kv + 1) * G].float().transpose(0, 1)
                z = torch.matmul(q, K[kv].t()) * D ** -0.5
                if case["softcap"]:
                    z = case["softcap"] * torch.tanh(z / case["softcap"])
                yield s, slice(a, b), kv, z.masked_fill_(hidden, -math.inf)


def _plain_weigh(state):
    case = state["case"]
    H, KH, D, T = case["heads"], case["kv_heads"], case["dim"], case["page"]
    G = H // KH
    w = state["weights"]
    starts, lens = state["starts"].long(), state["lens"].long()
    j = torch.arange(w.shape[2], device="cuda")
    old = j < (lens - starts[1:] + starts[:-1])[:, None, None]
    here = (j < lens[:, None, None]).expand_as(w)
    base = torch.where(old, state["before"] * case["keep"], 0.0)
    if case["news"].split("+")[0].startswith("1x") and "+" not in case["news"]:
        # one token each: all sequences at once
        K = state["k_pool"][state["ids"]].view(len(lens), -1, KH, D)[:, :w.shape[2]].float()
        q = state["q"].float().view(-1, KH, G, D)
        z = torch.matmul(q, K.permute(0, 2, 3, 1)) * D ** -0.5
        if case["softcap"]:
            z = case["softcap"] * torch.tanh(z / case["softcap"])
        seen = j < lens[:, None, None]
        if case["window"]:
            seen = seen & (j >= lens[:, None, None] - case["window"])
        z.masked_fill_(~seen[:, :, None], -math.inf)
        total = torch.exp(z - state["lse"].view(-1, KH, G, 1)).sum(2) + base
        return torch.where(here, total, w)
    total = base
    for s, rows, kv, z in _scores(state):
        p = torch.exp(z - state["lse"][rows, kv * G:(kv + 1) * G].t()[:, :, None])
        total[s, kv, :p.shape[2]] += p.sum((0, 1))
    return torch.where(here, total, w)


def _plain_evict(state):
    case = state["case"]
    T, KH, D, B = case["page"], case["kv_heads"], case["dim"], case["budget"]
    w, lens = state["weights"], state["lens"].long()
    S, WH, M = w.shape
    j = torch.arange(M, device="cuda")
    n = lens[:, None, None]
    rank = w.masked_fill((j < case["first"]) | (j >= n - case["recent"]), math.inf)
    rank = rank.masked_fill(j >= n, -math.inf)
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :B]
    best = torch.where(torch.arange(best.shape[2], device="cuda") < n, best, M)
    kept = torch.sort(best, -1).values
    kept = torch.nn.functional.pad(kept, (0, B - kept.shape[2]), value=M)
    there = kept < M
    at = kept.clamp(max=M - 1)
    state["kept"] = torch.where(there, kept, -1).int()
    state["weights_to"] = torch.where(there, torch.gather(w, 2, at), state["weights_to"])
    state["lens_to"] = lens.clamp(max=B).int()
    head = torch.arange(KH, device="cuda")
    for s in range(S):
        m = int(state["lens_to"][s])
        src = at[s, :, :m].t().expand(-1, KH)
        row = state["ids"][s][src // T] * T + src % T
        dst = torch.arange(m, device="cuda")
        to = state["to_ids"][s][dst // T] * T + dst % T
        for a, b in (("k_pool", "k_to"), ("v_pool", "v_to")):
            state[b].view(-1, KH, D)[to] = state[a].view(-1, KH, D)[row, head]
    return {x: state[x] for x in ("k_to", "v_to", "weights_to", "kept", "lens_to")}


def run(state):
    if own:
        return _run_own(state)
    return {"append": _plain_append, "absorbed": _plain_absorbed, "expanded": _plain_expanded,
            "weigh": _plain_weigh, "evict": _plain_evict}[state["case"]["op"]](state)


# ---- bytes and operations -------------------------------------------------------

def work(case):
    pairs, op = _lengths(case), case["op"]
    n, keys = sum(a for a, _ in pairs), sum(b for _, b in pairs)
    seen = sum(a * (b - a) + a * (a + 1) // 2 for a, b in pairs)
    if op == "append":
        H, L, R = case["heads"], case["latent"], case["rotary"]
        return {"bytes": n * (L + R + H * R) * (6 if case["wide"] else 4),
                "flops": n * (4 * L + 3 * R * (H + 1))}
    if op == "absorbed":
        H, L, R = case["heads"], case["latent"], case["rotary"]
        return {"bytes": 2 * (L + R) * keys + n * H * (2 * (2 * L + R) + 4),
                "flops": 2 * H * (2 * L + R) * seen}
    if op == "expanded":
        H, D, R, V = case["heads"], case["dim"], case["rotary"], case["value"]
        return {"bytes": 2 * keys * (H * (D + V) + R) + n * H * (2 * (D + R + V) + 4),
                "flops": 2 * H * (D + R + V) * seen}
    if op == "weigh":
        H, KH, D, W = case["heads"], case["kv_heads"], case["dim"], case["window"]
        if W:
            seen = keys = 0
            for a, b in pairs:
                first = b - a
                keys += b - max(0, first + 1 - W)
                below = max(0, min(a, W - first - 1))    # rows that the window does not cut
                seen += below * first + below * (below + 1) // 2 + (a - below) * W
        weights = sum(b for _, b in pairs) * KH * (8 if case["keep"] else 4)
        return {"bytes": 2 * KH * D * keys + n * H * (2 * D + 4) + weights,
                "flops": 2 * H * D * seen}
    KH, D = case["kv_heads"], case["dim"]
    WH = 1 if case["shared"] else KH
    kept = sum(min(b, case["budget"]) for _, b in pairs)
    return {"bytes": 8 * KH * D * kept + WH * (4 * keys + 8 * kept), "flops": WH * keys}


# ---- the definition, in 64 bits --------------------------------------------------

def _rows(case, pool, ids, length, width):
    """The first `length` rows of a sequence, from its pages."""
    T = case["page"]
    return torch.cat([pool[p].double().view(T, width) for p in ids[:-(-length // T)]])[:length]


def _exact_turn(case, x, positions):
    R, x = case["rotary"], x.double().clone()
    for i, f in enumerate(_frequencies(case)):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)
        angle = positions.double() * f
        z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(angle), angle)[:, None]
        x[..., a], x[..., b] = z.real, z.imag
    return x


def _exact_attend(case, state, keys_of, values_of, width):
    n, H = state["q"].shape[:2]
    out = torch.zeros(n, H, width, dtype=torch.float64, device="cuda")
    lse = torch.zeros(n, H, dtype=torch.float64, device="cuda")
    starts, lens = state["starts"].tolist(), state["lens"].tolist()
    for s, length in enumerate(lens):
        for h in range(H):
            k, v = keys_of(s, h), values_of(s, h)
            for a in range(starts[s], starts[s + 1], 2048):
                b = min(a + 2048, starts[s + 1])
                at = torch.arange(a, b, device="cuda") + (length - starts[s + 1])
                z = state["q"][a:b, h].double() @ k.t() * _scale(case)
                z[torch.arange(length, device="cuda")[None] > at[:, None]] = -math.inf
                lse[a:b, h] = torch.logsumexp(z, 1)
                out[a:b, h] = torch.softmax(z, 1) @ v
    return {"out": out, "lse": lse}


def _exact_weigh(case, state):
    H, KH, D, W = case["heads"], case["kv_heads"], case["dim"], case["window"]
    out = state["weights"].double()
    starts, lens, ids = (state[x].tolist() for x in ("starts", "lens", "ids"))
    for s, length in enumerate(lens):
        K = _rows(case, state["k_pool"], ids[s], length, KH * D).view(length, KH, D)
        new = starts[s + 1] - starts[s]
        out[s, :, :length] = state["before"][s, :, :length].double() * case["keep"]
        out[s, :, length - new:length] = 0
        j = torch.arange(length, device="cuda")[None]
        for a in range(starts[s], starts[s + 1], 2048):
            b = min(a + 2048, starts[s + 1])
            at = (torch.arange(a, b, device="cuda") + (length - starts[s + 1]))[:, None]
            seen = (j <= at) & ((at - j < W) if W else (j >= 0))
            for h in range(H):
                kv = h * KH // H
                z = state["q"][a:b, h].double() @ K[:, kv].t() / math.sqrt(D)
                if case["softcap"]:
                    z = torch.tanh(z / case["softcap"]) * case["softcap"]
                p = torch.exp(z - state["lse"][a:b, h].double()[:, None])
                out[s, kv, :length] += (p * seen).sum(0)
    return out


def _exact_evict(case, state):
    T, KH, D, B = case["page"], case["kv_heads"], case["dim"], case["budget"]
    w, lens = state["weights"].cpu().numpy(), state["lens"].tolist()
    S, WH, _ = w.shape
    kept = np.full((S, WH, B), -1, np.int32)
    weights = np.zeros((S, WH, B), np.float64)
    to = {x: state[x].double() for x in ("k_to", "v_to")}
    ids, to_ids = state["ids"].tolist(), state["to_ids"].tolist()
    for s, n in enumerate(lens):
        rows = {x: _rows(case, state[x], ids[s], n, KH * D).view(n, KH, D)
                for x in ("k_pool", "v_pool")}
        m = min(n, B)
        for h in range(WH):
            j = np.arange(n)
            safe = (j < case["first"]) | (j >= n - case["recent"])
            order = np.lexsort((j, -w[s, h, :n], ~safe))[:m]
            chosen = np.sort(order)
            kept[s, h, :m] = chosen
            weights[s, h, :m] = w[s, h, chosen]
        for a, b in (("k_pool", "k_to"), ("v_pool", "v_to")):
            for h in range(KH):
                pick = torch.from_numpy(kept[s, h % WH, :m].astype(np.int64)).cuda()
                got = rows[a][pick, h]
                for c in range(0, m, T):
                    page = to[b][to_ids[s][c // T]].view(T, KH, D)
                    page[:min(T, m - c), h] = got[c:c + T]
    return {"k_to": to["k_to"], "v_to": to["v_to"],
            "weights_to": torch.from_numpy(weights).cuda(), "kept": torch.from_numpy(kept).cuda(),
            "lens_to": state["lens"].clamp(max=B)}


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "weigh":
        return _exact_weigh(case, state)
    if op == "evict":
        return _exact_evict(case, state)
    lens = state["lens"].tolist()
    if op == "absorbed":
        L, ids = case["latent"], state["ids"].tolist()
        rows = {}

        def keys(s, h):
            if s not in rows:
                rows.clear()
                rows[s] = _rows(case, state["pool"], ids[s], lens[s], L + case["rotary"])
            return rows[s]
        return _exact_attend(case, state, keys, lambda s, h: rows[s][:, :L], L)
    if op == "expanded":
        at = state["key_starts"].tolist()
        return _exact_attend(
            case, state,
            lambda s, h: torch.cat([state["k"][at[s]:at[s] + lens[s], h],
                                    state["r"][at[s]:at[s] + lens[s], 0]], -1).double(),
            lambda s, h: state["v"][at[s]:at[s] + lens[s], h].double(), case["value"])
    T, L, W = case["page"], case["latent"], case["latent"] + case["rotary"]
    starts, ids = state["starts"].tolist(), state["ids"].tolist()
    where = torch.cat([torch.arange(n - (b - a), n, device="cuda")
                       for a, b, n in zip(starts, starts[1:], lens)])
    c = state["kv"][..., :L].double()
    c = c / torch.sqrt(c.pow(2).sum(-1, keepdim=True) / L + 1e-6) * state["weight"].double()
    new = torch.cat([c, _exact_turn(case, state["kv"][..., L:], where)], -1)[:, 0]
    pool = state["pool"].double()
    for s, n in enumerate(lens):
        at = n - (starts[s + 1] - starts[s])
        t = starts[s]
        while at < n:                                    # one page at a time
            upto = min(n, (at // T + 1) * T)
            pool[ids[s][at // T]].view(T, W)[at % T:at % T + upto - at] = new[t:t + upto - at]
            t += upto - at
            at = upto
    return {"pool": pool, "q": _exact_turn(case, state["q"], where)}
