"""Attention weights of cached tokens (sz_weigh_pages) and eviction by them
(sz_evict_pages) against plain 64-bit forms, at the sizes, layouts and masks
where they can go wrong."""
import math
import sys

import pytest

import kv_reference as ref
from test_gpu_kv import SHAPES, TOKENS, Setup

pytestmark = pytest.mark.gpu
SENTINEL = 768.0


def say(*a):
    print("[gpu-evict]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a ROCm device"
    t.cuda.set_device(0)
    return t


@pytest.fixture(scope="module")
def sz(torch):
    import lossless_bf16_kv_split_amd as m
    return m


# ---- weights ---------------------------------------------------------------

def weights_of(q, lse, keys, length, scale, causal=True, window=0, softcap=0.0):
    """sum over rows of exp(score - lse) for q [new, H, D], lse [new, H] and
    keys [length, KH, D]: [KH, length], and a bound of the error.  A score is
    off by D U32 sum|q k| (an FP32 sum of exact products in any order), its
    scaling, log2 e times the log-sum and their difference by 4 U32 of each of
    their sizes; a cap's score by 16 U32 of its own size (kv_reference.py).  The
    exponential is off by 2^-20 of itself, and n additions by n U32 of the
    sum."""
    new, H, D = q.shape
    KH = keys.shape[1]
    G = H // KH
    c = (length - new + torch_().arange(new))[:, None]
    j = torch_().arange(length)[None]
    seen = (j <= c) if causal else (j < length).expand(new, length)
    if window:
        seen = seen & (j > c - window)
    w = torch_().zeros(KH, length, dtype=torch_().float64)
    tol = torch_().zeros_like(w)
    for h in range(H):
        x, K = q[:, h].double(), keys[:, h // G].double()
        z = lse[:, h].double()[:, None]
        s = (x @ K.t()) * scale
        size = (x.abs() @ K.abs().t()) * scale
        ds = D * ref.U32 * size + 4 * ref.U32 * size
        if softcap:
            s = softcap * torch_().tanh(s / softcap)
            ds = ds + 16 * ref.U32 * s.abs()
        ds = ds + 4 * ref.U32 * (s.abs() + z.abs().clamp(max=1e30))
        p = torch_().where(seen & (z > -math.inf), torch_().exp(s - z), 0.0)
        w[h // G] += p.sum(0)
        tol[h // G] += (p * (2 * ds + 2.0 ** -20)).masked_fill(~seen, 0).sum(0)
    return w, tol + (G * new + 64) * ref.U32 * w


def torch_():
    import torch
    return torch


def weigh(torch, sz, S, lse, before, keep=1.0, max_len=0, pitch=None, cache=None, batch=None,
          scale=None, **kw):
    cache, batch = cache or S.cache, batch or S.batch
    KH = S.shape[1]
    pitch = pitch or S.width * S.page
    out = torch.full((len(S.pairs), KH, pitch), SENTINEL, device="cuda")
    size = sz.sz_weigh_workspace_size(S.q.shape[1], cache, batch, max_len)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    status = torch.full((len(S.pairs),), -1, dtype=torch.int32, device="cuda")
    sz.sz_weigh_pages(S.q.cuda(), lse, before, out, pitch, keep, cache, batch, max_len,
                      S.dim ** -0.5 if scale is None else scale,
                      workspace=ws if size else None, workspace_bytes=size, d_status=status, **kw)
    torch.cuda.synchronize()
    assert bool((ws[size:] == 0xFF).all())
    return out, status.tolist(), size


def check_weigh(torch, sz, S, label, keep=1.0, pitch=None, max_len=0, with_before=True, lse=None,
                **kw):
    say(label)
    pitch = pitch or S.width * S.page
    if lse is None:
        _, lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch, **kw)
    before = None
    if with_before:
        before = S.rand(len(S.pairs), S.shape[1], pitch).abs()
        for s, (new, n) in enumerate(S.pairs):   # what a new token's place held before
            before[s, :, max(0, n - new):] = math.nan
    out, status, size = weigh(torch, sz, S, lse, None if before is None else before.cuda(), keep,
                              max_len, pitch, **kw)
    assert status == [0] * len(S.pairs), label
    out, lse = out.cpu().double(), lse.cpu()
    for s, (new, n) in enumerate(S.pairs):
        a, b = S.starts[s], S.starts[s + 1]
        want, tol = weights_of(S.q[a:b], lse[a:b], S.rows(S.k, s), n, S.dim ** -0.5, **kw)
        if before is not None:
            old = max(0, n - new)
            part = before[s, :, :old].double() * keep
            want[:, :old] += part
            tol[:, :old] += 2 * ref.U32 * (part.abs() + want[:, :old])
        bad = ~((out[s, :, :n] - want).abs() <= tol)
        assert not bool(bad.any()), (label, s, bad.nonzero()[0].tolist(),
                                     float((out[s, :, :n] - want).abs().max()))
        assert bool((out[s, :, n:] == SENTINEL).all()), (label, s)
    return size


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_weigh_single_tokens(torch, sz, shape):
    S = Setup(torch, sz, TOKENS, *shape, seed=1, before=2, behind=3)
    check_weigh(torch, sz, S, f"single {shape}", keep=0.5)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("tokens_first", [True, False])
def test_weigh_chunks(torch, sz, shape, tokens_first):
    pairs = [(3, 3), (1, 70), (0, 40), (17, 50), (64, 64), (0, 0), (33, 200), (130, 331)]
    S = Setup(torch, sz, pairs, *shape, tokens_first=tokens_first, seed=2, behind=5)
    check_weigh(torch, sz, S, f"chunks {shape} {tokens_first}", keep=0.98)


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[1], SHAPES[3], SHAPES[7]], ids=str)
@pytest.mark.parametrize("kw", [dict(causal=False), dict(window=1), dict(window=16),
                                dict(window=37), dict(window=64), dict(window=4096),
                                dict(softcap=5.0), dict(softcap=30.0, window=50)], ids=str)
def test_weigh_masks(torch, sz, shape, kw):
    pairs = [(1, 90), (5, 5), (70, 150), (2, 300), (1, 1), (1, 64), (1, 65), (200, 520)]
    S = Setup(torch, sz, pairs, *shape, seed=3)
    check_weigh(torch, sz, S, f"masks {shape} {kw}", **kw)


def test_weigh_rows_that_see_nothing(torch, sz):
    pairs = [(5, 2), (3, 0), (1, 0), (40, 20), (0, 9)]
    for shape in (SHAPES[0], SHAPES[3]):
        S = Setup(torch, sz, pairs, *shape, seed=4)
        check_weigh(torch, sz, S, f"empty {shape}")
        check_weigh(torch, sz, S, f"empty window {shape}", window=3)
    check_weigh(torch, sz, S, "empty, not causal", causal=False)


@pytest.mark.parametrize("pairs,max_len", [
    ([(1, 5000)], 0), ([(1, 70), (1, 9000), (1, 2049)], 0), ([(20, 6000), (1, 33)], 0),
    ([(1500, 1600)], 1616), ([(700, 3333)], 0), ([(2048, 2048), (1, 900)], 0),
], ids=str)
@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[3], (16, 1, 64, 16), (2, 1, 128, 16)], ids=str)
@pytest.mark.parametrize("window", [0, 600])
def test_weigh_long(torch, sz, pairs, max_len, shape, window):
    S = Setup(torch, sz, pairs, *shape, seed=5)
    check_weigh(torch, sz, S, f"long {pairs} {shape}", max_len=max_len, window=window)


def test_weigh_shares_rows_among_workgroups(torch, sz):
    """Many rows on few keys of few heads: several workgroups a tile, joined
    through the workspace; the same result whatever it held."""
    S = Setup(torch, sz, [(1200, 1300), (5, 700)], 8, 1, 128, 16, seed=6)
    assert check_weigh(torch, sz, S, "shared", max_len=1310) > 0
    assert check_weigh(torch, sz, S, "shared, window", max_len=1310, window=100) > 0


@pytest.mark.parametrize("n", [65, 700])
def test_weigh_many_sequences(torch, sz, n):
    pairs = [((i * 7) % 3 and 1 + (i % 11 == 5), 2 + (i * 37) % 90) for i in range(n)]
    pairs[n // 2] = (2, 4000)
    S = Setup(torch, sz, pairs, 4, 1, 64, 16, seed=17, behind=1)
    check_weigh(torch, sz, S, f"many {n}")


def test_weigh_before_and_in_place(torch, sz):
    """Without `before`, with a factor of 0 (not read: NaN there), in place,
    and with wider rows than the lengths need."""
    pairs = [(1, 300), (9, 500), (200, 200)]
    S = Setup(torch, sz, pairs, 16, 4, 128, 16, seed=7)
    check_weigh(torch, sz, S, "none", with_before=False)
    check_weigh(torch, sz, S, "pitch", pitch=777)
    _, lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch)
    none, _, _ = weigh(torch, sz, S, lse, None)
    zero, _, _ = weigh(torch, sz, S, lse, torch.full_like(none, math.nan), keep=0.0)
    assert torch.equal(none, zero)
    before = torch.rand(none.shape, device="cuda")
    apart, _, _ = weigh(torch, sz, S, lse, before, keep=0.9)
    inplace = before.clone()
    sz.weigh_pages(S.q.cuda(), lse, S.cache, S.batch, inplace, keep=0.9)
    for s, (_, n) in enumerate(pairs):
        assert torch.equal(inplace[s, :, :n], apart[s, :, :n])
        assert torch.equal(inplace[s, :, n:], before[s, :, n:])
    fresh = sz.weigh_pages(S.q.cuda(), lse, S.cache, S.batch, max_len=500)
    assert fresh.shape == (3, 4, 500) and torch.equal(fresh[1], none[1, :, :500])
    # the weights of a token's keys sum to its heads
    first = fresh[0, :, :300].sum(-1)
    assert bool(((first - 4).abs() < 1e-3).all())


def test_weigh_unseen_content_has_no_effect(torch, sz):
    for dim, pairs, window in ((128, [(1, 37), (6, 70), (150, 333)], 0), (64, [(2, 100)], 0),
                               (256, [(1, 200), (5, 200), (80, 300)], 20)):
        S = Setup(torch, sz, pairs, 8, 2, dim, 16, seed=10)
        _, lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch, window=window)
        want, _, _ = weigh(torch, sz, S, lse, None, window=window)
        for value in (math.nan, math.inf, -math.inf):
            T = Setup(torch, sz, pairs, 8, 2, dim, 16, seed=10)
            used = torch.zeros(T.k.shape[0], 16, dtype=torch.bool)
            for s, (new, n) in enumerate(pairs):
                low = max(0, n - new + 1 - window) if window else 0
                for j in range(low, n):
                    used[T.ids[s, j // 16], j % 16] = True
            ref.page_view(T.k, T.shape, True)[~used] = value
            if window:
                for s, (new, n) in enumerate(pairs):
                    T.ids[s, :max(0, n - new + 1 - window) // 16] = -1
            T.upload()
            got, status, _ = weigh(torch, sz, T, lse, None, window=window)
            assert torch.equal(got, want) and status == [0] * len(pairs), (dim, window, value)
        # a key that some rows do not see, a row that is not a number, and a
        # log-sum of -infinity
        s, at = len(pairs) - 1, pairs[-1][1] - 1
        T = Setup(torch, sz, pairs, 8, 2, dim, 16, seed=10)
        ref.page_view(T.k, T.shape, True)[T.ids[s, at // 16], at % 16] = math.nan
        T.upload()
        got, _, _ = weigh(torch, sz, T, lse, None, window=window)
        assert bool(torch.isnan(got[s, :, at]).all())
        got[s, :, at] = want[s, :, at]
        assert torch.equal(got, want), dim
        T = Setup(torch, sz, pairs, 8, 2, dim, 16, seed=10)
        T.q[T.starts[s]] = math.nan                   # the sequence's first new token
        got, _, _ = weigh(torch, sz, T, lse, None, window=window)
        first = pairs[s][1] - pairs[s][0]
        assert torch.equal(got[:s], want[:s])
        assert torch.equal(got[s, :, first + 1:], want[s, :, first + 1:])
        assert bool(torch.isnan(got[s, :, first]).all())
        off = lse.clone()
        off[S.starts[s]] = -math.inf
        got, _, _ = weigh(torch, sz, T, off, None, window=window)
        if pairs[s][0] > 1 and not window:
            assert bool((got[s, :, :first] < want[s, :, :first]).all())
        assert bool(torch.isfinite(got[:, :, :1]).all())


def test_weigh_bad_sequences(torch, sz):
    pairs = [(2, 100), (1, 64), (40, 90), (1, 33)]
    S = Setup(torch, sz, pairs, 8, 2, 128, 16, seed=14)
    _, lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch)
    want, _, _ = weigh(torch, sz, S, lse, None)

    def run(ids=None, lens=None, starts=None, max_len=0):
        view = [ref.page_view(p, S.shape, True) for p in (S.kd, S.vd)]
        cache = S.cache if ids is None else sz.paged_cache(view[0], view[1], ids.cuda())
        i32 = dict(dtype=torch.int32, device="cuda")
        batch = sz.Batch(torch.tensor(starts or S.starts, **i32),
                         torch.tensor(lens or [n for _, n in pairs], **i32), S.n)
        out, status, _ = weigh(torch, sz, S, lse, None, cache=cache, batch=batch, max_len=max_len)
        return status, out
    ids = S.ids.clone()
    ids[2, 3] = -1
    st, out = run(ids)
    assert st == [0, 0, 1, 0] and torch.equal(out[[0, 1, 3]], want[[0, 1, 3]])
    st, out = run(lens=[100, -5, 90, 33])
    assert st == [0, 1, 0, 0] and torch.equal(out[[0, 2, 3]], want[[0, 2, 3]])
    assert bool((out[1] == SENTINEL).all())
    st, out = run(lens=[100, 64, S.width * 16 + 1, 2 ** 31 - 1])
    assert st == [0, 0, 1, 1] and bool((out[2:] == SENTINEL).all())
    st, out = run(max_len=95)
    assert st == [1, 0, 0, 0] and bool((out[0] == SENTINEL).all())
    assert run(starts=[0, 2, 3, 43, 45])[0] == [0, 0, 0, 1]
    # keys alone: the values' table is not read
    cache = sz.KVCache(S.cache._keep[0], torch.full_like(S.cache._keep[0], -8), 2, 128, 16)
    out, st, _ = weigh(torch, sz, S, lse, None, cache=cache)
    assert st == [0] * 4 and torch.equal(out, want)


# ---- eviction --------------------------------------------------------------

def pick(weights, n, budget, first, recent):
    """The positions that stay, from a list of weights."""
    if n <= budget:
        return list(range(n))
    safe = [j for j in range(n) if j < first or j >= n - recent]
    rest = [j for j in range(n) if first <= j < n - recent]
    key = [(-math.inf, 1) if math.isnan(x) else (x, 0) for x in weights]
    rest.sort(key=lambda j: (-key[j][0], key[j][1], j))
    return sorted(safe + rest[:budget - len(safe)])


class Cut:
    """A cache, its weights, and pages for what stays."""

    def __init__(self, torch, sz, lens, kv_heads, dim, page, budget, shared, to_page=None,
                 tokens_first=True, seed=0, make=None, pitch=None):
        self.torch, self.sz, self.budget = torch, sz, budget
        self.S = Setup(torch, sz, [(0, n) for n in lens], 1 * kv_heads, kv_heads, dim, page,
                       tokens_first, seed=seed)
        self.D = Setup(torch, sz, [(0, min(n, budget)) for n in lens], kv_heads, kv_heads, dim,
                       to_page or page, not tokens_first if seed % 2 else tokens_first,
                       seed=seed + 1, fill=SENTINEL)
        heads = 1 if shared else kv_heads
        pitch = pitch or max(lens + [1]) + 5
        g = torch.Generator().manual_seed(seed)
        self.w = (make or (lambda *s: torch.rand(*s, generator=g) ** 8))(len(lens), heads, pitch)
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.out = torch.full((len(lens), heads, budget), SENTINEL, device="cuda")
        self.kept = torch.full((len(lens), heads, budget), 99, dtype=torch.int32, device="cuda")
        self.lens_to = torch.full((len(lens),), 99, dtype=torch.int32, device="cuda")
        self.status = torch.full((len(lens),), -1, dtype=torch.int32, device="cuda")

    def run(self, first=0, recent=0, max_len=0, source=None, target=None, lens=None):
        most = self.S.width * self.S.page
        max_len = max_len or min(most, self.w.shape[2])
        self.sz.sz_evict_pages(self.w.cuda(), self.out, source or self.S.cache,
                               target or self.D.cache, self.lens if lens is None else lens,
                               self.lens_to, max_len, self.budget, first, recent, self.kept,
                               self.status)
        self.torch.cuda.synchronize()
        return self.status.tolist()

    def check(self, label, first=0, recent=0, only=None):
        torch, S, D = self.torch, self.S, self.D
        say(label)
        kept, out = self.kept.cpu(), self.out.cpu()
        pools = [ref.page_view(p.cpu(), D.shape, D.tokens_first) for p in (D.kd, D.vd)]
        stale = [torch.ones(p.shape[:2], dtype=torch.bool) for p in pools]
        for s, (_, n) in enumerate(S.pairs):
            if only is not None and s not in only:
                continue
            rows = [S.rows(p, s) for p in (S.k, S.v)]
            stay = min(n, self.budget)
            assert int(self.lens_to[s]) == stay, (label, s)
            d = torch.arange(stay)
            page, slot = D.ids[s, d // D.page], d % D.page
            for i in (0, 1):
                stale[i][page, slot] = False
            for h in range(S.shape[1]):
                line = 0 if self.w.shape[1] == 1 else h
                want = pick(self.w[s, line, :n].tolist(), n, self.budget, first, recent)
                assert kept[s, line].tolist() == want + [-1] * (self.budget - stay), (label, s, h)
                assert torch.equal(out[s, line, :stay].view(torch.int32),
                                   self.w[s, line, want].view(torch.int32)), (label, s)
                assert bool((out[s, line, stay:] == SENTINEL).all())
                for i in (0, 1):
                    assert torch.equal(pools[i][page, slot, h].view(torch.int16),
                                       rows[i][want, h].view(torch.int16)), (label, s, h, i)
        if only is None:
            for i in (0, 1):
                assert bool((pools[i][stale[i]] == SENTINEL).all()), label


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("shape", [(8, 128, 16), (2, 64, 32), (1, 256, 16), (3, 96, 64),
                                   (5, 8, 16), (1, 200, 128)], ids=str)
@pytest.mark.parametrize("cut", [(1, 0, 0), (40, 0, 0), (40, 4, 16), (40, 40, 0), (40, 0, 40),
                                 (40, 17, 23), (129, 4, 32), (2000, 4, 4)], ids=str)
def test_evict(torch, sz, shape, shared, cut):
    budget, first, recent = cut
    lens = [0, 1, 2, 39, 40, 41, 64, 129, 130, 1000, 300]
    for seed in (0, 1):
        C = Cut(torch, sz, lens, *shape, budget, shared, seed=seed,
                to_page=64 if seed else None)
        assert C.run(first, recent) == [0] * len(lens)
        C.check(f"evict {shape} {shared} {cut} {seed}", first, recent)


def test_evict_ties_and_odd_weights(torch, sz):
    """Equal weights (the earlier stay), zeros of both signs (equal),
    infinities, NaN (below every number), subnormal and negative ones."""
    odd = torch.tensor([0.0, -0.0, 1.0, -1.0, math.inf, -math.inf, math.nan, 1e-42, -1e-42, 3e38,
                        -3.4028234663852886e38, 1.0000001])
    g = torch.Generator().manual_seed(3)
    for make in (lambda *s: odd[torch.randint(len(odd), s, generator=g)],
                 lambda *s: torch.zeros(s),
                 lambda *s: torch.full(s, math.nan),
                 lambda *s: torch.full(s, -math.inf),
                 lambda *s: (torch.rand(*s, generator=g) * 4).round(),
                 lambda *s: torch.randint(-2 ** 31, 2 ** 31 - 1, s, generator=g,
                                          dtype=torch.int32).view(torch.float32)):
        for budget in (1, 100, 333, 699):
            C = Cut(torch, sz, [700, 40, 650], 2, 64, 16, budget, False, seed=5, make=make)
            first, recent = min(2, budget), min(30, budget - min(2, budget))
            assert C.run(first, recent) == [0] * 3
            C.check(f"ties {budget}", first, recent)


@pytest.mark.parametrize("budget", [1, 5000, 8192, 60000, 69999])
def test_evict_long(torch, sz, budget):
    """More weights than a pass of the workgroup holds."""
    for make in (None, lambda *s: (torch.rand(*s) * 3).round()):
        C = Cut(torch, sz, [70000, 8193], 1, 64, 256, budget, True, seed=6, make=make)
        assert C.run(min(4, budget), 0) == [0, 0]
        C.check(f"long {budget}", min(4, budget), 0)


def test_evict_bad_sequences(torch, sz):
    lens = [100, 64, 90, 33]

    def fresh():
        return Cut(torch, sz, lens, 2, 128, 16, 40, False, seed=8)

    def cache(S, ids):
        view = [ref.page_view(p, S.shape, S.tokens_first) for p in (S.kd, S.vd)]
        return sz.paged_cache(view[0], view[1], ids.cuda())
    C = fresh()
    ids = C.S.ids.clone()
    ids[2, 3] = -1
    assert C.run(source=cache(C.S, ids)) == [0, 0, 1, 0]
    C.check("bad source", only=(0, 1, 3))
    C = fresh()
    ids = C.D.ids.clone()
    ids[1, 2] = -1
    assert C.run(target=cache(C.D, ids)) == [0, 1, 0, 0]
    C.check("bad target", only=(0, 2, 3))
    C = fresh()
    assert C.run(lens=torch.tensor([100, -1, 2 ** 31 - 1, 33], dtype=torch.int32,
                                   device="cuda")) == [0, 1, 1, 0]
    C.check("bad lengths", only=(0, 3))
    assert C.lens_to.tolist() == [40, 0, 0, 33] and bool((C.kept[1:3] == -1).all())
    C = fresh()
    assert C.run(max_len=95) == [1, 0, 0, 0]
    C.check("short bound", only=(1, 2, 3))
    with pytest.raises(sz.SplitZipError):
        sz.evict_pages(C.w.cuda(), C.S.cache, C.D.cache, C.lens, 40, max_len=95)


def test_evict_refuses(torch, sz):
    C = Cut(torch, sz, [100, 64], 2, 128, 16, 40, False, seed=9)
    for kw in (dict(first=41), dict(first=20, recent=21), dict(max_len=200)):
        with pytest.raises(sz.SplitZipError):
            C.run(**kw)
    w = C.w.cuda()
    with pytest.raises(sz.SplitZipError):
        sz.evict_pages(w[:, :1].repeat(1, 3, 1), C.S.cache, C.D.cache, C.lens, 40)
    with pytest.raises(sz.SplitZipError):
        sz.evict_pages(w, C.S.cache, C.D.cache, C.lens, 0)
    with pytest.raises(sz.SplitZipError):             # no room
        sz.evict_pages(torch.zeros(2, 2, 200, device="cuda"), C.S.cache, C.D.cache, C.lens, 110)
    with pytest.raises(sz.SplitZipError):             # lens in place
        sz.sz_evict_pages(w, C.out, C.S.cache, C.D.cache, C.lens, C.lens, 100, 40, 0, 0, C.kept)
    with pytest.raises(ValueError):
        sz.sz_evict_pages(w[0], C.out, C.S.cache, C.D.cache, C.lens, C.lens_to, 100, 40, 0, 0,
                          C.kept)
    with pytest.raises(ValueError):
        sz.sz_evict_pages(w, C.out[:1], C.S.cache, C.D.cache, C.lens, C.lens_to, 100, 40, 0, 0,
                          C.kept)


# ---- together ----------------------------------------------------------------

@pytest.mark.parametrize("shared", [False, True])
def test_a_server_over_its_budget(torch, sz, shared):
    """Attention with its weights, eviction into other pages, the next token
    appended at the position that it would have had and attention over what is
    left, as one graph, replayed with other words; each replay checked against
    the tokens that stayed."""
    H, KH, D, page, budget = 8, 2, 64, 16, 96
    pairs = [(3, 300), (1, 90), (40, 150)]
    S = Setup(torch, sz, pairs, H, KH, D, page, seed=30)
    n, longest = len(pairs), 300
    T = Setup(torch, sz, [(1, min(length, budget) + 1) for _, length in pairs], H, KH, D, page,
              seed=31, fill=0.0)
    i32 = dict(dtype=torch.int32, device="cuda")
    q, q1 = S.q.cuda(), torch.zeros(n, H, D, dtype=torch.bfloat16, device="cuda")
    k1, v1 = (torch.zeros(n, KH, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out, lse = torch.zeros_like(q), torch.zeros(S.n, H, device="cuda")
    out1, q1_out = torch.zeros_like(q1), torch.zeros_like(q1)
    w = torch.zeros(n, KH, longest, device="cuda")
    pool = torch.zeros(n, 1, longest, device="cuda")
    WH = 1 if shared else KH
    w_to = torch.zeros(n, WH, budget, device="cuda")
    kept = torch.zeros(n, WH, budget, **i32)
    lens = torch.tensor([length for _, length in pairs], **i32)
    lens_to, lens1 = torch.zeros_like(lens), torch.zeros_like(lens)
    batch1 = sz.Batch(torch.arange(n + 1, **i32), lens1, n)
    rope = sz.rope(D)
    size = max(sz.sz_attend_workspace_size(H, S.cache, S.batch, longest),
               sz.sz_weigh_workspace_size(H, S.cache, S.batch, longest),
               sz.sz_attend_workspace_size(H, T.cache, batch1, budget + 1), 1)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def step():
        sz.sz_attend_pages(q, out, lse, S.cache, S.batch, longest, D ** -0.5, workspace=ws,
                           workspace_bytes=size)
        sz.sz_weigh_pages(q, lse, None, w, longest, 0.0, S.cache, S.batch, longest, D ** -0.5,
                          workspace=ws, workspace_bytes=size)
        if shared:
            torch.add(w[:, :1], w[:, 1:], out=pool)
        sz.sz_evict_pages(pool if shared else w, w_to, S.cache, T.cache, lens, lens_to, longest,
                          budget, 2, 8, kept)
        torch.add(lens_to, 1, out=lens1)
        sz.sz_kv_append(k1, v1, None, q1, q1_out, None, 0.0, rope, lens, T.cache, batch1)
        sz.sz_attend_pages(q1_out, out1, None, T.cache, batch1, budget + 1, D ** -0.5,
                           workspace=ws, workspace_bytes=size)

    g = torch.Generator().manual_seed(32)

    def words():
        for t in (q, q1, k1, v1, S.kd, S.vd):
            t.copy_(torch.randn(t.shape, generator=g).bfloat16())

    words()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for replay in range(4):
        words()
        w.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, lse, w, w_to, kept, lens_to, out1, T.kd, T.vd)]
        for t in (out, lse, w, out1):
            t.zero_()
        step()
        torch.cuda.synchronize()
        for s, (_, length) in enumerate(pairs):       # (past the lengths w was left)
            got[2][s, :, length:] = w[s, :, length:] = 0
        for a, b in zip(got, (out, lse, w, w_to, kept, lens_to, out1, T.kd, T.vd)):
            assert torch.equal(a, b), replay
        S.k, S.v = S.kd.cpu(), S.vd.cpu()
        say("server", replay)
        for s, (_, length) in enumerate(pairs):
            m = int(lens_to[s])
            assert m == min(length, budget)
            K, V = S.rows(S.k, s), S.rows(S.v, s)
            choose = kept[s].cpu().long()[:, :m].expand(KH, m)
            K1, V1 = (torch.stack([x[choose[h], h] for h in range(KH)], 1) for x in (K, V))
            # the new token's key as it lies in the pages, checked by the append's tests
            last = ref.page_view(T.kd.cpu(), T.shape, True)[T.ids[s, m // page], m % page]
            want, tol = ref.turn(k1[s:s + 1].cpu(), None, 0, torch.tensor([length]),
                                 [10000.0 ** (-2 * i / D) for i in range(D // 2)], D, False, 1.0)
            assert bool(((last.double() - want[0]).abs() <= tol[0]).all())
            K1, V1 = torch.cat([K1, last[None]]), torch.cat([V1, v1[s:s + 1].cpu()])
            want, _, tol, _ = ref.attend(q1_out[s:s + 1].cpu(), K1, V1, m + 1, D ** -0.5)
            assert bool(((out1[s:s + 1].cpu().double() - want).abs() <= tol).all()), (replay, s)
