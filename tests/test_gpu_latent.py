"""The operators on a paged cache of latents (sz_latent_append,
sz_attend_latent) against plain 64-bit forms, at the sizes, layouts and masks
where they can go wrong, with the bounds of kv_reference.py."""
import math
import sys

import pytest

import kv_reference as ref

pytestmark = pytest.mark.gpu
SENTINEL = 768.0


def say(*a):
    print("[gpu-latent]", *a, flush=True)
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


class Setup:
    """Shuffled pages of latents for sequences of the given (new, length), on
    the CPU too, with spare pages and spare rows around the sequences' own;
    `gap` elements between a page's rows."""

    def __init__(self, torch, sz, pairs, heads, latent, rotary, page, seed=0, before=0, behind=0,
                 spare=2, scale=1.0, gap=0):
        g = torch.Generator().manual_seed(seed)
        self.torch, self.sz, self.pairs, self.page = torch, sz, pairs, page
        self.latent, self.rotary, self.dim = latent, rotary, latent + rotary
        need = [-(-n // page) for _, n in pairs]
        self.width = max(need + [1]) + 1
        count = sum(need) + spare
        order = torch.randperm(count, generator=g).tolist()
        self.ids = torch.full((max(len(pairs), 1), self.width), -1, dtype=torch.int64)
        for s, n in enumerate(need):
            for i in range(n):
                self.ids[s, i] = order.pop()
        self.pool = torch.randn(count, page, self.dim + gap, generator=g).bfloat16()
        starts = [before]
        for new, _ in pairs:
            starts.append(starts[-1] + new)
        self.starts, self.n = starts, starts[-1] + behind
        self.rand = lambda *s: torch.randn(*s, generator=g)
        self.q = (scale * self.rand(self.n, heads, self.dim)).bfloat16()
        self.scale = (min(latent, 128) + rotary) ** -0.5
        self.upload()

    def upload(self):
        torch, sz = self.torch, self.sz
        self.dev = self.pool.cuda()
        self.cache = sz.latent_cache(self.dev[..., :self.dim], self.ids.cuda(), self.latent)
        self.batch = self.batch_of()

    def batch_of(self, starts=None, lens=None):
        i32 = dict(dtype=self.torch.int32, device="cuda")
        return self.sz.Batch(self.torch.tensor(starts or self.starts, **i32),
                             self.torch.tensor(lens or [n for _, n in self.pairs], **i32), self.n)

    def rows(self, s):
        length = self.pairs[s][1]
        pages = self.ids[s, :-(-length // self.page)]
        return self.pool[pages].reshape(-1, self.pool.shape[2])[:length, :self.dim]


def attend(torch, sz, S, out_type=None, max_len=0, causal=True, cache=None, batch=None):
    cache, batch = cache or S.cache, batch or S.batch
    H = S.q.shape[1]
    out = torch.full((S.n, H, S.latent), SENTINEL, dtype=out_type or torch.bfloat16, device="cuda")
    lse = torch.full((S.n, H), SENTINEL, device="cuda")
    size = sz.sz_attend_latent_workspace_size(H, cache, batch, max_len)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN patterns
    status = torch.full((len(S.pairs),), -1, dtype=torch.int32, device="cuda")
    sz.sz_attend_latent(S.q.cuda(), out, lse, cache, batch, max_len, S.scale, causal,
                        ws if size else None, size, status)
    torch.cuda.synchronize()
    assert bool((ws[size:] == 0xFF).all())
    return out, lse, status.tolist()


def check(torch, sz, S, label, out_type=None, max_len=0, causal=True):
    say(label)
    out, lse, status = attend(torch, sz, S, out_type, max_len, causal)
    assert status == [0] * len(S.pairs), label
    out, lse = out.cpu().double(), lse.cpu().double()
    covered = torch.zeros(S.n, dtype=torch.bool)
    for s, (new, length) in enumerate(S.pairs):
        a, b = S.starts[s], S.starts[s + 1]
        covered[a:b] = True
        if a == b:
            continue
        if length == 0:
            assert bool((out[a:b] == 0).all()) and bool((lse[a:b] == -math.inf).all()), (label, s)
            continue
        K = S.rows(s)[:, None]
        want, want_lse, tol, tol_lse = ref.attend(S.q[a:b], K, K[..., :S.latent], length, S.scale,
                                                  causal=causal,
                                                  f32_out=out_type == torch.float32)
        bad = ~((out[a:b] - want).abs() <= tol)
        assert not bool(bad.any()), (label, s, bad.nonzero()[0].tolist(),
                                     float((out[a:b] - want).abs().max()))
        empty = torch.isinf(want_lse)
        assert bool((lse[a:b][empty] == -math.inf).all()), (label, s)
        assert bool((out[a:b][empty] == 0).all()), (label, s)
        assert bool(((lse[a:b] - want_lse).abs()[~empty] <= tol_lse[~empty]).all()), (label, s)
    assert bool((out[~covered] == SENTINEL).all()) and bool((lse[~covered] == SENTINEL).all()), label


TOKENS = [(1, n) for n in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300, 1000)]
SHAPES = [  # heads, latent, rotary, page
    (16, 512, 64, 16), (128, 512, 64, 64), (1, 512, 64, 16), (40, 384, 32, 32), (64, 256, 64, 16),
    (20, 64, 0, 16), (33, 8, 8, 128), (7, 512, 0, 16), (65, 296, 56, 16), (32, 248, 40, 16),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_single_tokens(torch, sz, shape):
    S = Setup(torch, sz, TOKENS, *shape, seed=1, before=2, behind=3)
    check(torch, sz, S, f"single {shape}")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_chunks(torch, sz, shape, causal):
    pairs = [(3, 3), (1, 70), (0, 40), (17, 50), (9, 64), (0, 0), (5, 200), (2, 131)]
    S = Setup(torch, sz, pairs, *shape, seed=2, behind=5)
    check(torch, sz, S, f"chunks {shape} {causal}", causal=causal)


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[1], SHAPES[4]], ids=str)
def test_rows_that_see_nothing(torch, sz, shape):
    """More new tokens than cached ones: the first stand before the cache."""
    pairs = [(5, 2), (3, 0), (1, 0), (20, 9), (0, 9)]
    S = Setup(torch, sz, pairs, *shape, seed=3)
    check(torch, sz, S, f"empty {shape}")
    check(torch, sz, S, f"empty {shape}, not causal", causal=False)


@pytest.mark.parametrize("pairs,max_len", [
    ([(1, 5000)], 0), ([(1, 5000)], 5000), ([(1, 70), (1, 9000), (1, 2049)], 0),
    ([(4, 3777)], 3800), ([(20, 2000), (1, 33)], 0),
], ids=str)
@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[1], SHAPES[4], (24, 512, 64, 16)], ids=str)
def test_long(torch, sz, pairs, max_len, shape):
    S = Setup(torch, sz, pairs, *shape, seed=4)
    check(torch, sz, S, f"long {pairs} {shape}", max_len=max_len)


@pytest.mark.parametrize("n", [65, 300, 1025])
def test_many_sequences(torch, sz, n):
    """More sequences than lanes of a wave, and than the work is shared out for."""
    pairs = [((i * 7) % 3 and 1 + (i % 11 == 5), 2 + (i * 37) % 90) for i in range(n)]
    pairs[n // 2] = (2, 2000)
    S = Setup(torch, sz, pairs, 12, 64, 16, 16, seed=5, behind=1)
    check(torch, sz, S, f"many {n}")


def test_f32_output_and_large_scores(torch, sz):
    S = Setup(torch, sz, [(1, 300), (3, 500)], 40, 512, 64, 16, seed=6)
    check(torch, sz, S, "f32 out", out_type=torch.float32)
    S = Setup(torch, sz, [(1, 300), (3, 500), (1, 2000)], 40, 512, 64, 16, seed=7, scale=30.0)
    check(torch, sz, S, "large scores", out_type=torch.float32)
    S = Setup(torch, sz, [(1, 300), (1, 2000)], 16, 512, 64, 16, seed=7, scale=30.0)
    check(torch, sz, S, "large scores, few rows", out_type=torch.float32)


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("step", [0.004, 0.05])
def test_growing_scores(torch, sz, heads, step):
    """Keys that grow along the sequence: the running maximum moves in every
    step, and by small ones; and differs between the halves of a step."""
    S = Setup(torch, sz, [(1, 1500), (2, 1500)], heads, 512, 64, 16, seed=8)
    S.q = S.q.abs()
    for s in range(2):
        for j in range(1500):
            S.pool[S.ids[s, j // 16], j % 16] = step * j / 24
    S.upload()
    check(torch, sz, S, f"growing {step}")
    for s in range(2):
        for j in range(1500):
            S.pool[S.ids[s, j // 16], j % 16] = step * (1500 - j) / 24
    S.upload()
    check(torch, sz, S, f"falling {step}")


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[1], SHAPES[8]], ids=str)
def test_unseen_content_has_no_effect(torch, sz, shape):
    pairs = [(1, 37), (6, 70), (9, 133)]
    S = Setup(torch, sz, pairs, *shape, seed=10)
    want, want_lse, _ = attend(torch, sz, S)
    for value in (math.nan, math.inf, -math.inf):
        T = Setup(torch, sz, pairs, *shape, seed=10)
        used = torch.zeros(T.pool.shape[:2], dtype=torch.bool)
        for s, (_, n) in enumerate(pairs):
            for j in range(n):
                used[T.ids[s, j // T.page], j % T.page] = True
        T.pool[~used] = value
        T.upload()
        got, got_lse, _ = attend(torch, sz, T)
        assert torch.equal(got, want) and torch.equal(got_lse, want_lse), value
        # in a token that some rows of a tile see and others do not
        for s, at in ((1, 67), (2, 128)):
            for element in (slice(None), 5):
                T = Setup(torch, sz, pairs, *shape, seed=10)
                T.pool[T.ids[s, at // T.page], at % T.page, element] = value
                T.upload()
                got, got_lse, _ = attend(torch, sz, T)
                seen = torch.zeros(T.n, dtype=torch.bool)
                seen[T.starts[s + 1] - (pairs[s][1] - at):T.starts[s + 1]] = True
                assert torch.equal(got[~seen], want[~seen]), (value, s, element)
                assert torch.equal(got_lse[~seen], want_lse[~seen]), (value, s, element)
                assert bool((~torch.isfinite(got[seen][..., element])).all()), (value, s, element)


def test_strided_tensors(torch, sz):
    """Rows with room between them in the pages, queries within wider rows,
    outputs head by head."""
    S = Setup(torch, sz, [(1, 100), (3, 64), (1, 900)], 20, 512, 64, 16, seed=12, gap=24)
    check(torch, sz, S, "rows apart")
    want, _, _ = attend(torch, sz, S)
    wide = torch.full((S.n, 21, 600), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:, 8:584] = S.q.cuda()
    out = torch.zeros(20, S.n, 520, dtype=torch.bfloat16, device="cuda")
    size = sz.sz_attend_latent_workspace_size(20, S.cache, S.batch)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    sz.sz_attend_latent(wide[:, 1:, 8:584], out[:, :, :512].transpose(0, 1), None, S.cache,
                        S.batch, 0, S.scale, True, ws, size)
    assert torch.equal(out[:, :, :512].transpose(0, 1), want)
    assert bool((out[:, :, 512:] == 0).all())


def test_offsets_past_32_bits(torch, sz):
    """Pages whose last rows lie more than 2^32 bytes from their start."""
    page, stride, n = 65536, 36872, 66000
    pool = torch.empty(2 * page * stride, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(13)
    rows = torch.randn(n, 576, generator=g).bfloat16()
    view = torch.as_strided(pool, (n, 576), (stride, 1))
    view.copy_(rows.cuda())
    table = torch.tensor([[pool.data_ptr(), pool.data_ptr() + 2 * page * stride]], device="cuda")
    cache = sz.LatentCache(table, 512, 64, page, stride, keep=pool)
    scale = 192 ** -0.5
    for new, heads in ((1, 16), (2, 64)):
        q = torch.randn(new, heads, 576, generator=g).bfloat16()
        batch = sz.Batch(torch.tensor([0, new], dtype=torch.int32, device="cuda"),
                         torch.tensor([n], dtype=torch.int32, device="cuda"), new)
        say("far offsets", new)
        out, lse = sz.attend_latent(q.cuda(), cache, batch, scale)
        want, want_lse, tol, tol_lse = ref.attend(q, rows[:, None], rows[:, None, :512], n, scale)
        assert bool(((out.cpu().double() - want).abs() <= tol).all())
        assert bool(((lse.cpu().double() - want_lse).abs() <= tol_lse).all())
    x = torch.randn(100, 1, 576, generator=g).bfloat16().cuda()
    batch = sz.Batch(torch.tensor([0, 100], dtype=torch.int32, device="cuda"),
                     torch.tensor([page + 20], dtype=torch.int32, device="cuda"), 100)
    sz.latent_append(x[..., :512], cache, batch, x[..., 512:])
    assert torch.equal(view[page - 80:page + 20], x[:, 0])


def test_bad_sequences(torch, sz):
    pairs = [(2, 100), (1, 64), (4, 90), (1, 33)]
    S = Setup(torch, sz, pairs, 40, 512, 64, 16, seed=14)
    want, _, _ = attend(torch, sz, S)

    def run(ids=None, **kw):
        cache = None if ids is None else sz.latent_cache(S.dev, ids.cuda(), 512)
        batch = S.batch_of(**{k: v for k, v in kw.items() if k != "max_len"})
        out, _, status = attend(torch, sz, S, cache=cache, batch=batch,
                                max_len=kw.get("max_len", 0))
        return status, out
    ids = S.ids.clone()
    ids[2, 3] = -1
    st, out = run(ids)
    assert st == [0, 0, 1, 0] and torch.equal(out[:3], want[:3]) and torch.equal(out[7:], want[7:])
    st, out = run(lens=[100, -5, 90, 33])
    assert st == [0, 1, 0, 0] and torch.equal(out[:2], want[:2]) and torch.equal(out[3:], want[3:])
    st, out = run(lens=[100, 64, S.width * 16 + 1, 2 ** 31 - 1])
    assert st == [0, 0, 1, 1] and torch.equal(out[:3], want[:3])
    st, out = run(max_len=95)
    assert st == [1, 0, 0, 0] and torch.equal(out[2:], want[2:])
    assert run(starts=[0, 2, 3, 7, 9])[0] == [0, 0, 0, 1]
    st, _ = run(starts=[0, 2, 1, 7, 8])
    assert st[1] == 1 and st[3] == 0
    # addresses that are never followed
    for bad in (lambda x: x + 8, lambda x: x + (1 << 50), lambda x: x | (-1 << 48)):
        table = S.cache._keep[0].clone()
        table[2, 1] = bad(table[2, 1])
        out, _, st = attend(torch, sz, S, cache=sz.LatentCache(table, 512, 64, 16, keep=S.dev))
        assert st == [0, 0, 1, 0] and torch.equal(out[:3], want[:3])
    with pytest.raises(sz.SplitZipError):
        sz.attend_latent(S.q.cuda(), S.cache, S.batch, S.scale, max_len=95)


APPENDS = [  # latent, rotary, interleaved, normed
    (512, 64, True, True), (512, 64, False, True), (384, 32, False, False), (8, 8, False, True),
    (504, 24, False, True), (256, 56, True, True), (512, 0, False, True), (64, 40, False, False),
]


@pytest.mark.parametrize("case", APPENDS, ids=str)
@pytest.mark.parametrize("wide", [False, True])
def test_append(torch, sz, case, wide):
    latent, rotary, interleaved, normed = case
    pairs = [(1, 1), (5, 20), (0, 7), (16, 16), (40, 100), (1, 33), (0, 0), (3, 67)]
    kind = torch.float32 if wide else torch.bfloat16
    for heads in (1, 9, 128):
        S = Setup(torch, sz, pairs, 1, latent, rotary, 16, seed=21, before=1, behind=2, gap=8)
        x = S.rand(S.n, 1, S.dim).to(kind)
        q = S.rand(S.n, heads, rotary).to(kind) if rotary else None
        freq, m = sz.sz_rope_frequencies(rotary, 10000.0, sz.SZ_ROPE_RAMP, 8.0, 4096.0) \
            if rotary else ([], 1.0)
        rope = sz.Rope(sz.rope_phases(freq).cuda(), interleaved, m) if rotary else None
        w = 1 + 0.3 * S.rand(latent) if normed else None
        for positions in (None, torch.arange(S.n, dtype=torch.int32) * 1000 - 7):
            S.upload()
            rows = torch.full((S.n, heads, latent + rotary), SENTINEL, dtype=torch.bfloat16,
                              device="cuda")
            out = rows[..., latent:] if rotary else None
            status = torch.full((len(pairs),), -1, dtype=torch.int32, device="cuda")
            xd = x.cuda()
            say("append", case, wide, heads)
            sz.sz_latent_append(xd[..., :latent], w.cuda() if normed else None, 1e-6,
                                xd[..., latent:] if rotary else None,
                                q.cuda() if rotary else None, out, rope,
                                None if positions is None else positions.cuda(), S.cache, S.batch,
                                status)
            torch.cuda.synchronize()
            assert status.tolist() == [0] * len(pairs)
            got = S.dev.cpu()
            same = torch.ones(got.shape[:2], dtype=torch.bool)
            covered = torch.zeros(S.n, dtype=torch.bool)
            for s, (new, n) in enumerate(pairs):
                a, b = S.starts[s], S.starts[s + 1]
                covered[a:b] = True
                c = torch.arange(n - new, n)
                pos = c if positions is None else positions[a:b]
                page, slot = S.ids[s, c // 16], c % 16
                same[page, slot] = False
                parts = [ref.turn(x[a:b, :, :latent], w, 1e-6, pos, [], 0, False, 1.0)]
                if rotary:
                    parts.append(ref.turn(x[a:b, :, latent:], None, 0, pos, freq, rotary,
                                          interleaved, m))
                want, tol = (torch.cat([p[i][:, 0] for p in parts], -1) for i in (0, 1))
                row = got[page, slot][:, :S.dim].double()
                assert bool(((row - want).abs() <= tol).all()), (case, s)
                if rotary:
                    want, tol = ref.turn(q[a:b], None, 0, pos, freq, rotary, interleaved, m)
                    assert bool(((out[a:b].cpu().double() - want).abs() <= tol).all()), (case, s)
            assert torch.equal(got[same], S.pool[same])               # nothing else changed
            assert torch.equal(got[..., S.dim:], S.pool[..., S.dim:])
            assert bool((rows[..., :latent] == SENTINEL).all())
            assert bool((rows[~covered.cuda()] == SENTINEL).all())


def test_append_in_place_and_without_queries(torch, sz):
    S = Setup(torch, sz, [(3, 30), (1, 9)], 6, 512, 64, 16, seed=22)
    x, rope = S.rand(4, 1, 576).bfloat16().cuda(), sz.rope(64)
    q = S.q.cuda()
    turned = sz.latent_append(x[..., :512], S.cache, S.batch, x[..., 512:], rope,
                              q=q[..., 512:])
    pool = S.dev.clone()
    same = q.clone()
    sz.sz_latent_append(x[..., :512], None, 0.0, x[..., 512:], same[..., 512:], same[..., 512:],
                        rope, None, S.cache, S.batch)
    assert torch.equal(same[..., 512:], turned) and torch.equal(same[..., :512], q[..., :512])
    S.upload()
    assert sz.latent_append(x[..., :512], S.cache, S.batch, x[..., 512:], rope) is None
    assert torch.equal(S.dev, pool)


def test_append_bad_sequences(torch, sz):
    pairs = [(2, 20), (1, 64), (40, 90), (1, 33)]
    S = Setup(torch, sz, pairs, 4, 512, 64, 16, seed=23)
    x = S.rand(S.n, 1, 576).bfloat16().cuda()

    def run(ids=None, **kw):
        S.upload()
        cache = S.cache if ids is None else sz.latent_cache(S.dev, ids.cuda(), 512)
        status = torch.full((4,), -1, dtype=torch.int32, device="cuda")
        sz.sz_latent_append(x[..., :512], None, 0.0, x[..., 512:], None, None, None, None, cache,
                            S.batch_of(**kw), status)
        changed = (S.dev.cpu() != S.pool).flatten(1).any(1).nonzero().flatten().tolist()
        return status.tolist(), set(changed)
    pages = lambda s, a, b: {int(S.ids[s, j // 16]) for j in range(a, b)}  # noqa: E731
    every = pages(0, 18, 20) | pages(1, 63, 64) | pages(2, 50, 90) | pages(3, 32, 33)
    assert run() == ([0] * 4, every)
    ids = S.ids.clone()
    ids[2, 4] = -1
    assert run(ids) == ([0, 0, 1, 0], every - {int(S.ids[2, 4])})
    st, changed = run(lens=[20, 64, 39, 33])
    assert st == [0, 0, 1, 0]
    assert changed <= pages(0, 18, 20) | pages(1, 63, 64) | pages(2, 0, 39) | pages(3, 32, 33)
    st, changed = run(lens=[20, 64, S.width * 16 + 1, -1])
    assert st == [0, 0, 1, 1] and changed == pages(0, 18, 20) | pages(1, 63, 64)
    assert run(starts=[0, 2, 3, 43, 45]) == ([0, 0, 0, 1], every - pages(3, 32, 33))


def test_nothing_to_do(torch, sz):
    S = Setup(torch, sz, [(0, 40), (0, 0)], 8, 512, 64, 16, seed=24)
    q = torch.zeros(0, 8, 576, dtype=torch.bfloat16, device="cuda")
    out, lse = sz.attend_latent(q, S.cache, S.batch, 0.1)
    assert out.shape == (0, 8, 512) and lse.shape == (0, 8)
    x = torch.zeros(0, 1, 576, dtype=torch.bfloat16, device="cuda")
    assert sz.latent_append(x[..., :512], S.cache, S.batch, x[..., 512:]) is None
    torch.cuda.synchronize()


# ---- both ways of cutting the work up ------------------------------------------

@pytest.mark.parametrize("heads,n,shape", [(16, 600, (512, 64)), (40, 530, (64, 16)),
                                           (128, 260, (512, 64)), (128, 270, (200, 8))], ids=str)
def test_whole_tiles(torch, sz, heads, n, shape):
    """More tiles than two for each CU, of 32, 64 and 128 rows: every one whole."""
    pairs = [(1, 1 + 37 * s % 150) for s in range(n)]
    S = Setup(torch, sz, pairs, heads, *shape, 16, seed=40)
    assert sz.sz_attend_latent_workspace_size(heads, S.cache, S.batch, 0) == 0
    check(torch, sz, S, f"whole {heads} {n}")


@pytest.mark.parametrize("heads,n,shape", [(16, 200, (512, 64)), (40, 130, (64, 16)),
                                           (128, 70, (512, 64))], ids=str)
def test_many_sequences_share_the_chip(torch, sz, heads, n, shape):
    """More sequences than a wave has lanes, one of them long: shared out."""
    pairs = [(1, 1 + 37 * s % 150) for s in range(n)]
    pairs[n // 3] = (1, 5000)
    S = Setup(torch, sz, pairs, heads, *shape, 64, seed=41)
    assert sz.sz_attend_latent_workspace_size(heads, S.cache, S.batch, 5000) > 0
    check(torch, sz, S, f"shared {heads} {n}", max_len=5000)
