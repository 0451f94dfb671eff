"""The operators on a paged cache (sz_kv_append, sz_qk_norm_rope,
sz_attend_pages) against plain 64-bit forms, at the sizes, layouts and masks
where they can go wrong, with bounds that follow from the number formats
(kv_reference.py); what no sequence owns stays as it was; refusals and bad
pages report; graphs replay; and a cache that travels through the codec
gives the same answers."""
import math
import sys

import pytest

import kv_reference as ref

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-kv]", *a, flush=True)
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
    """Pools of shuffled pages for sequences of the given (new, length), their
    contents on the CPU too, and the batch with spare rows before and after
    the sequences' own."""

    def __init__(self, torch, sz, pairs, heads, kv_heads, dim, page, tokens_first=True, seed=0,
                 before=0, behind=0, spare=2, fill=None, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.torch, self.sz, self.pairs, self.dim = torch, sz, pairs, dim
        self.shape = (page, kv_heads, dim)
        self.page, self.tokens_first = page, tokens_first
        need = [-(-n // page) for _, n in pairs]
        self.width = max(need + [1]) + 1
        count = sum(need) + spare
        order = torch.randperm(count, generator=g).tolist()
        self.ids = torch.full((max(len(pairs), 1), self.width), -1, dtype=torch.int64)
        for s, n in enumerate(need):
            for i in range(n):
                self.ids[s, i] = order.pop()
        words = page * kv_heads * dim

        def make():
            if fill is not None:
                return torch.full((count, words), fill, dtype=torch.bfloat16)
            return torch.randn(count, words, generator=g).bfloat16()
        self.k, self.v = make(), make()
        self.rand = lambda *s: torch.randn(*s, generator=g)
        starts = [before]
        for new, _ in pairs:
            starts.append(starts[-1] + new)
        self.starts = starts
        self.n = starts[-1] + behind
        self.q = (scale * torch.randn(self.n, heads, dim, generator=g)).bfloat16()
        self.upload()

    def upload(self):
        torch, sz = self.torch, self.sz
        self.kd, self.vd = self.k.cuda(), self.v.cuda()
        view = [ref.page_view(p, self.shape, self.tokens_first) for p in (self.kd, self.vd)]
        self.cache = sz.paged_cache(view[0], view[1], self.ids.cuda())
        self.batch = sz.Batch(torch.tensor(self.starts, dtype=torch.int32, device="cuda"),
                              torch.tensor([n for _, n in self.pairs], dtype=torch.int32,
                                           device="cuda"), self.n)

    def rows(self, pool, s):
        """The cached rows of sequence s in a CPU pool."""
        length = self.pairs[s][1]
        pages = self.ids[s, :-(-length // self.page)]
        x = ref.page_view(pool, self.shape, self.tokens_first)[pages]
        return x.reshape(-1, *x.shape[2:])[:length]


SENTINEL = 768.0


def check_attend(torch, sz, S, label, scale=None, max_len=0, out_type=None, status_ok=True, **kw):
    out_type = out_type or torch.bfloat16
    D = S.dim
    scale = D ** -0.5 if scale is None else scale
    out = torch.full(S.q.shape, SENTINEL, dtype=out_type, device="cuda")
    lse = torch.full(S.q.shape[:2], SENTINEL, dtype=torch.float32, device="cuda")
    size = sz.sz_attend_workspace_size(S.q.shape[1], S.cache, S.batch, max_len)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN patterns
    status = torch.full((len(S.pairs),), -1, dtype=torch.int32, device="cuda")
    sz.sz_attend_pages(S.q.cuda(), out, lse, S.cache, S.batch, max_len, scale,
                       workspace=ws if size else None, workspace_bytes=size, d_status=status, **kw)
    torch.cuda.synchronize()
    say(label, "workspace", size)
    if status_ok:
        assert status.tolist() == [0] * len(S.pairs), label
    assert bool((ws[size:] == 0xFF).all()), label
    out, lse = out.cpu().double(), lse.cpu().double()
    covered = torch.zeros(S.n, dtype=torch.bool)
    for s, (new, length) in enumerate(S.pairs):
        a, b = S.starts[s], S.starts[s + 1]
        covered[a:b] = True
        if a == b:
            continue
        want, want_lse, tol, tol_lse = ref.attend(S.q[a:b], S.rows(S.k, s), S.rows(S.v, s), length,
                                                  scale, f32_out=out_type == torch.float32, **kw)
        bad = ~((out[a:b] - want).abs() <= tol)
        assert not bool(bad.any()), (label, s, bad.nonzero()[0].tolist(),
                                     float((out[a:b] - want).abs().max()))
        empty = torch.isinf(want_lse)
        assert bool((lse[a:b][empty] == -math.inf).all()), (label, s)
        assert bool((out[a:b][empty] == 0).all()), (label, s)
        off = (lse[a:b] - want_lse).abs()[~empty] <= tol_lse[~empty]
        assert bool(off.all()), (label, s)
    assert bool((out[~covered] == SENTINEL).all()) and bool((lse[~covered] == SENTINEL).all()), label


# (new tokens, cached length) of each sequence
TOKENS = [(1, n) for n in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300, 1000)]
SHAPES = [  # heads, kv_heads, dim, page
    (32, 8, 128, 16), (8, 8, 64, 16), (8, 1, 128, 64), (6, 2, 256, 32), (7, 1, 8, 16),
    (12, 4, 80, 128), (4, 4, 200, 16), (48, 2, 96, 32), (40, 1, 72, 16), (2, 1, 136, 16),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_attend_single_tokens(torch, sz, shape):
    S = Setup(torch, sz, TOKENS, *shape, seed=1, before=2, behind=3)
    check_attend(torch, sz, S, f"single {shape}")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("tokens_first", [True, False])
def test_attend_chunks(torch, sz, shape, tokens_first):
    pairs = [(3, 3), (1, 70), (0, 40), (17, 50), (64, 64), (0, 0), (33, 200), (130, 131)]
    S = Setup(torch, sz, pairs, *shape, tokens_first=tokens_first, seed=2, behind=5)
    check_attend(torch, sz, S, f"chunks {shape} {tokens_first}")


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[1], SHAPES[3], SHAPES[7]], ids=str)
@pytest.mark.parametrize("kw", [dict(causal=False), dict(window=1), dict(window=16),
                                dict(window=37), dict(window=64), dict(window=4096),
                                dict(softcap=5.0), dict(softcap=30.0, window=50)], ids=str)
def test_attend_masks(torch, sz, shape, kw):
    pairs = [(1, 90), (5, 5), (70, 150), (2, 300), (1, 1), (1, 64), (1, 65)]
    S = Setup(torch, sz, pairs, *shape, seed=3)
    check_attend(torch, sz, S, f"masks {shape} {kw}", **kw)


def test_attend_rows_that_see_nothing(torch, sz):
    """More new tokens than cached ones: the first stand before the cache."""
    pairs = [(5, 2), (3, 0), (1, 0), (40, 20), (0, 9)]
    for shape in (SHAPES[0], SHAPES[3]):
        S = Setup(torch, sz, pairs, *shape, seed=4)
        check_attend(torch, sz, S, f"empty {shape}")
        check_attend(torch, sz, S, f"empty window {shape}", window=3)
    check_attend(torch, sz, S, "empty, not causal", causal=False)


@pytest.mark.parametrize("pairs,max_len", [
    ([(1, 5000)], 0), ([(1, 5000)], 5000), ([(1, 70), (1, 9000), (1, 2049)], 0),
    ([(4, 7777)], 7800), ([(20, 6000), (1, 33)], 0), ([(150, 3333)], 0),
], ids=str)
@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[3], (16, 1, 64, 16)], ids=str)
def test_attend_long(torch, sz, pairs, max_len, shape):
    S = Setup(torch, sz, pairs, *shape, seed=5)
    check_attend(torch, sz, S, f"long {pairs} {shape}", max_len=max_len)


@pytest.mark.parametrize("window", [600, 3000])
@pytest.mark.parametrize("shape", [(8, 1, 128, 64), (8, 1, 64, 16), (4, 1, 256, 16)], ids=str)
def test_attend_shared_out_under_a_window(torch, sz, shape, window):
    """Several tiles of one sequence whose keys begin at different places,
    cut into parts."""
    S = Setup(torch, sz, [(130, 5000), (40, 900), (1, 4000), (7, 4100)], *shape, seed=15)
    check_attend(torch, sz, S, f"shared out {shape} {window}", window=window)
    S = Setup(torch, sz, [(1, 700), (3, 5000), (2, 2222)], *shape, seed=16)
    check_attend(torch, sz, S, f"shared out, few rows {shape} {window}", window=window)


@pytest.mark.parametrize("n", [65, 130, 700, 1025])
def test_attend_many_sequences(torch, sz, n):
    """More sequences than lanes of a wave, empty ones among them."""
    pairs = [((i * 7) % 3 and 1 + (i % 11 == 5), 2 + (i * 37) % 90) for i in range(n)]
    pairs[n // 2] = (2, 4000)
    S = Setup(torch, sz, pairs, 4, 1, 64, 16, seed=17, behind=1)
    check_attend(torch, sz, S, f"many {n}")


def test_attend_f32_output_and_large_scores(torch, sz):
    S = Setup(torch, sz, [(1, 300), (9, 500)], 16, 4, 128, 16, seed=6)
    check_attend(torch, sz, S, "f32 out", out_type=torch.float32)
    # scores of several hundred: the weights are nearly one key's
    S = Setup(torch, sz, [(1, 300), (9, 500), (140, 700)], 16, 4, 128, 16, seed=7, scale=30.0)
    check_attend(torch, sz, S, "large scores", out_type=torch.float32)


def test_attend_growing_scores(torch, sz):
    """Keys that grow along the sequence: the running maximum moves in every
    tile, and by small steps."""
    for step in (0.004, 0.05):
        S = Setup(torch, sz, [(1, 1500), (130, 1500)], 8, 2, 128, 16, seed=8)
        S.q = S.q.abs()
        for s in range(2):
            page = ref.page_view(S.k, S.shape, True)
            for j in range(1500):
                page[S.ids[s, j // 16], j % 16] = step * j / 128 ** 0.5
        S.upload()
        check_attend(torch, sz, S, f"growing {step}")


def test_attend_scores_of_minus_infinity_and_lowest(torch, sz):
    """A key of the type's lowest value or of -infinity gets no weight where
    other keys have some."""
    S = Setup(torch, sz, [(1, 100), (40, 100)], 8, 2, 64, 16, seed=9)
    S.q = S.q.abs()
    page = ref.page_view(S.k, S.shape, True)
    for s in range(2):
        for j in (0, 3, 50, 59):
            page[S.ids[s, j // 16], j % 16] = -3.3e38 if j % 2 else -math.inf
    S.upload()
    out, lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch)
    for s in range(2):
        a, b = S.starts[s], S.starts[s + 1]
        keys, values = S.rows(S.k, s), S.rows(S.v, s)
        left = [j for j in range(100) if j not in (0, 3, 50, 59)]
        # the causal rows end at 60 and later: all four keys lie before them
        for i in range(b - a):
            c = 100 - (b - a) + i
            kept = [j for j in left if j <= c]
            want, want_lse, tol, _ = ref.attend(S.q[a + i:a + i + 1], keys[kept], values[kept],
                                                len(kept), 64 ** -0.5, causal=False)
            assert bool(((out[a + i:a + i + 1].cpu().double() - want).abs() <= tol).all()), (s, i)


def test_attend_unseen_content_has_no_effect(torch, sz):
    """NaN and infinities where a row does not look: past the length, ahead
    of the row, before its window; and pages there may be missing."""
    for dim, pairs, window in ((128, [(1, 37), (6, 70), (150, 333)], 0), (64, [(2, 100)], 0),
                               (128, [(1, 200), (5, 200), (80, 300)], 20), (256, [(9, 40)], 0)):
        S = Setup(torch, sz, pairs, 8, 2, dim, 16, seed=10)
        want, want_lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch, window=window)
        for value in (math.nan, math.inf, -math.inf):
            T = Setup(torch, sz, pairs, 8, 2, dim, 16, seed=10)
            for pool in (T.k, T.v):
                used = torch.zeros(pool.shape[0], 16, dtype=torch.bool)
                for s, (new, n) in enumerate(pairs):
                    low = max(0, n - new + 1 - window) if window else 0
                    for j in range(low, n):
                        used[T.ids[s, j // 16], j % 16] = True
                page = ref.page_view(pool, T.shape, True)
                page[~used] = value
            if window:   # pages that no row sees any more
                for s, (new, n) in enumerate(pairs):
                    T.ids[s, :max(0, n - new + 1 - window) // 16] = -1
            T.upload()
            got, got_lse = sz.attend_pages(T.q.cuda(), T.cache, T.batch, window=window)
            assert torch.equal(got, want) and torch.equal(got_lse, want_lse), (dim, window, value)
    # ahead of a row within its own tile: rows before the bad token are
    # untouched, whatever the token's key and value hold
    for pairs, at in (([(6, 70)], 68), ([(100, 150)], 120), ([(3, 3)], 1), ([(300, 300)], 255)):
        for dim in (64, 128, 256):
            S = Setup(torch, sz, pairs, 8, 2, dim, 16, seed=11)
            want, want_lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch)
            first = pairs[0][1] - pairs[0][0]
            for value in (math.nan, math.inf, -math.inf):
                T = Setup(torch, sz, pairs, 8, 2, dim, 16, seed=11)
                for pool in (T.k, T.v):
                    ref.page_view(pool, T.shape, True)[T.ids[0, at // 16], at % 16] = value
                T.upload()
                got, got_lse = sz.attend_pages(T.q.cuda(), T.cache, T.batch)
                n = at - first
                assert torch.equal(got[:n], want[:n]), (pairs, dim, value)
                assert torch.equal(got_lse[:n], want_lse[:n]), (pairs, dim, value)
                # an infinite value alone reaches the rows that see it
                T = Setup(torch, sz, pairs, 8, 2, dim, 16, seed=11)
                page = ref.page_view(T.v, T.shape, True)
                page[T.ids[0, at // 16], at % 16, :, 5] = value
                T.upload()
                got, _ = sz.attend_pages(T.q.cuda(), T.cache, T.batch)
                assert torch.equal(got[:n], want[:n])
                hit = got[n:, :, 5].float().cpu()
                assert bool(torch.isnan(hit).all() if math.isnan(value) else (hit == value).all())
                rest = [d for d in range(dim) if d != 5]
                assert torch.equal(got[n:, :, rest], want[n:, :, rest]), (pairs, dim, value)


def test_attend_strided_tensors(torch, sz):
    """Queries that are slices of a fused projection, and head-major ones."""
    S = Setup(torch, sz, [(1, 100), (30, 64)], 8, 2, 128, 16, seed=12)
    want, want_lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch)
    fused = torch.randn(S.n, 8 + 2 + 2, 128, device="cuda").bfloat16()
    fused[:, 2:10] = S.q.cuda()
    got, got_lse = sz.attend_pages(fused[:, 2:10], S.cache, S.batch)
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    turned = S.q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.zeros(8, S.n, 136, dtype=torch.bfloat16, device="cuda")
    size = sz.sz_attend_workspace_size(8, S.cache, S.batch)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    sz.sz_attend_pages(turned, out[:, :, :128].transpose(0, 1), None, S.cache, S.batch, 0,
                       128 ** -0.5, workspace=ws, workspace_bytes=size)
    assert torch.equal(out[:, :, :128].transpose(0, 1), want)
    assert bool((out[:, :, 128:] == 0).all())


def test_attend_offsets_past_32_bits(torch, sz):
    """Pages whose last rows lie more than 2^32 elements from their start."""
    page, stride, dim, n = 65536, 65544, 128, 66000
    words = (page - 1) * stride + 2 * dim
    pool = torch.empty(words + page * stride, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(13)
    K, V = torch.randn(n, 1, dim, generator=g).bfloat16(), torch.randn(n, 1, dim, generator=g).bfloat16()
    base = [pool.data_ptr(), pool.data_ptr() + 2 * ((page - 1) * stride + 2 * dim) // 16 * 16]
    rows = torch.as_strided(pool, (page, 2, dim), (stride, dim, 1))
    rows[:, 0], rows[:, 1] = K[:page, 0].cuda(), V[:page, 0].cuda()
    off = (base[1] - base[0]) // 2
    tail = torch.as_strided(pool, (n - page, 2, dim), (stride, dim, 1), off)
    tail[:, 0], tail[:, 1] = K[page:, 0].cuda(), V[page:, 0].cuda()
    tables = [torch.tensor([[b + 2 * dim * which for b in base]], dtype=torch.int64, device="cuda")
              for which in (0, 1)]
    cache = sz.KVCache(tables[0], tables[1], 1, dim, page, stride, dim, keep=pool)
    for new in (1, 20, 130):
        q = torch.randn(new, 8, dim, generator=g).bfloat16()
        batch = sz.Batch(torch.tensor([0, new], dtype=torch.int32, device="cuda"),
                         torch.tensor([n], dtype=torch.int32, device="cuda"), new)
        out, lse = sz.attend_pages(q.cuda(), cache, batch, window=3000)
        want, want_lse, tol, tol_lse = ref.attend(q, K, V, n, dim ** -0.5, window=3000)
        say("far offsets", new)
        assert bool(((out.cpu().double() - want).abs() <= tol).all())
        assert bool(((lse.cpu().double() - want_lse).abs() <= tol_lse).all())
    # and the append into the far end of such a page
    k = torch.randn(100, 1, dim, generator=g).bfloat16().cuda()
    batch = sz.Batch(torch.tensor([0, 100], dtype=torch.int32, device="cuda"),
                     torch.tensor([page + 20], dtype=torch.int32, device="cuda"), 100)
    sz.kv_append(k, k + 1, cache, batch)
    assert torch.equal(rows[page - 80:, 0], k[:80, 0]) and torch.equal(tail[:20, 0], k[80:, 0])
    assert torch.equal(rows[page - 80:, 1], (k + 1)[:80, 0])


def test_attend_bad_sequences(torch, sz):
    """Faults in one sequence are reported for it and leave the others alone;
    nothing outside valid pages is touched."""
    pairs = [(2, 100), (1, 64), (40, 90), (1, 33)]
    S = Setup(torch, sz, pairs, 8, 2, 128, 16, seed=14)
    want, _ = sz.attend_pages(S.q.cuda(), S.cache, S.batch)

    def status_of(ids=None, lens=None, starts=None, window=0, max_len=0):
        cache, batch = S.cache, S.batch
        if ids is not None:
            view = [ref.page_view(p, S.shape, True) for p in (S.kd, S.vd)]
            cache = sz.paged_cache(view[0], view[1], ids.cuda())
        if lens is not None or starts is not None:
            i32 = dict(dtype=torch.int32, device="cuda")
            batch = sz.Batch(torch.tensor(starts or S.starts, **i32),
                             torch.tensor(lens or [n for _, n in pairs], **i32), S.n)
        out = torch.full(S.q.shape, SENTINEL, dtype=torch.bfloat16, device="cuda")
        size = sz.sz_attend_workspace_size(8, cache, batch, max_len)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
        status = torch.full((4,), -1, dtype=torch.int32, device="cuda")
        sz.sz_attend_pages(S.q.cuda(), out, None, cache, batch, max_len, 128 ** -0.5,
                           window=window, workspace=ws, workspace_bytes=size, d_status=status)
        torch.cuda.synchronize()
        return status.tolist(), out

    ids = S.ids.clone()
    ids[2, 3] = -1
    st, out = status_of(ids=ids)
    assert st == [0, 0, 1, 0]
    assert torch.equal(out[:3], want[:3]) and torch.equal(out[43:], want[43:])
    # a missing page that no row needs is no fault
    ids = S.ids.clone()
    ids[0, 0] = -1
    st, _ = status_of(ids=ids, window=30)
    assert st == [0, 0, 0, 0]
    width = S.width * 16
    st, out = status_of(lens=[100, -5, 90, 33])
    assert st == [0, 1, 0, 0] and torch.equal(out[:2], want[:2]) and torch.equal(out[3:], want[3:])
    st, out = status_of(lens=[100, 64, width + 1, 2 ** 31 - 1])
    assert st == [0, 0, 1, 1] and torch.equal(out[:3], want[:3])
    st, out = status_of(max_len=95)
    assert st == [1, 0, 0, 0] and torch.equal(out[2:], want[2:])
    st, _ = status_of(starts=[0, 2, 3, 43, 45])        # past the rows
    assert st == [0, 0, 0, 1]
    st, _ = status_of(starts=[0, 2, 1, 43, 44])        # out of order
    assert st[1] == 1 and st[3] == 0
    st, _ = status_of(starts=[-1, 2, 3, 43, 44])
    assert st[0] == 1 and st[3] == 0


def test_attend_page_addresses_are_checked(torch, sz):
    """Misaligned addresses and ones of more than 48 bits are never followed."""
    S = Setup(torch, sz, [(1, 100), (20, 64), (1, 3000)], 8, 2, 128, 16, seed=18)
    want, _ = sz.attend_pages(S.q.cuda(), S.cache, S.batch)
    for bad in (lambda x: x + 8, lambda x: x + (1 << 50), lambda x: x | (-1 << 48)):
        for which in (0, 1):
            tables = [t.clone() for t in S.cache._keep[:2]]
            tables[which][2, 100] = bad(tables[which][2, 100])
            cache = sz.KVCache(*tables, 2, 128, 16, keep=S.cache)
            out = torch.zeros_like(want)
            size = sz.sz_attend_workspace_size(8, cache, S.batch)
            ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
            status = torch.full((3,), -1, dtype=torch.int32, device="cuda")
            sz.sz_attend_pages(S.q.cuda(), out, None, cache, S.batch, 0, 128 ** -0.5,
                               workspace=ws, workspace_bytes=size, d_status=status)
            assert status.tolist() == [0, 0, 1]
            assert torch.equal(out[:21], want[:21])


def test_attend_twice_in_one_workspace(torch, sz):
    """Two captured graphs with one workspace, replayed one after the other in
    either order, and eager calls between them."""
    sets = []
    for pairs, seed in (([(1, 3000), (1, 17)], 34), ([(5, 900), (1, 4000), (30, 30)], 35)):
        S = Setup(torch, sz, pairs, 8, 2, 128, 16, seed=seed)
        sets.append((S, S.q.cuda(), torch.zeros(S.q.shape, dtype=torch.bfloat16, device="cuda"),
                     sz.attend_pages(S.q.cuda(), S.cache, S.batch)[0]))
    size = max(sz.sz_attend_workspace_size(8, S.cache, S.batch) for S, *_ in sets)
    assert size > 0
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(S, q, out):
        sz.sz_attend_pages(q, out, None, S.cache, S.batch, 0, 128 ** -0.5, workspace=ws,
                           workspace_bytes=size)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for S, q, out, _ in sets:
            call(S, q, out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for S, q, out, _ in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(S, q, out)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1), (0, 1)):
        for i in order:
            sets[i][2].zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(sets[i][2], sets[i][3]), order
        sets[0][2].zero_()
        call(*sets[0][:3])
        assert torch.equal(sets[0][2], sets[0][3]), order


def test_nothing_to_do(torch, sz):
    """No tokens, no sequences, and sequences without new tokens."""
    S = Setup(torch, sz, [(0, 40), (0, 0)], 8, 2, 128, 16, seed=19)
    q = torch.zeros(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    out, lse = sz.attend_pages(q, S.cache, S.batch)
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    k = torch.zeros(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    assert sz.kv_append(k, k, S.cache, S.batch) is None
    none = sz.Batch(torch.zeros(1, dtype=torch.int32, device="cuda"),
                    torch.zeros(0, dtype=torch.int32, device="cuda"), 0)
    sz.attend_pages(q, S.cache, none)
    sz.kv_append(k, k, S.cache, none)
    x, _ = sz.qk_norm_rope(q, None, torch.zeros(0, dtype=torch.int32, device="cuda"), sz.rope(128))
    assert x.shape == q.shape
    torch.cuda.synchronize()


# ---- append, norm and rotation ---------------------------------------------

TURNS = [  # dim, rotary, interleaved, normed
    (128, 128, False, False), (128, 128, True, True), (128, 64, False, True), (64, 64, False, True),
    (96, 24, False, True), (96, 24, True, False), (80, 40, False, True), (256, 64, True, True),
    (256, 256, False, False), (8, 8, False, True), (200, 8, True, True), (200, 200, False, True),
    (128, 0, False, True), (72, 0, False, False), (136, 120, False, True),
]


@pytest.mark.parametrize("case", TURNS, ids=str)
@pytest.mark.parametrize("wide", [False, True])
def test_norm_rope(torch, sz, case, wide):
    dim, rotary, interleaved, normed = case
    g = torch.Generator().manual_seed(20)
    kind = torch.float32 if wide else torch.bfloat16
    for n, H, KH in ((1, 5, 3), (37, 8, 2), (700, 3, 1)):
        q, k = (torch.randn(n, h, dim, generator=g).to(kind) for h in (H, KH))
        if n > 1:
            q[1] = 0
            q[2] *= 1e-3
        pos = torch.randint(-2 ** 31, 2 ** 31, (n,), generator=g, dtype=torch.int64).int()
        pos[0] = 1048577
        freq, m = sz.sz_rope_frequencies(rotary, 10000.0, sz.SZ_ROPE_RAMP, 8.0, 4096.0) \
            if rotary else ([], 1.0)
        rope = sz.Rope(sz.rope_phases(freq).cuda(), interleaved, m) if rotary else None
        w = [1 + 0.3 * torch.randn(dim, generator=g) for _ in range(2)] if normed else [None] * 2
        wd = [x.cuda() if normed else None for x in w]
        got = sz.qk_norm_rope(q.cuda(), k.cuda(), pos.cuda(), rope, wd[0], wd[1], eps=1e-5)
        for x, weight, y in zip((q, k), w, got):
            want, tol = ref.turn(x, weight, 1e-5, pos, freq, rotary, interleaved, m)
            bad = ~((y.cpu().double() - want).abs() <= tol)
            assert not bool(bad.any()), (case, wide, n, bad.nonzero()[0].tolist())
        # one of the two alone, and in place
        alone, _ = sz.qk_norm_rope(q.cuda(), None, pos.cuda(), rope, wd[0], None, eps=1e-5)
        assert torch.equal(alone, got[0])
        if not wide:
            both = torch.cat([q, k], 1).cuda()
            qv, kv = both[:, :H], both[:, H:]
            sz.sz_qk_norm_rope(qv, qv, wd[0], kv, kv, wd[1], dim, n, pos.cuda(), 1e-5, rope)
            assert torch.equal(both[:, :H], got[0]) and torch.equal(both[:, H:], got[1])


def test_rope_of_position_zero_and_opposites(torch, sz):
    """Position 0 changes nothing; p and then -p give the words back to
    within their roundings."""
    x = torch.randn(64, 4, 128).bfloat16().cuda()
    rope = sz.rope(128, 500000.0)
    zero = torch.zeros(64, dtype=torch.int32, device="cuda")
    y, _ = sz.qk_norm_rope(x, None, zero, rope)
    assert torch.equal(x, y)
    p = torch.arange(64, dtype=torch.int32, device="cuda") * 33333
    there, _ = sz.qk_norm_rope(x, None, p, rope)
    back, _ = sz.qk_norm_rope(there, None, -p, rope)
    # each of two roundings is half a step of elements no larger than the
    # pair's length
    size = torch.hypot(x[..., :64].float(), x[..., 64:].float()).repeat(1, 1, 2)
    assert bool(((back.float() - x.float()).abs() <= 3 * ref.U16 * size).all())


@pytest.mark.parametrize("case", TURNS, ids=str)
@pytest.mark.parametrize("tokens_first", [True, False])
def test_append(torch, sz, case, tokens_first):
    dim, rotary, interleaved, normed = case
    pairs = [(1, 1), (5, 20), (0, 7), (16, 16), (40, 100), (1, 33), (0, 0), (3, 67)]
    for wide in (False, True):
        S = Setup(torch, sz, pairs, 6, 2, dim, 16, tokens_first, seed=21, before=1, behind=2)
        kind = torch.float32 if wide else torch.bfloat16
        k, v = S.rand(S.n, 2, dim).to(kind), S.rand(S.n, 2, dim).to(kind)
        q = S.rand(S.n, 6, dim).to(kind)
        freq, m = sz.sz_rope_frequencies(rotary, 10000.0) if rotary else ([], 1.0)
        rope = sz.Rope(sz.rope_phases(freq).cuda(), interleaved, m) if rotary else None
        w = [1 + 0.3 * S.rand(dim) for _ in range(2)] if normed else [None] * 2
        wd = [x.cuda() if normed else None for x in w]
        for positions in (None, torch.arange(S.n, dtype=torch.int32) * 1000 - 7):
            if positions is not None and not rotary:
                continue
            S.upload()
            out = torch.full(q.shape, SENTINEL, dtype=torch.bfloat16, device="cuda")
            status = torch.full((len(pairs),), -1, dtype=torch.int32, device="cuda")
            sz.sz_kv_append(k.cuda(), v.cuda(), wd[1], q.cuda(), out, wd[0], 1e-6, rope,
                            None if positions is None else positions.cuda(), S.cache, S.batch,
                            status)
            torch.cuda.synchronize()
            assert status.tolist() == [0] * len(pairs)
            got_k, got_v, out = S.kd.cpu(), S.vd.cpu(), out.cpu()
            same = [torch.ones(p.shape[0], 16, dtype=torch.bool) for p in (got_k, got_v)]
            view = [ref.page_view(p, S.shape, tokens_first) for p in (got_k, got_v, S.k, S.v)]
            covered = torch.zeros(S.n, dtype=torch.bool)
            for s, (new, n) in enumerate(pairs):
                a, b = S.starts[s], S.starts[s + 1]
                covered[a:b] = True
                c = torch.arange(n - new, n)
                pos = c if positions is None else positions[a:b]
                want, tol = ref.turn(k[a:b], w[1], 1e-6, pos, freq, rotary, interleaved, m)
                page, slot = S.ids[s, c // 16], c % 16
                same[0][page, slot] = same[1][page, slot] = False
                assert bool(((view[0][page, slot].double() - want).abs() <= tol).all()), (case, s)
                assert torch.equal(view[1][page, slot].view(torch.int16),
                                   v[a:b].bfloat16().view(torch.int16)), (case, s)
                want, tol = ref.turn(q[a:b], w[0], 1e-6, pos, freq, rotary, interleaved, m)
                assert bool(((out[a:b].double() - want).abs() <= tol).all()), (case, s)
            assert bool((out[~covered] == SENTINEL).all())
            for i in (0, 1):     # nothing else in any page changed
                assert torch.equal(view[i][same[i]], view[i + 2][same[i]])


def test_append_keeps_value_bits(torch, sz):
    """BF16 values go into the cache bit for bit, NaN payloads included, and
    without a rotation so do unrotated finite keys."""
    S = Setup(torch, sz, [(512, 512)], 2, 2, 64, 16, seed=22)
    words = torch.arange(512 * 2 * 64, dtype=torch.int32).to(torch.int16).view(512, 2, 64)
    x = words.view(torch.bfloat16).cuda()
    finite = torch.randn(512, 2, 64).bfloat16().cuda()
    sz.kv_append(finite, x, S.cache, S.batch)
    S.v, S.k = S.vd.cpu(), S.kd.cpu()
    assert torch.equal(S.rows(S.v, 0).contiguous().view(torch.int16), words)
    assert torch.equal(S.rows(S.k, 0), finite.cpu())


def test_append_bad_sequences(torch, sz):
    pairs = [(2, 20), (1, 64), (40, 90), (1, 33)]
    S = Setup(torch, sz, pairs, 8, 2, 128, 16, seed=23)
    k = S.rand(S.n, 2, 128).bfloat16().cuda()

    def status_of(ids=None, lens=None, starts=None):
        S.upload()
        view = [ref.page_view(p, S.shape, True) for p in (S.kd, S.vd)]
        cache = S.cache if ids is None else sz.paged_cache(view[0], view[1], ids.cuda())
        i32 = dict(dtype=torch.int32, device="cuda")
        batch = sz.Batch(torch.tensor(starts or S.starts, **i32),
                         torch.tensor(lens or [n for _, n in pairs], **i32), S.n)
        status = torch.full((4,), -1, dtype=torch.int32, device="cuda")
        sz.sz_kv_append(k, k, None, None, None, None, 0.0, None, None, cache, batch, status)
        torch.cuda.synchronize()
        changed = ((S.kd.cpu() != S.k) | (S.vd.cpu() != S.v)).any(1).nonzero().flatten().tolist()
        return status.tolist(), set(changed)

    pages = lambda s, a, b: {int(S.ids[s, j // 16]) for j in range(a, b)}  # noqa: E731
    st, changed = status_of()
    everything = pages(0, 18, 20) | pages(1, 63, 64) | pages(2, 50, 90) | pages(3, 32, 33)
    assert st == [0] * 4 and changed == everything
    ids = S.ids.clone()
    ids[2, 4] = -1                                   # in the middle of what is written
    st, changed = status_of(ids=ids)
    assert st == [0, 0, 1, 0] and changed == everything - {int(S.ids[2, 4])}
    ids = S.ids.clone()
    ids[2, 0] = -1                                   # before it: not touched, no fault
    st, changed = status_of(ids=ids)
    assert st == [0] * 4 and changed == everything
    st, changed = status_of(lens=[20, 64, 39, 33])   # shorter than its new tokens
    assert st == [0, 0, 1, 0]
    assert changed <= pages(0, 18, 20) | pages(1, 63, 64) | pages(2, 0, 39) | pages(3, 32, 33)
    st, changed = status_of(lens=[20, 64, S.width * 16 + 1, -1])
    assert st == [0, 0, 1, 1] and changed == pages(0, 18, 20) | pages(1, 63, 64)
    st, changed = status_of(starts=[0, 2, 3, 43, 45])
    assert st == [0, 0, 0, 1] and changed == everything - pages(3, 32, 33)
    with pytest.raises(sz.SplitZipError):
        sz.kv_append(k, k, S.cache, sz.Batch(
            torch.tensor(S.starts, dtype=torch.int32, device="cuda"),
            torch.tensor([1, 64, 90, 33], dtype=torch.int32, device="cuda"), S.n))


def test_wrong_device_side_arguments_raise(torch, sz):
    S = Setup(torch, sz, [(1, 20)], 8, 2, 128, 16, seed=24)
    q = S.q.cuda()
    with pytest.raises(ValueError):
        sz.attend_pages(q[:, :, :64], S.cache, S.batch)
    with pytest.raises(ValueError):
        sz.attend_pages(torch.cat([q, q]), S.cache, S.batch)
    with pytest.raises(ValueError):
        sz.attend_pages(q.float().half(), S.cache, S.batch)
    with pytest.raises(sz.SplitZipError):
        sz.attend_pages(q.float(), S.cache, S.batch)
    with pytest.raises(ValueError):
        sz.Heads(q.transpose(1, 2))
    with pytest.raises(ValueError):
        sz.qk_norm_rope(q, None, torch.zeros(1, dtype=torch.int64, device="cuda"), sz.rope(128))


# ---- together ----------------------------------------------------------------

def test_serving_steps_in_a_graph(torch, sz):
    """Append and attention of single tokens captured once and replayed with
    other tokens and lengths, each replay equal to the eager calls."""
    pairs = [(1, 200), (1, 31), (1, 1), (1, 129)]
    S = Setup(torch, sz, pairs, 8, 2, 128, 16, seed=30, spare=60)
    E = Setup(torch, sz, pairs, 8, 2, 128, 16, seed=30, spare=60)
    for X in (S, E):      # room for the tokens to come
        free = sorted(set(range(X.k.shape[0])) - set(X.ids.flatten().tolist()))
        X.ids = torch.cat([X.ids, torch.full((4, 3), -1)], 1)
        for s, (_, n) in enumerate(pairs):
            for i in range(-(-n // 16), -(-n // 16) + 3):
                X.ids[s, i] = free.pop()
        X.upload()
    rope = sz.rope(128)
    weight = 1 + 0.1 * torch.randn(128, device="cuda")
    k, v, q = (torch.randn(4, h, 128, device="cuda").bfloat16() for h in (2, 2, 8))
    lens = torch.tensor([n for _, n in pairs], dtype=torch.int32, device="cuda")
    starts = torch.arange(5, dtype=torch.int32, device="cuda")
    batch = sz.Batch(starts, lens, 4)
    qo, out = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.zeros(4, 8, device="cuda")
    size = sz.sz_attend_workspace_size(8, S.cache, batch, 0)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")

    def step(X, qo, out, lse):
        sz.sz_kv_append(k, v, weight, q, qo, weight, 1e-6, rope, None, X.cache, batch)
        sz.sz_attend_pages(qo, out, lse, X.cache, batch, 0, 0.09, workspace=ws, workspace_bytes=size)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(S, qo, out, lse)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(S, qo, out, lse)
    e = [torch.zeros_like(x) for x in (qo, out, lse)]
    for replay in range(5):
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, device="cuda"))
        if replay:
            lens += 1
        graph.replay()
        torch.cuda.synchronize()
        step(E, *e)
        torch.cuda.synchronize()
        for a, b in zip((qo, out, lse), e):
            assert torch.equal(a, b), replay
        # S was also appended to by the warm-up call, in the slot that the
        # first replay writes again
        assert torch.equal(S.kd, E.kd) and torch.equal(S.vd, E.vd), replay


def test_cache_through_the_codec(torch, sz):
    """One side reads a prompt in two chunks; its pages travel as containers
    (sz_encode_pages, sz_decode_pages) into another side's pages; both sides
    append and attend to the next token, with the same answers; and they
    match the 64-bit form over all that went in."""
    KH, H, D, page, prompt = 8, 16, 128, 16, 150
    elems = page * KH * D
    pages = -(-(prompt + 1) // page)
    g = torch.Generator().manual_seed(31)
    rand = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    k, v, q = rand(prompt + 1, KH, D), rand(prompt + 1, KH, D), rand(prompt + 1, H, D)
    rope = sz.rope(D, 500000.0)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    class Side:
        def __init__(self, seed):
            self.pools = [torch.zeros(pages + 3, page, KH, D, dtype=torch.bfloat16, device="cuda")
                          for _ in range(2)]
            gen = torch.Generator().manual_seed(seed)
            self.ids = torch.randperm(pages + 3, generator=gen)[:pages].view(1, -1).cuda()
            self.cache = sz.paged_cache(*self.pools, self.ids)

        def take(self, a, b):
            batch = sz.Batch(i32(0, b - a), i32(b), b - a)
            turned = sz.kv_append(k[a:b].cuda(), v[a:b].cuda(), self.cache, batch, rope,
                                  q=q[a:b].cuda())
            return sz.attend_pages(turned, self.cache, batch)

    one, two = Side(1), Side(2)
    first = [one.take(0, 100), one.take(100, prompt)]
    n = prompt * KH * D
    for which in range(2):
        table = [c.cache._keep[which] for c in (one, two)]
        cap = sz.sz_max_compressed_size(n)
        box = torch.empty(cap, dtype=torch.uint8, device="cuda")
        size = torch.zeros(1, dtype=torch.int64, device="cuda")
        status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        sz.sz_encode_pages(table[0], pages, elems, n, box, cap, size, status)
        total = int(size.item())
        assert int(status.item()) == 0 and total < 2 * n
        sz.sz_decode_pages(box[:total], total, table[1], pages, elems, n, status)
        assert int(status.item()) == 0
    a, b = one.take(prompt, prompt + 1), two.take(prompt, prompt + 1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # the keys as they lie in the second side's pages are the rotated ones
    ids = two.ids.cpu()[0]
    keys = two.pools[0].cpu()[ids].reshape(-1, KH, D)[:prompt + 1]
    freq, _ = sz.sz_rope_frequencies(D, 500000.0)
    want, tol = ref.turn(k, None, 0.0, torch.arange(prompt + 1), freq, D, False, 1.0)
    assert bool(((keys.double() - want).abs() <= tol).all())
    turned, _ = sz.qk_norm_rope(q.cuda(), None, torch.arange(prompt + 1, dtype=torch.int32,
                                                             device="cuda"), rope)
    want, want_lse, tol, tol_lse = ref.attend(turned.cpu(), keys, v, prompt + 1, D ** -0.5)
    got = torch.cat([first[0][0], first[1][0], b[0]]).cpu().double()
    got_lse = torch.cat([first[0][1], first[1][1], b[1]]).cpu().double()
    assert bool(((got - want).abs() <= tol).all())
    assert bool(((got_lse - want_lse).abs() <= tol_lse).all())


def test_other_streams(torch, sz):
    """Two calls on two streams with workspaces of their own."""
    S = Setup(torch, sz, [(1, 3000)], 32, 8, 128, 16, seed=32)
    T = Setup(torch, sz, [(33, 700)], 32, 8, 128, 16, seed=33)
    want = [sz.attend_pages(X.q.cuda(), X.cache, X.batch) for X in (S, T)]
    args = []
    for X in (S, T):
        size = sz.sz_attend_workspace_size(32, X.cache, X.batch)
        args.append((X.q.cuda(), torch.zeros(X.q.shape, dtype=torch.bfloat16, device="cuda"),
                     torch.zeros(X.n, 32, device="cuda"), X.cache, X.batch, 0, 128 ** -0.5, 0.0,
                     True, 0, torch.empty(max(size, 1), dtype=torch.uint8, device="cuda"), size,
                     None))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, s in zip(args, streams):
            sz.sz_attend_pages(*a, stream=s)
    torch.cuda.synchronize()
    for a, w in zip(args, want):
        assert torch.equal(a[1], w[0]) and torch.equal(a[2], w[1])


@pytest.mark.parametrize("n", [40, 64, 65, 300])
@pytest.mark.parametrize("new", [4, 900])
def test_attend_starts_out_of_order(torch, sz, n, new):
    """Ranges of rows that lie over one another, as wrong starts can make
    them: reported, nothing written past the workspace, and a sequence whose
    rows lie apart from the rest is answered."""
    page, width = 16, 160
    S = Setup(torch, sz, [(new, 2400)], 8, 2, 128, page, seed=31, before=n)
    S.ids = S.ids[:, :1].new_full((1, width), -1).index_put(
        (torch.tensor(0), torch.arange(S.ids.shape[1])), S.ids[0])
    for spread in ("over all rows", "apart"):
        hi = S.n if spread == "over all rows" else n
        starts = [0 if s % 2 == 0 else hi for s in range(n)] + [n, S.n]
        if n % 2 == 1 and spread == "over all rows":
            starts[n] = 0
        view = [ref.page_view(p, S.shape, True) for p in (S.kd, S.vd)]
        cache = sz.paged_cache(view[0], view[1], S.ids.expand(n + 1, width).cuda())
        i32 = dict(dtype=torch.int32, device="cuda")
        batch = sz.Batch(torch.tensor(starts, **i32), torch.full((n + 1,), 2400, **i32), S.n)
        out = torch.full(S.q.shape, SENTINEL, dtype=torch.bfloat16, device="cuda")
        size = sz.sz_attend_workspace_size(8, cache, batch, 2400)
        assert size > 0
        ws = torch.full((size + (1 << 22),), 0xFF, dtype=torch.uint8, device="cuda")
        status = torch.full((n + 1,), -1, dtype=torch.int32, device="cuda")
        say("out of order", n, new, spread, "workspace", size)
        sz.sz_attend_pages(S.q.cuda(), out, None, cache, batch, 2400, 128 ** -0.5, workspace=ws,
                           workspace_bytes=size, d_status=status)
        torch.cuda.synchronize()
        assert bool((ws[size:] == 0xFF).all())
        st = status.tolist()
        assert sum(st[:n]) >= n - 2
        if spread == "apart":
            assert st[n] == 0
            want, _, tol, _ = ref.attend(S.q[n:], S.rows(S.k, 0), S.rows(S.v, 0), 2400,
                                         128 ** -0.5)
            assert bool(((out[n:].cpu().double() - want).abs() <= tol).all())
        elif n % 2 == 0:
            assert st[n] == 1


def test_append_starts_out_of_order(torch, sz):
    """Every sequence that is reported good is written whole."""
    S = Setup(torch, sz, [(n, 40) for n in (3, 2, 4, 5, 1)], 8, 2, 128, 16, seed=32)
    k = S.rand(S.n, 2, 128).bfloat16().cuda()
    for starts in ([0, 3, 5, 9, 14, 15], [0, 3, 2, 9, 14, 15], [0, 12, 5, 9, 14, 15],
                   [0, 3, 5, 1, 14, 15], [0, 3, 5, 9, 14, -1], [15, 0, 3, 5, 9, 14]):
        S.upload()
        i32 = dict(dtype=torch.int32, device="cuda")
        batch = sz.Batch(torch.tensor(starts, **i32), torch.full((5,), 40, **i32), S.n)
        status = torch.full((5,), -1, dtype=torch.int32, device="cuda")
        sz.sz_kv_append(k, k, None, None, None, None, 0.0, None, None, S.cache, batch, status)
        torch.cuda.synchronize()
        for s, st in enumerate(status.tolist()):
            a, b = starts[s], starts[s + 1]
            apart = a <= b and all(x <= a for x in starts[:s]) and \
                all(x >= b for x in starts[s + 1:]) and 0 <= a and b <= S.n
            assert st == (0 if apart else 1), (starts, s)
            if apart:
                for pool in (S.kd, S.vd):
                    assert torch.equal(S.rows(pool.cpu(), s)[40 - (b - a):], k[a:b].cpu())


@pytest.mark.parametrize("window", [2 ** 30, 2 ** 31 + 5, 2 ** 32, 2 ** 63, 2 ** 64 - 1])
def test_attend_windows_past_any_length(torch, sz, window):
    S = Setup(torch, sz, [(1, 300), (70, 500)], 8, 2, 128, 16, seed=33)
    want, want_lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch)
    out, lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch, window=window)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_more_tokens_than_one_launch_takes(torch, sz):
    """2^26 and some rows, against the same rows in calls of their own."""
    n, page, R = (1 << 26) + 5, 65536, sz.rope(8)
    x = (torch.arange(n, dtype=torch.int32, device="cuda") * 40503).to(torch.int16)
    x = (x & 0x3FFF).view(torch.bfloat16).view(n, 1, 1).expand(n, 1, 8).contiguous()
    positions = torch.arange(n, dtype=torch.int32, device="cuda")
    say("rotation of", n)
    out, _ = sz.qk_norm_rope(x, None, positions, R)
    spots = [(0, 3), ((1 << 25) - 3, (1 << 25) + 3), ((1 << 26) - 3, n)]
    for a, b in spots:
        want, _ = sz.qk_norm_rope(x[a:b], None, positions[a:b], R)
        assert torch.equal(out[a:b].view(torch.int16), want.view(torch.int16)), a
    pool = torch.zeros(1025, page, 1, 8, dtype=torch.bfloat16, device="cuda")
    cache = sz.paged_cache(pool, pool, torch.arange(1025, device="cuda").view(1, -1))
    batch = sz.Batch(torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                     torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    say("append of", n)
    sz.kv_append(out, out, cache, batch)    # (keys and values to the same pages)
    got = pool.view(-1, 1, 8)
    for a, b in spots:
        assert torch.equal(got[a:b].view(torch.int16), out[a:b].view(torch.int16)), a
    assert bool((got[n:] == 0).all())


def test_as_many_sequences_as_there_can_be(torch, sz):
    """One key each: the output is its value. Then one start out of order."""
    n = 65535
    g = torch.Generator().manual_seed(34)
    pool = torch.zeros(2, n, 16, 1, 8, dtype=torch.bfloat16, device="cuda")
    cache = sz.paged_cache(pool[0], pool[1], torch.randperm(n, generator=g).view(n, 1).cuda())
    x = torch.randn(3, n, 1, 8, generator=g).bfloat16().cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    starts, lens = torch.arange(n + 1, **i32), torch.ones(n, **i32)
    batch = sz.Batch(starts, lens, n)
    say("append and attention", n)
    q = sz.kv_append(x[0], x[1], cache, batch, sz.rope(8), q=x[2])
    out, _ = sz.attend_pages(q, cache, batch)
    assert torch.equal(out, x[1])
    at = 40000
    starts[at] = 7
    want = torch.zeros(n, **i32)
    want[7:at + 1] = 1                 # what ends past row 7 before it, and the one it begins
    for call in ("append", "attend"):
        status = torch.full((n,), -1, **i32)
        if call == "append":
            sz.sz_kv_append(x[0], x[1], None, None, None, None, 0.0, None, None, cache, batch,
                            status)
        else:
            sz.sz_attend_pages(q, out.zero_(), None, cache, batch, 0, 1.0, d_status=status)
        torch.cuda.synchronize()
        got = status.cpu()
        assert torch.equal(got, want.cpu()), (call, (got != want.cpu()).nonzero()[:4].tolist())
    assert torch.equal(out[:7], x[1][:7]) and torch.equal(out[at + 1:], x[1][at + 1:])


@pytest.mark.parametrize("cap", [2.0, 50.0])
@pytest.mark.parametrize("pairs", [[(1, 1), (1, 3), (1, 40)], [(30, 30), (5, 40), (100, 100)]],
                         ids=["tokens", "chunks"])
def test_attend_caps_keep_small_scores(torch, sz, cap, pairs):
    """Scores far below the cap are as exact as without one: each within
    (head_dim / 2 + 8) rounding steps of its terms' size, and so the log-sum,
    an average of them, with as many steps of its own for the sum."""
    S = Setup(torch, sz, pairs, 8, 2, 128, 16, seed=35, scale=0.25)
    _, lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch, softcap=cap)
    for s, (new, length) in enumerate(pairs):
        a, b = S.starts[s], S.starts[s + 1]
        q, k = S.q[a:b].double(), S.rows(S.k, s).double().repeat_interleave(4, 1)
        raw = torch.einsum("ihd,jhd->ihj", q, k) * 128 ** -0.5
        size = torch.einsum("ihd,jhd->ihj", q.abs(), k.abs()) * 128 ** -0.5
        hidden = torch.arange(length)[None, :] > torch.arange(length - new, length)[:, None]
        t = (cap * torch.tanh(raw / cap)).masked_fill(hidden[:, None], -math.inf)
        want = torch.logsumexp(t, -1)
        most = size.masked_fill(hidden[:, None], 0).amax(-1)
        tol = 2.0 ** -24 * ((64 + 8) * most + 16 * (1 + want.abs()))
        got = lse[a:b].cpu().double()
        assert bool(((got - want).abs() <= tol).all()), (s, float(((got - want).abs() / tol).max()))
