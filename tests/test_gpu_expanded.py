"""Attention over keys and values expanded from latents (sz_attend_expanded)
against a plain 64-bit form, at the sizes, layouts and masks where it can go
wrong, with the bounds of kv_reference.py; and the two forms of latent
attention against each other."""
import math
import sys

import pytest

import kv_reference as ref

pytestmark = pytest.mark.gpu
SENTINEL = 768.0


def say(*a):
    print("[gpu-expanded]", *a, flush=True)
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
    """Sequences of (new, length) with their keys in shuffled order of
    sequences and spare rows between them; keys and values side by side in
    every head, the rotary part behind wider rows."""

    def __init__(self, torch, pairs, heads, dims, seed=0, before=0, behind=0, gap=3, scale=1.0,
                 own_rotary=False):
        g = torch.Generator().manual_seed(seed)
        self.torch, self.pairs, self.dims = torch, pairs, dims
        D, R, V = dims
        order = torch.randperm(max(len(pairs), 1), generator=g).tolist()
        self.key_starts, at = [0] * len(pairs), gap
        for s in order[:len(pairs)]:
            self.key_starts[s] = at
            at += pairs[s][1] + gap
        self.n_keys = at
        self.kv = torch.randn(at, heads, D + V, generator=g).bfloat16()
        self.r = torch.randn(at, heads if own_rotary else 1, 40 + R, generator=g).bfloat16()
        starts = [before]
        for new, _ in pairs:
            starts.append(starts[-1] + new)
        self.starts, self.n = starts, starts[-1] + behind
        self.q = (scale * torch.randn(self.n, heads, D + R, generator=g)).bfloat16()
        self.scale = (D + R) ** -0.5
        self.heads = heads

    def tensors(self):
        D, R, _ = self.dims
        kv, r = self.kv.cuda(), self.r.cuda()
        return kv[..., :D], r[..., 40:] if R else None, kv[..., D:]

    def rows(self, s):
        D, R, _ = self.dims
        at = slice(self.key_starts[s], self.key_starts[s] + self.pairs[s][1])
        r = self.r[at, :, 40:].expand(-1, self.heads, -1)
        return self.torch.cat([self.kv[at, :, :D], r], -1), self.kv[at, :, D:]


def attend(torch, sz, S, out_type=None, max_len=0, causal=True, starts=None, lens=None,
           key_starts=None):
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = sz.Batch(torch.tensor(starts or S.starts, **i32),
                     torch.tensor(lens or [n for _, n in S.pairs], **i32), S.n)
    V = S.dims[2]
    out = torch.full((S.n, S.heads, V), SENTINEL, dtype=out_type or torch.bfloat16, device="cuda")
    lse = torch.full((S.n, S.heads), SENTINEL, device="cuda")
    k, r, v = S.tensors()
    most = max_len if 0 < max_len < S.n_keys else S.n_keys
    size = sz.sz_attend_expanded_workspace_size(S.heads, V, batch, most)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    status = torch.full((len(S.pairs),), -1, dtype=torch.int32, device="cuda")
    sz.sz_attend_expanded(S.q.cuda(), out, lse, k, r, v,
                          torch.tensor(key_starts or S.key_starts, **i32), batch, max_len, S.scale,
                          causal, ws if size else None, size, status)
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
        K, V = S.rows(s)
        want, want_lse, tol, tol_lse = ref.attend(S.q[a:b], K, V, length, S.scale, causal=causal,
                                                  f32_out=out_type == torch.float32)
        bad = ~((out[a:b] - want).abs() <= tol)
        assert not bool(bad.any()), (label, s, bad.nonzero()[0].tolist(),
                                     float((out[a:b] - want).abs().max()))
        empty = torch.isinf(want_lse)
        assert bool((lse[a:b][empty] == -math.inf).all()), (label, s)
        assert bool((out[a:b][empty] == 0).all()), (label, s)
        assert bool(((lse[a:b] - want_lse).abs()[~empty] <= tol_lse[~empty]).all()), (label, s)
    assert bool((out[~covered] == SENTINEL).all()) and bool((lse[~covered] == SENTINEL).all()), label


DIMS = [(128, 64, 128), (96, 32, 96), (64, 64, 128), (128, 0, 64), (8, 8, 8), (120, 56, 104),
        (16, 0, 128)]
PAIRS = [(3, 3), (1, 70), (0, 40), (17, 50), (64, 64), (0, 0), (33, 200), (130, 131), (1, 1)]


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("own_rotary", [True, False])
def test_chunks(torch, sz, dims, causal, own_rotary):
    S = Setup(torch, PAIRS, 5, dims, seed=1, before=2, behind=4, own_rotary=own_rotary)
    check(torch, sz, S, f"chunks {dims} {causal} {own_rotary}", causal=causal)


@pytest.mark.parametrize("pairs,heads,max_len", [
    ([(300, 300)], 3, 0), ([(300, 900), (40, 1300)], 2, 1300), ([(1, 3000)], 4, 0),
    ([(700, 700)], 130, 0), ([(256, 513), (257, 600)], 160, 600), ([(1030, 1100)], 64, 0),
    ([(140, 2500), (1, 65), (128, 128)], 1, 0), ([(100, 100)], 300, 0),
], ids=str)
@pytest.mark.parametrize("dims", [DIMS[0], DIMS[5]], ids=str)
def test_long(torch, sz, pairs, heads, max_len, dims):
    """Tiles of 128 and 256 rows, whole and shared out, more heads than CUs."""
    S = Setup(torch, pairs, heads, dims, seed=2)
    check(torch, sz, S, f"long {pairs} {heads} {dims}", max_len=max_len)


def test_rows_that_see_nothing(torch, sz):
    S = Setup(torch, [(5, 2), (3, 0), (1, 0), (200, 100), (0, 9)], 3, DIMS[0], seed=3)
    check(torch, sz, S, "empty")
    check(torch, sz, S, "empty, not causal", causal=False)


@pytest.mark.parametrize("n", [65, 1025])
def test_many_sequences(torch, sz, n):
    pairs = [((i * 7) % 3 and 1 + (i % 11 == 5), 2 + (i * 37) % 90) for i in range(n)]
    pairs[n // 2] = (2, 900)
    S = Setup(torch, pairs, 2, (64, 32, 64), seed=4, behind=1)
    check(torch, sz, S, f"many {n}")


def test_f32_output_and_large_scores(torch, sz):
    S = Setup(torch, [(10, 300), (150, 700)], 4, DIMS[0], seed=5)
    check(torch, sz, S, "f32 out", out_type=torch.float32)
    S = Setup(torch, [(10, 300), (150, 700)], 4, DIMS[0], seed=6, scale=30.0)
    check(torch, sz, S, "large scores", out_type=torch.float32)


@pytest.mark.parametrize("pairs,heads", [([(6, 70), (150, 333)], 2), ([(600, 700)], 128)], ids=str)
def test_unseen_content_has_no_effect(torch, sz, pairs, heads):
    S = Setup(torch, pairs, heads, DIMS[0], seed=7)
    want, want_lse, _ = attend(torch, sz, S)
    D = S.dims[0]
    for value in (math.nan, math.inf, -math.inf):
        T = Setup(torch, pairs, heads, DIMS[0], seed=7)
        used = torch.zeros(T.n_keys, dtype=torch.bool)
        for s, (_, n) in enumerate(pairs):
            used[T.key_starts[s]:T.key_starts[s] + n] = True
        T.kv[~used], T.r[~used], T.r[..., :40] = value, value, value
        got, got_lse, _ = attend(torch, sz, T)
        assert torch.equal(got, want) and torch.equal(got_lse, want_lse), value
        # ahead of a row within its own tile
        s = len(pairs) - 1
        new, n = pairs[s]
        for at in (n - 1, n - new + 3, n - new // 2):
            first = S.starts[s] + new - (n - at)     # the first row that sees the key
            for which in ("key", "rotary", "value"):
                T = Setup(torch, pairs, heads, DIMS[0], seed=7)
                row = T.key_starts[s] + at
                if which == "key":
                    T.kv[row, :, :D] = value
                elif which == "rotary":
                    T.r[row] = value
                else:
                    T.kv[row, :, D + 5] = value
                got, got_lse, _ = attend(torch, sz, T)
                assert torch.equal(got[:first], want[:first]), (value, at, which)
                assert torch.equal(got_lse[:first], want_lse[:first]), (value, at, which)
                if which == "value":                 # reaches the rows that see it
                    hit = got[first:, :, 5].float()
                    assert bool(torch.isnan(hit).all() if math.isnan(value)
                                else (hit == value).all()), (value, at)
                    rest = [e for e in range(128) if e != 5]
                    assert torch.equal(got[first:][..., rest], want[first:][..., rest])


def test_strided_and_head_major_tensors(torch, sz):
    S = Setup(torch, [(40, 100), (130, 200)], 4, DIMS[0], seed=8)
    want, want_lse, _ = attend(torch, sz, S)
    k, r, v = S.tensors()
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = sz.Batch(torch.tensor(S.starts, **i32),
                     torch.tensor([n for _, n in S.pairs], **i32), S.n)
    starts = torch.tensor(S.key_starts, **i32)
    major = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (S.q.cuda(), k, v)]
    got, got_lse = sz.attend_expanded(major[0], major[1], major[2], starts, batch, S.scale,
                                      r.contiguous())
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)
    with pytest.raises(ValueError):
        sz.attend_expanded(S.q.cuda(), k, v[:-1], starts, batch, S.scale, r)
    with pytest.raises(ValueError):
        sz.attend_expanded(S.q.cuda(), k, v, starts, batch, S.scale)
    with pytest.raises(sz.SplitZipError):
        sz.attend_expanded(S.q.cuda(), k.float(), v, starts, batch, S.scale, r)


def test_rows_past_32_bits(torch, sz):
    """Keys and values that lie more than 2^32 elements from their tensors' start."""
    n, stride = 70000, (1 << 16) + 8
    pool = torch.empty(n * stride + 512, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(9)
    rows = torch.randn(300, 1, 320, generator=g).bfloat16()
    view = torch.as_strided(pool, (n, 1, 320), (stride, 320, 1))
    view[n - 300:] = rows.cuda()
    q = torch.randn(200, 1, 192, generator=g).bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = sz.Batch(torch.tensor([0, 200], **i32), torch.tensor([300], **i32), 200)
    say("far rows")
    out, lse = sz.attend_expanded(q.cuda(), view[..., :128], view[..., 192:],
                                  torch.tensor([n - 300], **i32), batch, 0.07,
                                  view[..., 128:192], max_len=300)
    want, want_lse, tol, tol_lse = ref.attend(q, rows[..., :192], rows[..., 192:], 300, 0.07)
    assert bool(((out.cpu().double() - want).abs() <= tol).all())
    assert bool(((lse.cpu().double() - want_lse).abs() <= tol_lse).all())


def test_bad_sequences(torch, sz):
    pairs = [(20, 100), (1, 64), (40, 90), (130, 133)]
    S = Setup(torch, pairs, 3, DIMS[0], seed=10)
    want, _, st = attend(torch, sz, S)
    assert st == [0] * 4
    for bad in (-1, S.n_keys - 89, S.n_keys, 2 ** 31 - 1, -2 ** 31):
        starts = list(S.key_starts)
        starts[2] = bad
        out, _, st = attend(torch, sz, S, key_starts=starts)
        assert st == [0, 0, 1, 0], bad
        assert torch.equal(out[:21], want[:21]) and torch.equal(out[61:], want[61:]), bad
    out, _, st = attend(torch, sz, S, lens=[100, -5, 90, 2 ** 31 - 1])
    assert st == [0, 1, 0, 1] and torch.equal(out[:20], want[:20])
    assert torch.equal(out[21:61], want[21:61])
    out, _, st = attend(torch, sz, S, max_len=100)
    assert st == [0, 0, 0, 1] and torch.equal(out[:61], want[:61])
    assert attend(torch, sz, S, starts=[0, 20, 21, 61, 192])[2] == [0, 0, 0, 1]


def test_nothing_to_do(torch, sz):
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = sz.Batch(torch.zeros(3, **i32), torch.zeros(2, **i32), 0)
    new = lambda n, d: torch.zeros(n, 4, d, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    starts = torch.zeros(2, **i32)
    out, lse = sz.attend_expanded(new(0, 192), new(9, 128), new(9, 128), starts, batch, 0.1,
                                  new(9, 64))
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    batch = sz.Batch(torch.tensor([0, 2, 3], **i32), torch.zeros(2, **i32), 3)
    out, lse = sz.attend_expanded(new(3, 192), new(0, 128), new(0, 128), starts, batch, 0.1,
                                  new(0, 64))
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


# ---- together ----------------------------------------------------------------

def test_both_forms_of_latent_attention(torch, sz):
    """A prompt's latents appended in two chunks, the second attended to in the
    expanded form over what the pages hold, then single tokens in the absorbed
    form, captured and replayed; both against the same attention in 64 bits."""
    H, L, R, D, V, page = 6, 256, 32, 64, 64, 16
    g = torch.Generator().manual_seed(20)
    lens, chunk = [150, 61], [100, 40]
    i32 = dict(dtype=torch.int32, device="cuda")
    up_k = (torch.randn(H, D, L, generator=g) * L ** -0.5).bfloat16().double()
    up_v = (torch.randn(H, V, L, generator=g) * L ** -0.5).bfloat16().double()
    ids = torch.randperm(24, generator=g)[:22].view(2, 11)
    pool = torch.zeros(24, page, L + R, dtype=torch.bfloat16, device="cuda")
    cache = sz.latent_cache(pool, ids.cuda(), L)
    rope, weight = sz.rope(R, interleaved=True), 1 + 0.2 * torch.randn(L, generator=g)
    scale = (D + R) ** -0.5

    def append(news, lengths, q=None):
        n = sum(news)
        x = torch.randn(n, 1, L + R, generator=g).bfloat16().cuda()
        starts = torch.tensor([0, news[0], n], **i32)
        batch = sz.Batch(starts, torch.tensor(lengths, **i32), n)
        return batch, sz.latent_append(x[..., :L], cache, batch, x[..., L:], rope, q,
                                       weight.cuda())

    def rows(s, length):
        return pool[ids[s].cuda()].reshape(-1, L + R)[:length]

    def want(q_nope, q_rot, s, length):
        """q_nope [new, H, D], q_rot [new, H, R] in 64 bits."""
        c = rows(s, length).cpu().double()
        k = torch.cat([torch.einsum("hdl,jl->jhd", up_k, c[:, :L]),
                       c[:, None, L:].expand(-1, H, -1)], -1)
        v = torch.einsum("hdl,jl->jhd", up_v, c[:, :L])
        return ref.attend(torch.cat([q_nope, q_rot], -1), k, v, length, scale)

    append(chunk, chunk)
    news = [a - b for a, b in zip(lens, chunk)]
    q = torch.randn(sum(news), H, D + R, generator=g).bfloat16()
    batch, turned = append(news, lens, q[..., D:].contiguous().cuda())
    q[..., D:] = turned.cpu()
    # the expansion, one product over the gathered rows
    c = torch.cat([rows(s, lens[s]) for s in range(2)])
    up = torch.cat([up_k, up_v], 1).float().cuda()                       # [H, D + V, L]
    kv = (c[:, :L].float() @ up.view(-1, L).t()).bfloat16().view(-1, H, D + V)
    out, _ = sz.attend_expanded(q.cuda(), kv[..., :D], kv[..., D:],
                                torch.tensor([0, lens[0]], **i32), batch, scale, c[:, None, L:])
    say("expanded")
    for s in range(2):
        a, b = sum(news[:s]), sum(news[:s + 1])
        w, _, tol, _ = want(q[a:b, :, :D].double(), q[a:b, :, D:].double(), s, lens[s])
        # keys and values have been rounded once more: half a step of each
        k_size = (q[a:b].double().abs().amax() * (D + R) * 4 * ref.U16 * scale)
        assert bool(((out[a:b].cpu().double() - w).abs() <= tol + ref.U16 * 4 + k_size * 4).all())

    # single tokens: queries absorbed, outputs projected back
    batch = sz.Batch(torch.tensor([0, 1, 2], **i32), torch.tensor([x + 1 for x in lens], **i32), 2)
    x = torch.zeros(2, 1, L + R, dtype=torch.bfloat16, device="cuda")
    q_all = torch.zeros(2, H, L + R, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.zeros(2, H, L, device="cuda"), torch.zeros(2, H, device="cuda")
    size = sz.sz_attend_latent_workspace_size(H, cache, batch, 160)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    weight = weight.cuda()

    def step():
        sz.sz_latent_append(x[..., :L], weight, 1e-6, x[..., L:], q_all[..., L:], q_all[..., L:],
                            rope, None, cache, batch)
        sz.sz_attend_latent(q_all, o, lse, cache, batch, 160, scale, True, ws, size)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for replay in range(3):
        q_nope = torch.randn(2, H, D, generator=g).bfloat16().double()
        absorbed = torch.einsum("nhd,hdl->nhl", q_nope, up_k)
        q_all.copy_(torch.cat([absorbed, torch.randn(2, H, R, generator=g).double()], -1))
        x.copy_(torch.randn(2, 1, L + R, generator=g).bfloat16())
        before = q_all.clone()
        graph.replay()
        torch.cuda.synchronize()
        got, got_lse, got_pool, got_q = o.clone(), lse.clone(), pool.clone(), q_all.clone()
        q_all.copy_(before)
        o.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in ((got, o), (got_lse, lse), (got_pool, pool), (got_q, q_all)):
            assert torch.equal(a, b), replay
        say("absorbed", replay)
        for s in range(2):
            n = lens[s] + 1
            K = rows(s, n).cpu()[:, None]
            w, wl, tol, tl = ref.attend(q_all[s:s + 1].cpu(), K, K[..., :L], n, scale,
                                        f32_out=True)
            assert bool(((o[s:s + 1].cpu().double() - w).abs() <= tol).all()), (replay, s)
            assert bool(((lse[s:s + 1].cpu().double() - wl).abs() <= tl).all()), (replay, s)
            # and the same as attention in the heads, but for the absorbed
            # queries' rounding: half a step of L products, in the exponent
            out = torch.einsum("nhl,hdl->nhd", o[s:s + 1].cpu().double(), up_v)
            w, _, _, _ = want(q_nope[s:s + 1], got_q[s:s + 1, :, L:].cpu().double(), s, n)
            size_q = (q_all[s, :, :L].cpu().double().abs()[None] @
                      K[:, 0, :L].double().abs().t()).amax() * scale
            weights = 2 * ref.U16 * size_q + 2 * ref.U16
            biggest = torch.einsum("hdl,jl->jhd", up_v.abs(), K[:, 0, :L].double().abs()).amax()
            assert bool(((out - w).abs() <= weights * biggest).all()), (replay, s)
