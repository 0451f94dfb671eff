"""Attention of chunks over a paged cache (sz_attend_pages) where tiles have
128 and 256 rows: sampled rows of long calls against the plain 64-bit form,
with the bounds of kv_reference.py."""
import ctypes
import math
import re

import pytest

import kv_reference as ref
from test_gpu_kv import Setup, SENTINEL, say, sz, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def some_rows(n, count, seed, torch):  # noqa: F811
    """Row numbers below n: the first and last, tiles' borders, others at
    random."""
    g = torch.Generator().manual_seed(seed)
    borders = [0, 1, 15, 16, 31, 32, 33, 63, 64, 127, 128, 129, 255, 256, 257, 511, 512, n - 2, n - 1]
    picked = {x for x in borders if 0 <= x < n}
    picked |= set(torch.randint(0, n, (count,), generator=g).tolist())
    return torch.tensor(sorted(picked), dtype=torch.int64)


def run(torch, sz, S, out_type=None, max_len=0, scale=None, **kw):  # noqa: F811
    out = torch.full(S.q.shape, SENTINEL, dtype=out_type or torch.bfloat16, device="cuda")
    lse = torch.full(S.q.shape[:2], SENTINEL, dtype=torch.float32, device="cuda")
    size = sz.sz_attend_workspace_size(S.q.shape[1], S.cache, S.batch, max_len)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    status = torch.full((len(S.pairs),), -1, dtype=torch.int32, device="cuda")
    sz.sz_attend_pages(S.q.cuda(), out, lse, S.cache, S.batch, max_len,
                       S.dim ** -0.5 if scale is None else scale,
                       workspace=ws if size else None, workspace_bytes=size, d_status=status, **kw)
    torch.cuda.synchronize()
    assert status.tolist() == [0] * len(S.pairs)
    assert bool((ws[size:] == 0xFF).all())
    return out.cpu(), lse.cpu()


def check(torch, sz, S, label, count=24, out_type=None, max_len=0, every=1, **kw):  # noqa: F811
    say(label)
    out, lse = run(torch, sz, S, out_type, max_len, **kw)
    covered = torch.zeros(S.n, dtype=torch.bool)
    for s, (new, length) in enumerate(S.pairs):
        a, b = S.starts[s], S.starts[s + 1]
        covered[a:b] = True
        if new == 0 or (s % every and new < 16):
            continue
        rows = some_rows(new, count, s, torch)
        want, want_lse, tol, tol_lse = ref.attend_rows(
            S.q[a + rows], length - new + rows, S.rows(S.k, s), S.rows(S.v, s), length,
            S.dim ** -0.5, f32_out=out_type == torch.float32, **kw)
        got, got_lse = out[a + rows].double(), lse[a + rows].double()
        bad = ~((got - want).abs() <= tol)
        assert not bool(bad.any()), (label, s, rows[bad.nonzero()[0][0]].item(),
                                     float(((got - want).abs() / tol).nan_to_num(1e30).max()))
        empty = torch.isinf(want_lse)
        assert bool((got_lse[empty] == -math.inf).all()) and bool((got[empty] == 0).all()), (label, s)
        off = ((got_lse - want_lse).abs() / tol_lse)[~empty]
        assert bool((off <= 1).all()), (label, s, float(off.max()))
    assert bool((out[~covered] == SENTINEL).all()) and bool((lse[~covered] == SENTINEL).all()), label
    return out, lse


CAPS = [2.0, 30.0, 64.0, 65.0, 1e3, 1e5, 1e6, 1e8, 1e30, 9e37]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("shape", [(8, 2, 64, 16), (8, 2, 128, 16), (4, 1, 96, 32), (4, 1, 256, 64)],
                         ids=str)
@pytest.mark.parametrize("max_len", [0, 1200], ids=["shared out", "whole"])
def test_caps_of_any_size(torch, sz, shape, cap, max_len):  # noqa: F811
    """Long rows, most of whose keys lie in steps that every row sees."""
    pairs = [(200, 1100), (1, 900), (70, 1200)]
    S = Setup(torch, sz, pairs, *shape, seed=50, behind=1)
    if max_len == 0:
        S.ids = torch.cat([S.ids, S.ids.new_full((S.ids.shape[0], 16384 // shape[3]), -1)], 1)
        S.upload()
    check(torch, sz, S, f"cap {cap} {shape} {max_len}", max_len=max_len, softcap=cap,
          out_type=torch.float32)


# ---- tiles of 256 rows: calls of many rows -----------------------------------

class NodeParams(ctypes.Structure):
    _fields_ = [("block", ctypes.c_uint32 * 3), ("extra", ctypes.c_void_p),
                ("func", ctypes.c_void_p), ("grid", ctypes.c_uint32 * 3),
                ("params", ctypes.c_void_p), ("shared", ctypes.c_uint32)]


def kernels(torch, sz, S, **kw):  # noqa: F811
    """What an attention call launches, from a graph that it is captured into:
    ("few" or "chunk", head size compiled for, waves or blocks of 32 rows a
    wave), or ("join",)."""
    q, out = S.q.cuda(), torch.zeros(S.q.shape, dtype=torch.bfloat16, device="cuda")
    size = sz.sz_attend_workspace_size(S.q.shape[1], S.cache, S.batch)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        sz.sz_attend_pages(q, out, None, S.cache, S.batch, 0, S.dim ** -0.5, workspace=ws,
                           workspace_bytes=size, **kw)
    hip = ctypes.CDLL(next(x.split()[-1] for x in open("/proc/self/maps") if "libamdhip64" in x))
    hip.hipKernelNameRefByPtr.restype = ctypes.c_char_p
    hip.hipKernelNameRefByPtr.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    raw, count = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert hip.hipGraphGetNodes(raw, None, ctypes.byref(count)) == 0
    nodes = (ctypes.c_void_p * count.value)()
    assert hip.hipGraphGetNodes(raw, nodes, ctypes.byref(count)) == 0
    found = []
    for node in nodes:
        p = NodeParams()
        assert hip.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        name = hip.hipKernelNameRefByPtr(p.func, None).decode()
        kind = re.search(r"k_attend_(few|chunk|join)(?:I|<)(?:Li)?(\d+)(?:E(?:Li)?|, )?(\d*)", name)
        assert kind, name
        found.append(("join",) if kind[1] == "join" else (kind[1], int(kind[2]), int(kind[3])))
    return found


# (new tokens, cached length): two chunks whose rows end inside a tile, a short
# sequence whose first rows see nothing, one without tokens
RAGGED = [(37, 20), (2101, 2101), (0, 0), (3377, 3877)]
LARGE = [  # heads, kv_heads, dim, page
    (64, 16, 64, 16), (64, 16, 128, 64), (64, 16, 72, 32), (64, 16, 96, 16), (48, 16, 128, 16),
]
MASKS = [dict(), dict(window=1), dict(window=100), dict(window=1000), dict(causal=False),
         dict(softcap=30.0), dict(softcap=200.0, window=300)]


@pytest.mark.parametrize("shape", LARGE, ids=str)
@pytest.mark.parametrize("kw", MASKS, ids=str)
def test_large_tiles(torch, sz, shape, kw):  # noqa: F811
    S = Setup(torch, sz, RAGGED, *shape, tokens_first=shape[3] != 32, seed=51, before=1, behind=2)
    check(torch, sz, S, f"large tiles {shape} {kw}", **kw)
    assert kernels(torch, sz, S, **kw) == [("chunk", 64 if shape[2] <= 64 else 128, 2)]


def test_large_tiles_f32_output_and_growing_scores(torch, sz):  # noqa: F811
    """Keys that grow along the sequence: the running maximum of both blocks
    of 32 rows moves in every step."""
    S = Setup(torch, sz, [(2700, 3000)], 64, 16, 128, 64, seed=52)
    S.q = S.q.abs()
    page = ref.page_view(S.k, S.shape, True)
    for j in range(3000):
        page[S.ids[0, j // 64], j % 64] = 0.01 * j / 128 ** 0.5
    S.upload()
    check(torch, sz, S, "growing, large tiles", out_type=torch.float32)


@pytest.mark.parametrize("dim", [64, 96, 128])
def test_large_tiles_and_unseen_content(torch, sz, dim):  # noqa: F811
    """NaN and infinities ahead of a row in its own tile, before its window,
    past the length: no effect, bit for bit; on the rows that see them, their
    own."""
    window = 700
    pairs = [(2200, 2300), (64, 64)]
    at = 1333                                  # a position inside a tile
    first = pairs[0][1] - pairs[0][0]

    def setup():
        return Setup(torch, sz, pairs, 64, 16, dim, 16, seed=53)
    S = setup()
    want, want_lse = run(torch, sz, S, window=window)
    assert kernels(torch, sz, S, window=window) == [("chunk", 64 if dim == 64 else 128, 2)]
    blind = torch.ones(S.n, dtype=torch.bool)  # rows that do not see the position
    blind[at - first:at - first + window] = False
    for value in (math.nan, math.inf, -math.inf):
        say("large tiles, unseen", dim, value)
        T = setup()
        for pool in (T.k, T.v):
            ref.page_view(pool, T.shape, True)[T.ids[0, at // 16], at % 16] = value
            # past the lengths, and in pages of no sequence
            page = ref.page_view(pool, T.shape, True)
            page[T.ids[0, 2300 // 16], 2300 % 16:] = value
            used = torch.zeros(pool.shape[0], dtype=torch.bool)
            used[T.ids[T.ids >= 0]] = True
            page[~used] = value
        T.upload()
        got, got_lse = run(torch, sz, T, window=window)
        assert torch.equal(got[blind], want[blind]) and torch.equal(got_lse[blind], want_lse[blind])
        # one element of a value alone: that element of the rows that see it
        T = setup()
        ref.page_view(T.v, T.shape, True)[T.ids[0, at // 16], at % 16, :, 5] = value
        T.upload()
        got, got_lse = run(torch, sz, T, window=window)
        assert torch.equal(got_lse, want_lse)
        assert torch.equal(got[blind], want[blind])
        rest = [d for d in range(dim) if d != 5]
        assert torch.equal(got[:, :, rest], want[:, :, rest])
        hit = got[~blind][:, :, 5].float()
        assert bool(torch.isnan(hit).all() if math.isnan(value) else (hit == value).all())


@pytest.mark.parametrize("case", [
    ("few", 64, [(1, 20 + i * 7 % 50) for i in range(2048)]),            # a large decode batch
    ("few", 32, [(4, 20 + i * 7 % 50) for i in range(1024)]),            # drafts
    ("chunk", 32, [(8, 20 + i * 7 % 50) for i in range(512)]),
    ("chunk", 32, [(1, 40)] * 60 + [(4090, 4090)] + [(1, 70)] * 40),     # decodes and a prompt
], ids=["tokens", "drafts", "more rows", "mixed"])
def test_short_sequences_keep_small_tiles(torch, sz, case):  # noqa: F811
    """Tiles of 256 rows are for sequences that fill them, not for calls that
    have many rows in all."""
    kind, heads, pairs = case
    # (no spare rows: they count among a call's, and drafts have just 16 a tile)
    S = Setup(torch, sz, pairs, heads, 8, 128, 16, seed=54)
    check(torch, sz, S, f"{kind} {len(pairs)}", every=29)
    assert kernels(torch, sz, S) == [(kind, 128, 4 if kind == "few" else 1)]


def test_slices_of_every_head(torch, sz):  # noqa: F811
    """Queries, keys and outputs side by side in every head of one tensor."""
    g = torch.Generator().manual_seed(55)
    n, H, D = 150, 4, 64
    x = torch.randn(n, H, 3, D, generator=g).bfloat16().cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    rope, w = sz.rope(D), 1 + 0.2 * torch.randn(D, generator=g).cuda()
    want = sz.qk_norm_rope(x[:, :, 0].contiguous(), x[:, :, 1].contiguous(), pos, rope, w, w)
    y = x.clone()
    q, k = y[:, :, 0], y[:, :, 1]
    sz.sz_qk_norm_rope(q, q, w, k, k, w, D, n, pos, 1e-6, rope)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(y[:, :, 2], x[:, :, 2])
    pool = torch.randn(2, 10, 16, H, D, generator=g).bfloat16().cuda()
    cache = sz.paged_cache(pool[0], pool[1], torch.arange(10, device="cuda").view(1, -1))
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = sz.Batch(torch.tensor([0, n], **i32), torch.tensor([n], **i32), n)
    want, _ = sz.attend_pages(q.contiguous(), cache, batch, max_len=n)
    size = sz.sz_attend_workspace_size(H, cache, batch, n)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    sz.sz_attend_pages(q, y[:, :, 2], None, cache, batch, n, D ** -0.5, workspace=ws,
                       workspace_bytes=size)
    assert torch.equal(y[:, :, 2], want)


def test_sizes_that_would_be_cut(torch, sz):  # noqa: F811
    """Sizes outside their C type are refused, not taken modulo 2^32 or 2^64."""
    S = Setup(torch, sz, [(1, 100), (20, 300)], 8, 2, 64, 16, seed=56)
    tables = S.cache._keep[:2]
    for kw in (dict(kv_heads=2 ** 32 + 2), dict(head_dim=2 ** 32 + 64), dict(page_tokens=2 ** 32 + 16),
               dict(page_tokens=-16), dict(token_stride=2 ** 64 + 128), dict(head_stride=-64)):
        args = dict(kv_heads=2, head_dim=64, page_tokens=16)
        args.update(kw)
        with pytest.raises(ValueError):
            sz.KVCache(*tables, **args)
    starts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for n in (-1, 2 ** 64 + 1):
        with pytest.raises(ValueError):
            sz.Batch(starts, starts[:1], n)
    q = S.q.cuda()
    for kw in (dict(window=-1), dict(window=2 ** 64 + 5), dict(max_len=-1), dict(max_len=2 ** 64 + 300)):
        with pytest.raises(ValueError):
            sz.attend_pages(q, S.cache, S.batch, **kw)
    out = torch.zeros_like(q)
    for size in (-1, 2 ** 64):
        with pytest.raises(ValueError):
            sz.sz_attend_pages(q, out, None, S.cache, S.batch, 0, 0.1, workspace=None,
                               workspace_bytes=size)
    with pytest.raises(ValueError):
        sz.sz_attend_workspace_size(2 ** 64 + 8, S.cache, S.batch)
    with pytest.raises(ValueError):
        sz.sz_attend_workspace_size(8, S.cache, S.batch, -1)


@pytest.mark.parametrize("new,length", [(1, 300), (1, 5000), (200, 300), (200, 5000)])
def test_ends_of_the_range(torch, sz, new, length):  # noqa: F811
    """Values of 2^127 / 2^8 / keys, scores of 2^28 and scores that are all
    -infinity (rows that see equal keys: the output is the value, to the
    weights' rounding and the output's, the log-sum the score plus ln keys to
    FP32's steps at that size)."""
    S = Setup(torch, sz, [(new, length)], 8, 2, 64, 16, seed=57)
    S.q.fill_(1.0)
    for key, value in ((0.0, 2.0 ** 127 / 2 ** 8 / 8192), (2.0 ** 28 / 8, 3.0), (-math.inf, 3.0)):
        S.k.fill_(key)
        S.v.fill_(value)
        S.upload()
        out, lse = run(torch, sz, S)
        out, lse = out.double(), lse.double()
        say("ends", new, length, key, value)
        if key == -math.inf:
            assert bool((out == 0).all()) and bool((lse == -math.inf).all())
            continue
        assert bool(((out - value).abs() <= value * (2 * ref.U16 + ref.U16 ** 2 + 2.0 ** -12)).all())
        n = torch.arange(length - new, length)[:, None] + 1.0
        want = key * 8 + n.double().log()
        assert bool(((lse - want).abs() <= 8 * ref.U32 * want.abs() + 2.0 ** -16).all())
