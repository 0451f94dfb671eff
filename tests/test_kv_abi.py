"""The operators on a paged cache, on a machine without a GPU: their host
checks refuse what include/splitzip.h does not allow before anything touches
a device, and the rotation's frequencies and phases match their formulas.
No kernel is launched here."""
import ctypes
import math
from fractions import Fraction

import pytest

A = 0x7F0000000000  # fake device addresses: never dereferenced


@pytest.fixture(scope="module")
def sz():
    import lossless_bf16_kv_split_amd as m
    return m


class H(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("heads", ctypes.c_uint64),
                ("token_stride", ctypes.c_uint64), ("head_stride", ctypes.c_uint64),
                ("type", ctypes.c_uint32)]


class C(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_uint64),
                ("pitch", ctypes.c_uint64), ("token_stride", ctypes.c_uint64),
                ("head_stride", ctypes.c_uint64), ("kv_heads", ctypes.c_uint32),
                ("dim", ctypes.c_uint32), ("page", ctypes.c_uint32)]


class B(ctypes.Structure):
    _fields_ = [("starts", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("seqs", ctypes.c_uint64),
                ("tokens", ctypes.c_uint64)]


class R(ctypes.Structure):
    _fields_ = [("phases", ctypes.c_void_p), ("dims", ctypes.c_uint32),
                ("interleaved", ctypes.c_uint32), ("magnitude", ctypes.c_float)]


def heads(at=A, n=8, dim=128, type=1, **kw):
    d = dict(data=at, heads=n, token_stride=n * dim, head_stride=dim, type=type)
    d.update(kw)
    return H(**d)


def cache(**kw):
    d = dict(k=A + (1 << 40), v=A + (2 << 40), pages=64, pitch=64, token_stride=1024,
             head_stride=128, kv_heads=8, dim=128, page=16)
    d.update(kw)
    return C(**d)


def batch(**kw):
    d = dict(starts=A + (3 << 40), lens=A + (4 << 40), seqs=3, tokens=10)
    d.update(kw)
    return B(**d)


def rope(**kw):
    d = dict(phases=A + (5 << 40), dims=128, interleaved=0, magnitude=1.0)
    d.update(kw)
    return R(**d)


def at(x):
    return None if x is None else ctypes.byref(x)  # keeps x alive


GB = 1 << 30


def attend(sz, q=None, out=None, lse=None, c=None, b=None, max_len=0, scale=0.1, cap=0.0,
           causal=1, window=0, ws=A + (6 << 40), bytes=1 << 40, status=None):
    q = q or heads(n=32)
    out = out or heads(A + GB, n=32)
    return sz._lib.sz_attend_pages(at(q), at(out), lse, at(c or cache()), at(b or batch()),
                                   max_len, scale, cap, causal, window, ws, bytes, status, None)


def test_attend_refuses(sz):
    bad = [
        dict(q=heads(n=30), out=heads(A + GB, n=30)),               # not a multiple of kv_heads
        dict(q=heads(n=16)),                                        # as many as out
        dict(q=heads(n=32, type=2)),                                # BF16 queries only
        dict(out=heads(A + GB, n=32, type=3)),
        dict(q=heads(A + 8, n=32)),                                 # misaligned
        dict(q=heads(0, n=32)),
        dict(q=heads(n=32, token_stride=4100)),                     # strides of 8 elements
        dict(out=heads(A + GB, n=32, token_stride=4088)),           # rows overlap
        dict(out=heads(A + GB, n=32, head_stride=120)),
        dict(out=heads(A + 4096, n=32)),                            # on the queries
        dict(out=heads(A, n=32)),                                   # in place
        dict(lse=A + GB), dict(lse=A + 64), dict(lse=A + 2 * GB + 2),
        dict(c=cache(page=24)), dict(c=cache(page=8)), dict(c=cache(page=1 << 17)),
        dict(c=cache(dim=264, head_stride=264, token_stride=264 * 8)),
        dict(c=cache(dim=4)), dict(c=cache(dim=0)), dict(c=cache(kv_heads=0)),
        dict(c=cache(head_stride=64)), dict(c=cache(token_stride=1016)),
        dict(c=cache(token_stride=1 << 33)), dict(c=cache(token_stride=1 << 26)),
        dict(b=batch(tokens=(1 << 26) + 1), q=heads(n=32), out=heads(A + (1 << 45), n=32)),
        dict(b=batch(seqs=65535), c=cache(kv_heads=65528, token_stride=65528 * 128),
             q=heads(n=65528), out=heads(A + (1 << 45), n=65528)),
        dict(c=cache(pages=0)), dict(c=cache(pitch=63)),
        dict(c=cache(k=None)), dict(c=cache(v=A + 4)),
        dict(b=batch(seqs=65536)), dict(b=batch(tokens=1 << 31)),
        dict(b=batch(starts=None)), dict(b=batch(lens=A + 2)),
        dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan),
        dict(cap=-1.0), dict(cap=math.nan), dict(cap=math.inf), dict(cap=1e-38, scale=1.0),
        dict(scale=3e38),
        dict(causal=0, window=5), dict(status=A + 2),
    ]
    for kw in bad:
        assert attend(sz, **kw) == 1, kw
    # nothing to do: accepted, nothing launched
    assert attend(sz, b=batch(seqs=0, starts=None, lens=None)) == 0
    assert attend(sz, q=heads(0, n=32), out=heads(0, n=32), b=batch(tokens=0)) == 0


def test_attend_workspace_checks(sz):
    c, b = cache(pages=4096, pitch=4096), batch(seqs=1, tokens=1)
    size = sz._lib.sz_attend_workspace_size(32, at(c), at(b), 0)
    assert size == sz._lib.sz_attend_workspace_size(32, at(c), at(b), 65536)
    assert sz._lib.sz_attend_workspace_size(30, at(c), at(b), 0) == 0
    assert size == sz._lib.sz_attend_workspace_size(32, at(c), at(b), 1 << 40)
    assert sz._lib.sz_attend_workspace_size(32, None, at(b), 0) == 0
    assert sz._lib.sz_attend_workspace_size(32, at(c), None, 0) == 0
    assert sz._lib.sz_attend_workspace_size(32, at(c), at(batch(tokens=0)), 0) == 0
    if size:
        for kw in (dict(ws=None), dict(ws=A + (6 << 40) + 16), dict(bytes=size - 1),
                   dict(ws=A), dict(ws=A + GB)):
            assert attend(sz, c=c, b=b, **kw) == 1, kw


def append(sz, k=None, v=None, kw=None, q=None, q_out=None, qw=None, eps=1e-6, r=None, pos=None,
           c=None, b=None, status=None):
    k, v = k or heads(), v or heads(A + GB)
    return sz._lib.sz_kv_append(at(k), at(v), kw, at(q), at(q_out), qw, eps, at(r), pos,
                                at(c or cache()), at(b or batch()), status, None)


def test_append_refuses(sz):
    q, out = heads(A + 2 * GB, n=32), heads(A + 3 * GB, n=32)
    bad = [
        dict(k=heads(n=4)), dict(v=heads(A + GB, n=16)), dict(k=heads(type=0)),
        dict(k=heads(A + 4)), dict(k=heads(head_stride=124)),
        dict(kw=A + 8), dict(q=q), dict(q_out=out),
        dict(q=q, q_out=heads(A + 3 * GB, n=16)),
        dict(q=q, q_out=heads(A + 3 * GB, n=32, type=2)),
        dict(q=q, q_out=heads(A + 1024, n=32)),                  # on the keys
        dict(q=q, q_out=heads(A + GB - 4096, n=32)),             # on the values
        dict(q=q, q_out=heads(A + 2 * GB + 2048, n=32)),         # on itself, shifted
        dict(q=heads(A + 2 * GB, n=32, type=2), q_out=heads(A + 2 * GB, n=32)),
        dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
        dict(r=rope(dims=12)), dict(r=rope(dims=136)), dict(r=rope(phases=None)),
        dict(r=rope(phases=A + 4)), dict(r=rope(interleaved=2)), dict(r=rope(magnitude=math.inf)),
        dict(pos=A + 2), dict(status=A + 1), dict(c=cache(page=0)), dict(b=batch(tokens=1 << 31)),
    ]
    for kw in bad:
        assert append(sz, **kw) == 1, kw
    assert append(sz, b=batch(seqs=0, starts=None, lens=None)) == 0
    assert append(sz, b=batch(tokens=0)) == 0


def test_norm_rope_refuses(sz):
    def call(q=heads(A, n=32), qo=heads(A + GB, n=32), qw=None, k=heads(A + 2 * GB),
             ko=heads(A + 3 * GB), kw=None, dim=128, n=10, pos=A + (7 << 40), eps=1e-6, r=None):
        return sz._lib.sz_qk_norm_rope(at(q), at(qo), qw, at(k), at(ko), kw, dim, n, pos, eps,
                                       at(r), None)
    bad = [
        dict(q=None), dict(ko=None), dict(q=None, qo=None, k=None, ko=None),
        dict(dim=0), dict(dim=12), dict(dim=264), dict(n=1 << 31), dict(qw=A + 4),
        dict(qo=heads(A + GB, n=8)), dict(qo=heads(A + GB, n=32, type=2)),
        dict(ko=heads(A + GB)),                                  # both outputs in one place
        dict(ko=heads(A)),                                       # the keys on the queries
        dict(qo=heads(A + 2 * GB, n=32)),
        dict(qo=heads(A + 256, n=32)),
        dict(r=rope(), pos=None), dict(r=rope(), pos=A + 2), dict(r=rope(dims=132)), dict(eps=-1.0),
        dict(ko=heads(A + 3 * GB, token_stride=1000)),
    ]
    for kw in bad:
        assert call(**kw) == 1, kw
    assert call(n=0) == 0
    # slices of one fused projection do not collide, rows that reach into
    # the next slice do
    fused = dict(token_stride=48 * 128)
    q, k = heads(A, n=32, **fused), heads(A + 32 * 256, **fused)
    assert call(q=q, qo=q, k=k, ko=k, n=0) == 0
    assert call(q=q, qo=q, k=k, ko=heads(A + 31 * 256, **fused)) == 1


def test_python_layer_refuses(sz):
    import torch
    cpu = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sz.Heads(cpu)
    with pytest.raises(ValueError):
        sz.Batch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        sz.KVCache(torch.zeros(2, 2, dtype=torch.int64), torch.zeros(2, 2, dtype=torch.int64),
                   8, 128, 16)
    with pytest.raises(ValueError):
        sz.Rope(torch.zeros(64, dtype=torch.int64))
    with pytest.raises(ValueError):
        sz.paged_cache(cpu.view(1, 4, 8, 128), cpu.view(1, 4, 8, 128),
                       torch.zeros(1, 1, dtype=torch.int64))


def test_rope_phases_are_the_fraction_of_a_turn(sz):
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    freq = [0.0, 1.0, 0.5, 1e-9, 6.283185307179586, 7.0, -0.25, 123.456, 2.0 ** -70]
    for f, got in zip(freq, sz.sz_rope_phases(freq)):
        t = Fraction(f) / (2 * pi)
        want = (t - math.floor(t)) * 2 ** 64
        # a long double holds the turns to 64 bits (half a unit of its last
        # place, above one turn scaled by the turns), then the fraction is
        # rounded once
        off = abs(got - want)
        off = min(off, 2 ** 64 - off)
        assert off <= 2 + 2 * abs(t), (f, got)
    for bad in (math.inf, math.nan):
        with pytest.raises(sz.SplitZipError):
            sz.sz_rope_phases([bad])


def test_rope_frequencies(sz):
    f, m = sz.sz_rope_frequencies(64, 10000.0)
    assert m == 1.0
    for i, x in enumerate(f):
        assert math.isclose(x, 10000.0 ** (-2 * i / 64), rel_tol=1e-14)
    g, m = sz.sz_rope_frequencies(64, 10000.0, sz.SZ_ROPE_LINEAR, 4.0)
    assert all(math.isclose(a, b / 4, rel_tol=1e-14) for a, b in zip(g, f)) and m == 1.0
    # BASE: the slowest pair turns exactly `factor` times slower
    g, m = sz.sz_rope_frequencies(64, 10000.0, sz.SZ_ROPE_BASE, 4.0)
    assert g[0] == 1.0 and math.isclose(g[-1], f[-1] / 4, rel_tol=1e-12)
    # RAMP: ends kept and stretched, a line in between, the magnitude
    g, m = sz.sz_rope_frequencies(64, 10000.0, sz.SZ_ROPE_RAMP, 4.0, 4096.0)
    assert math.isclose(m, 0.1 * math.log(4.0) + 1, rel_tol=1e-6)
    pair = [64 * math.log(4096 / (t * 2 * math.pi)) / (2 * math.log(10000.0)) for t in (32.0, 1.0)]
    low, high = math.floor(pair[0]), math.ceil(pair[1])
    for i, (x, y) in enumerate(zip(g, f)):
        share = min(1.0, max(0.0, (i - low) / (high - low)))
        assert math.isclose(x, y * (1 - share) + y / 4 * share, rel_tol=1e-12), i
    # BANDS: by turns in original_len positions
    g, m = sz.sz_rope_frequencies(128, 500000.0, sz.SZ_ROPE_BANDS, 8.0, 8192.0, 1.0, 4.0)
    assert m == 1.0
    f, _ = sz.sz_rope_frequencies(128, 500000.0)
    kinds = set()
    for x, y in zip(g, f):
        turns = 8192 * y / (2 * math.pi)
        kinds.add((turns > 4) - (turns < 1))
        share = min(1.0, max(0.0, (turns - 1) / 3))
        assert math.isclose(x, share * y + (1 - share) * y / 8, rel_tol=1e-12)
    assert kinds == {-1, 0, 1}
    for bad in ((63, 1e4), (0, 1e4), (64, 1.0), (64, math.inf), (64, 1e4, 5), (64, 1e4, -1),
                (64, 1e4, 1, 0.5), (64, 1e4, 1, math.nan), (2, 1e4, 2, 2.0),
                (64, 1e4, 3, 2.0, 0.0), (64, 1e4, 3, 2.0, 4096.0, 0.0), (64, 1e4, 4, 2.0, 4096.0, 4.0, 1.0)):
        with pytest.raises(sz.SplitZipError):
            sz.sz_rope_frequencies(*bad)


def test_attend_refuses_more_than_a_launch(sz):
    def call(seqs, kv_heads, tokens):
        c = cache(kv_heads=kv_heads, dim=8, head_stride=8, token_stride=8 * kv_heads)
        b = batch(seqs=seqs, tokens=tokens)
        h = dict(n=kv_heads, head_stride=8, token_stride=8 * kv_heads)
        assert sz._lib.sz_attend_workspace_size(kv_heads, at(c), at(b), 0) == 0
        return attend(sz, c=c, b=b, q=heads(A + (1 << 42), **h), out=heads(A + (1 << 45), **h))
    assert call(65535, 128, 65535) == 1
    assert call(1, 128, 1 << 24) == 1


@pytest.mark.parametrize("dims", [0, -2, -128, 2 ** 32 + 2])
def test_rope_frequencies_of_impossible_sizes(sz, dims):
    with pytest.raises(sz.SplitZipError):
        sz.sz_rope_frequencies(dims, 10000.0)
    with pytest.raises(sz.SplitZipError):
        sz.rope(dims)


def test_slices_that_interleave_head_by_head(sz):
    """Queries and keys (and more) side by side in every head of one tensor
    lie apart, as slices of its tokens do; rows that reach into the next
    slice do not."""
    def call(q, k):  # (no sequences: checked, and nothing launched)
        return append(sz, k=k, v=heads(A + GB), q=q, q_out=q,
                      b=batch(seqs=0, starts=None, lens=None))
    step = dict(n=8, head_stride=3 * 128, token_stride=24 * 128)
    assert call(heads(A + 256, **step), heads(A, **step)) == 0
    assert call(heads(A, **step), heads(A + 512, **step)) == 0
    assert call(heads(A + 256 + 768 * 3, **step), heads(A, **step)) == 0    # some heads further on
    assert call(heads(A + 128, **step), heads(A, **step)) == 1              # reaches into it
    assert call(heads(A + 640, **step), heads(A, **step)) == 1              # into the next head's
    odd = dict(n=8, head_stride=3 * 128, token_stride=25 * 128)             # spare room in a token
    assert call(heads(A + 256, **odd), heads(A, **odd)) == 0
    assert call(heads(A + 256 + 768 * 3, **odd), heads(A, **odd)) == 1      # into the next token's
    assert call(heads(A + 256, n=8, head_stride=256, token_stride=24 * 128), heads(A, **step)) == 1


def test_neither_queries_nor_keys(sz):
    with pytest.raises(ValueError):
        sz.qk_norm_rope(None, None, None)
