"""The caches of latents, the expanded form of their attention, attention weights
and eviction, on a machine without a GPU: the host checks refuse what
include/splitzip.h does not allow before anything touches a device.  No kernel
is launched here."""
import ctypes
import math

import pytest

from test_kv_abi import A, GB, at, batch, cache, heads, rope, sz  # noqa: F401

WS = A + (6 << 40)


class L(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("n", ctypes.c_uint64), ("pitch", ctypes.c_uint64),
                ("token_stride", ctypes.c_uint64), ("latent", ctypes.c_uint32),
                ("rotary", ctypes.c_uint32), ("page", ctypes.c_uint32)]


def latents(**kw):
    d = dict(pages=A + (1 << 40), n=64, pitch=64, token_stride=576, latent=512, rotary=64, page=16)
    d.update(kw)
    return L(**d)


BAD_LATENTS = [
    dict(latent=0), dict(latent=4), dict(latent=516), dict(latent=520, token_stride=584),
    dict(rotary=4), dict(rotary=72, token_stride=584), dict(token_stride=568),
    dict(token_stride=580), dict(token_stride=1 << 26), dict(page=8), dict(page=24),
    dict(page=1 << 17), dict(n=0), dict(pitch=63), dict(pages=None), dict(pages=A + 4),
    dict(pitch=1 << 41),
]
BAD_BATCHES = [dict(seqs=65536), dict(tokens=1 << 31), dict(starts=None), dict(lens=A + 2)]


# ---- appending latents -----------------------------------------------------------
def append(sz, latent=None, w=None, eps=1e-6, k=0, q=None, q_out=None, r=None, pos=None, c=None,
           b=None, status=None):
    latent = latent or heads(n=1, dim=512)
    k = heads(A + GB, n=1, dim=64) if k == 0 else k
    return sz._lib.sz_latent_append(at(latent), w, eps, at(k), at(q), at(q_out), at(r), pos,
                                    at(c or latents()), at(b or batch()), status, None)


def test_append_refuses(sz):
    q = heads(A + 2 * GB, n=16, dim=64)
    out = heads(A + 3 * GB, n=16, dim=64)
    for kw in BAD_LATENTS:
        assert append(sz, c=latents(**kw)) == 1, kw
    for kw in BAD_BATCHES:
        assert append(sz, b=batch(**kw)) == 1, kw
    bad = [
        dict(latent=heads(n=2, dim=512)), dict(latent=heads(0, n=1, dim=512)),
        dict(latent=heads(A + 8, n=1, dim=512)), dict(latent=heads(n=1, dim=512, type=7)),
        dict(latent=heads(n=1, dim=512, token_stride=516)),
        dict(k=None), dict(k=heads(A + GB, n=2, dim=64)), dict(k=heads(A + GB + 4, n=1, dim=64)),
        dict(k=heads(A + GB, n=1, dim=64, type=9)),
        dict(c=latents(rotary=0)),                          # rotary rows of none
        dict(q=q), dict(q_out=out),                         # one without the other
        dict(q=q, q_out=heads(A + 3 * GB, n=15, dim=64)),
        dict(q=q, q_out=heads(A + 3 * GB, n=16, dim=64, type=3)),
        dict(q=q, q_out=heads(A + 2 * GB + 128, n=16, dim=64)),   # across its input
        dict(q=q, q_out=heads(A + 64, n=16, dim=64)),             # over the latents
        dict(q=q, q_out=heads(A + GB, n=16, dim=64)),             # over the keys' rotary parts
        dict(c=latents(rotary=0, token_stride=512), k=None, q=q, q_out=out),
        dict(w=A + GB + 4), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
        dict(pos=A + 2), dict(status=A + 1),
        dict(r=rope(dims=32)), dict(r=rope(dims=128)), dict(r=rope(dims=64, phases=None)),
        dict(r=rope(dims=64, magnitude=math.nan)),
    ]
    for i, kw in enumerate(bad):
        assert append(sz, **kw) == 1, (i, kw)
    # nothing to do: accepted, nothing launched
    none = batch(seqs=0, starts=None, lens=None)
    assert append(sz, b=none) == 0
    assert append(sz, b=none, q=q, q_out=q, r=rope(dims=64)) == 0    # in place
    assert append(sz, b=none, r=rope(dims=0)) == 0
    assert append(sz, b=none, c=latents(rotary=0, token_stride=512), k=None) == 0
    # the rotary parts of queries whose rows the attention reads
    wide = heads(A + 3 * GB + 1024, n=16, dim=64, head_stride=576, token_stride=16 * 576)
    assert append(sz, b=none, q=q, q_out=wide) == 0


# ---- the absorbed form -----------------------------------------------------------
def absorbed(sz, q=None, out=None, lse=None, c=None, b=None, max_len=0, scale=0.1, causal=1,
             ws=WS, bytes=1 << 40, status=None):
    q = q or heads(n=16, dim=576)
    out = out or heads(A + GB, n=16, dim=512)
    return sz._lib.sz_attend_latent(at(q), at(out), lse, at(c or latents()), at(b or batch()),
                                    max_len, scale, causal, ws, bytes, status, None)


def test_absorbed_refuses(sz):
    for kw in BAD_LATENTS:
        assert absorbed(sz, c=latents(**kw)) == 1, kw
    for kw in BAD_BATCHES:
        assert absorbed(sz, b=batch(**kw)) == 1, kw
    bad = [
        dict(q=heads(n=15, dim=576)), dict(q=heads(n=16, dim=576, type=2)),
        dict(q=heads(0, n=16, dim=576)),
        dict(q=heads(A + 8, n=16, dim=576)), dict(q=heads(n=0, dim=576)),
        dict(out=heads(A + GB, n=16, dim=512, type=3)), dict(out=heads(0, n=16, dim=512)),
        dict(out=heads(A + GB, n=16, dim=504)), dict(out=heads(A, n=16, dim=512)),
        dict(out=heads(A + 4096, n=16, dim=512)),
        dict(lse=A), dict(lse=A + GB + 64), dict(lse=A + 2 * GB + 2),
        dict(scale=0.0), dict(scale=-0.1), dict(scale=math.nan), dict(scale=math.inf),
        dict(scale=3e38), dict(status=A + 2),
    ]
    for i, kw in enumerate(bad):
        assert absorbed(sz, **kw) == 1, (i, kw)
    assert absorbed(sz, b=batch(seqs=0, starts=None, lens=None)) == 0
    assert absorbed(sz, q=heads(0, n=16, dim=576), out=heads(0, n=16, dim=512),
                    b=batch(tokens=0)) == 0


def test_absorbed_workspace(sz):
    size = lambda h=16, c=latents(n=4096, pitch=4096), b=batch(seqs=1, tokens=1), m=0: \
        sz._lib.sz_attend_latent_workspace_size(h, at(c), at(b), m)
    need = size()
    assert need > 0 and need == size(m=65536) == size(m=1 << 40)
    assert size(h=0) == 0 and size(c=None) == 0 and size(b=None) == 0
    assert size(b=batch(tokens=0)) == 0 and size(b=batch(seqs=0)) == 0
    assert size(c=latents(latent=516)) == 0
    one = dict(c=latents(n=4096, pitch=4096), b=batch(seqs=1, tokens=1))
    for kw in (dict(ws=None), dict(ws=WS + 16), dict(bytes=need - 1), dict(ws=A),
               dict(ws=A + GB), dict(lse=WS + need - 4), dict(ws=A + 2 * GB, lse=A + 2 * GB)):
        assert absorbed(sz, **one, **kw) == 1, kw


def test_absorbed_refuses_more_than_a_launch(sz):
    def call(seqs, n, tokens):
        c = latents(latent=8, rotary=0, token_stride=8)
        b = batch(seqs=seqs, tokens=tokens)
        assert sz._lib.sz_attend_latent_workspace_size(n, at(c), at(b), 0) == 0
        return absorbed(sz, c=c, b=b, q=heads(A + (1 << 42), n=n, dim=8),
                        out=heads(A + (1 << 45), n=n, dim=8))
    assert call(1, 1 << 10, 1 << 20) == 1          # 2^30 rows: 2^24 halves of tiles
    assert call(1, 1, 1 << 30) == 1
    assert call(65535, 65535, 16384) == 1


# ---- the expanded form -------------------------------------------------------------
def expanded(sz, q=None, out=None, lse=None, k=None, r=0, v=None, dims=(128, 64, 128),
             starts=A + (5 << 40), n_keys=1000, b=None, max_len=0, scale=0.1, causal=1, ws=WS,
             bytes=1 << 40, status=None):
    q = q or heads(n=16, dim=192)
    out = out or heads(A + GB, n=16)
    k = k or heads(A + 2 * GB, n=16)
    v = v or heads(A + 3 * GB, n=16)
    r = heads(A + 4 * GB, n=1, dim=64) if r == 0 else r
    return sz._lib.sz_attend_expanded(at(q), at(out), lse, at(k), at(r), at(v), *dims, starts,
                                      n_keys, at(b or batch()), max_len, scale, causal, ws, bytes,
                                      status, None)


def test_expanded_refuses(sz):
    for kw in BAD_BATCHES:
        assert expanded(sz, b=batch(**kw)) == 1, kw
    big = A + (1 << 44)
    bad = [
        dict(dims=(0, 64, 128)), dict(dims=(136, 64, 128)), dict(dims=(124, 64, 128)),
        dict(dims=(128, 72, 128)), dict(dims=(128, 4, 128)), dict(dims=(128, 64, 0)),
        dict(dims=(128, 64, 136)), dict(dims=(128, 0, 128)), dict(r=None),
        dict(q=heads(n=15, dim=192)), dict(q=heads(n=16, dim=192, type=2)),
        dict(q=heads(A + 8, n=16, dim=192)),
        dict(out=heads(A + GB, n=16, type=3)), dict(out=heads(A, n=16)),
        dict(k=heads(A + 2 * GB, n=8)), dict(k=heads(A + 2 * GB, n=16, type=2)),
        dict(k=heads(0, n=16)), dict(k=heads(A + 2 * GB + 8, n=16)),
        dict(k=heads(big, n=16, token_stride=1 << 26)),
        dict(v=heads(big, n=16, token_stride=1 << 26)),
        dict(v=heads(A + 3 * GB, n=15)), dict(v=heads(A + 3 * GB, n=16, type=2)),
        dict(k=heads(A + GB + 256, n=16)), dict(v=heads(A + GB, n=16)),   # written by the call
        dict(r=heads(A + GB, n=1, dim=64)), dict(r=heads(A + 4 * GB, n=2, dim=64)),
        dict(r=heads(A + 4 * GB, n=1, dim=64, type=2)), dict(r=heads(0, n=1, dim=64)),
        dict(starts=None), dict(starts=A + 2), dict(n_keys=1 << 31),
        dict(lse=A), dict(lse=A + GB), dict(lse=A + 2 * GB), dict(lse=A + 3 * GB),
        dict(lse=A + 4 * GB), dict(lse=A + 5 * GB + 2),
        dict(scale=0.0), dict(scale=math.nan), dict(scale=3e38), dict(status=A + 2),
    ]
    for i, kw in enumerate(bad):
        assert expanded(sz, **kw) == 1, (i, kw)
    none = batch(seqs=0, starts=None, lens=None)
    assert expanded(sz, b=none, starts=None) == 0
    # keys and values as slices of one tensor; a rotary part of every head
    both = dict(n=16, head_stride=256, token_stride=4096)
    assert expanded(sz, b=none, k=heads(A + 2 * GB, **both), v=heads(A + 2 * GB + 256, **both)) == 0
    assert expanded(sz, b=none, r=heads(A + 4 * GB, n=16, dim=64)) == 0
    assert expanded(sz, b=none, r=None, dims=(128, 0, 128), q=heads(n=16)) == 0
    assert expanded(sz, q=heads(0, n=16, dim=192), out=heads(0, n=16), b=batch(tokens=0)) == 0


def test_expanded_workspace(sz):
    size = lambda h=16, v=128, b=batch(seqs=1, tokens=100), m=8192: \
        sz._lib.sz_attend_expanded_workspace_size(h, v, at(b), m)
    need = size()
    assert need > 0 and size(m=0) == size(m=1 << 40)
    for tokens in (1, 100, 1024, 2000):     # with 0: enough for any length
        b = batch(seqs=1, tokens=tokens)
        lengths = [1 << i for i in range(31)] + [777, 1500, 200000]
        assert size(b=b, m=0) == max(size(b=b, m=m) for m in lengths)
    assert size(h=0) == 0 and size(v=12) == 0 and size(v=136) == 0 and size(b=None) == 0
    assert size(b=batch(tokens=0)) == 0 and size(b=batch(seqs=0)) == 0
    one = dict(b=batch(seqs=1, tokens=100), n_keys=8192)
    for kw in (dict(ws=None), dict(ws=WS + 16), dict(bytes=need - 1), dict(ws=A), dict(ws=A + GB),
               dict(ws=A + 2 * GB), dict(ws=A + 3 * GB), dict(ws=A + 4 * GB),
               dict(lse=WS + need - 4)):
        assert expanded(sz, **one, **kw) == 1, kw


def test_expanded_refuses_more_than_a_launch(sz):
    def call(seqs, n, tokens):
        b = batch(seqs=seqs, tokens=tokens)
        assert sz._lib.sz_attend_expanded_workspace_size(n, 8, at(b), 0) == 0
        at_ = [A + (i << 45) for i in range(1, 4)]
        return expanded(sz, q=heads(A + (1 << 42), n=n, dim=8), out=heads(at_[0], n=n, dim=8),
                        k=heads(at_[1], n=n, dim=8), v=heads(at_[2], n=n, dim=8), r=None,
                        dims=(8, 0, 8), b=b)
    assert call(65535, 128, 65535) == 1
    assert call(1, 128, 1 << 24) == 1


# ---- attention weights ---------------------------------------------------------------
def weigh(sz, q=None, lse=A + GB, before=None, w=A + 2 * GB, pitch=1024, keep=1.0, c=None, b=None,
          max_len=0, scale=0.1, cap=0.0, causal=1, window=0, ws=WS, bytes=1 << 40, status=None):
    q = q or heads(n=32)
    return sz._lib.sz_weigh_pages(at(q), lse, before, w, pitch, keep, at(c or cache()),
                                  at(b or batch()), max_len, scale, cap, causal, window, ws, bytes,
                                  status, None)


def test_weigh_refuses(sz):
    for kw in BAD_BATCHES:
        assert weigh(sz, b=batch(**kw)) == 1, kw
    bad = [
        dict(q=heads(n=30)), dict(q=heads(n=32, type=2)), dict(q=heads(0, n=32)),
        dict(q=heads(A + 8, n=32)),
        dict(c=cache(page=24)), dict(c=cache(dim=264, head_stride=264, token_stride=264 * 8)),
        dict(c=cache(k=None)), dict(c=cache(v=None)), dict(c=cache(pitch=63)),
        dict(lse=None), dict(lse=A + GB + 2), dict(before=A + 3 * GB + 1), dict(w=None),
        dict(w=A + 2 * GB + 2), dict(pitch=1023), dict(pitch=1 << 31), dict(pitch=99, max_len=100),
        dict(keep=math.nan), dict(keep=math.inf),
        dict(w=A), dict(w=A + GB), dict(before=A + 2 * GB + 4), dict(before=A + 2 * GB - 4),
        dict(scale=0.0), dict(scale=math.inf), dict(cap=-1.0), dict(cap=math.nan),
        dict(causal=0, window=5), dict(status=A + 2),
    ]
    for i, kw in enumerate(bad):
        assert weigh(sz, **kw) == 1, (i, kw)
    assert weigh(sz, b=batch(seqs=0, starts=None, lens=None)) == 0
    # (what is not read may lie anywhere: checked, and nothing launched)
    assert weigh(sz, b=batch(seqs=0, starts=None, lens=None), lse=None, w=None, ws=None) == 0


def test_weigh_workspace(sz):
    b = batch(seqs=1, tokens=4096)
    size = lambda h=32, c=cache(pages=256, pitch=256), b=b, m=0: \
        sz._lib.sz_weigh_workspace_size(h, at(c), at(b), m)
    need = size()
    assert need > 0 and need == size(m=4096) == size(m=1 << 40)
    assert size(h=30) == 0 and size(h=0) == 0 and size(c=None) == 0 and size(b=None) == 0
    assert size(b=batch(seqs=0)) == 0 and size(b=batch(tokens=0)) == 0
    assert size(c=cache(page=24)) == 0 and size(c=cache(kv_heads=0)) == 0
    one = dict(b=b, c=cache(pages=256, pitch=256), pitch=4096)
    for kw in (dict(ws=None), dict(ws=WS + 16), dict(bytes=need - 1), dict(ws=A), dict(ws=A + GB),
               dict(ws=A + 2 * GB), dict(ws=A + 3 * GB, before=A + 3 * GB)):
        assert weigh(sz, **one, **kw) == 1, kw


@pytest.mark.parametrize("tokens,kv_heads", [(65535, 1024), (1 << 20, 1024), (100, 1024),
                                             (0, 1024), (2000, 65528)])
def test_weigh_refuses_more_than_a_launch(sz, tokens, kv_heads):
    c = cache(kv_heads=kv_heads, dim=8, head_stride=8, token_stride=8 * kv_heads, pages=1 << 20,
              pitch=1 << 20, page=1024)                        # 2^30 positions
    b = batch(seqs=1, tokens=tokens)
    sz._lib.sz_weigh_workspace_size(kv_heads, at(c), at(b), 0)
    q = heads(A, n=kv_heads, dim=8)
    assert weigh(sz, q=q, lse=A + (1 << 42), w=A + (1 << 44), pitch=1 << 30, c=c, b=b) == 1


# ---- eviction ------------------------------------------------------------------------
def evict(sz, w=A, wh=8, pitch=1024, src=None, lens=A + GB, n=3, max_len=0, budget=256, first=4,
          recent=64, dst=None, w_to=A + 2 * GB, kept=A + 3 * GB, lens_to=A + 4 * GB, status=None):
    return sz._lib.sz_evict_pages(w, wh, pitch, at(src or cache()), lens, n, max_len, budget, first,
                                  recent, at(dst or cache()), w_to, kept, lens_to, status, None)


def test_evict_refuses(sz):
    bad = [
        dict(wh=0), dict(wh=2), dict(wh=9), dict(pitch=1023), dict(pitch=1 << 31),
        dict(src=cache(page=24)), dict(dst=cache(page=24)), dict(src=cache(k=None)),
        dict(dst=cache(v=A + 4)), dict(dst=cache(dim=64)), dict(dst=cache(kv_heads=4)),
        dict(n=65536), dict(budget=0), dict(budget=(1 << 30) + 1), dict(first=257),
        dict(first=200), dict(recent=253), dict(recent=1 << 63, first=256),
        dict(first=1 << 63, recent=1 << 63), dict(recent=(1 << 64) - 1),
        dict(dst=cache(pages=15, pitch=15)),                       # no room for 256
        dict(w=None), dict(lens=None), dict(w_to=None), dict(kept=None), dict(lens_to=None),
        dict(w=A + 2), dict(lens=A + GB + 1), dict(w_to=A + 2 * GB + 2), dict(kept=A + 3 * GB + 3),
        dict(lens_to=A + 4 * GB + 2), dict(status=A + 2),
        dict(w_to=A), dict(kept=A + 4), dict(lens_to=A + 8), dict(w_to=A + GB), dict(kept=A + GB),
        dict(lens_to=A + GB), dict(status=A + GB + 4), dict(status=A), dict(kept=A + 2 * GB),
        dict(lens_to=A + 2 * GB), dict(lens_to=A + 3 * GB), dict(status=A + 4 * GB),
        dict(n=1 << 15, wh=128, src=cache(kv_heads=128, token_stride=128 * 128),
             dst=cache(kv_heads=128, token_stride=128 * 128)),     # 2^22 rows of weights
        dict(n=65535, src=cache(pages=1 << 14, pitch=1 << 14), pitch=1 << 18, budget=1 << 12,
             dst=cache(pages=1 << 14, pitch=1 << 14)),             # 2^24 blocks to copy
    ]
    for i, kw in enumerate(bad):
        assert evict(sz, **kw) == 1, (i, kw)
    assert evict(sz, n=0) == 0
    assert evict(sz, n=0, w=None, lens=None, w_to=None, kept=None, lens_to=None) == 0
    assert evict(sz, n=0, wh=1, budget=4096, dst=cache()) == 0     # room for all that there can be


def test_python_layer_refuses(sz):
    import torch
    rows = torch.zeros(4, 16, 72, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sz.LatentCache(torch.zeros(2, 2, dtype=torch.int64), 64, 8, 16)
    with pytest.raises(ValueError):
        sz.latent_cache(rows, torch.zeros(1, 1, dtype=torch.int64), 64)
    with pytest.raises((ValueError, AttributeError)):
        sz.sz_attend_latent(rows, rows, None, None, None, 0, 1.0)
    with pytest.raises(ValueError):
        sz.sz_evict_pages(torch.zeros(2, 2), None, None, None, None, None, 0, 1, 0, 0, None)
