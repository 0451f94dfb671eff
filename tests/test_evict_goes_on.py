"""Eviction step after step: the weights of the tokens that stay are what the
next step's weights are added to (sz_evict_pages_pitched, evict_pages with
room), every step against 64 bits."""
import sys

import pytest

import kv_reference as ref
from test_gpu_evict import pick, weights_of
from test_gpu_kv import Setup
from test_latent_abi import A, GB, at, cache, evict, sz as host_sz  # noqa: F401

SENTINEL = 768.0


def say(*a):
    print("[evict-goes-on]", *a, flush=True)
    sys.stdout.flush()


def pitched(sz, w=A, wh=8, pitch=1024, lens=A + GB, n=3, budget=256, w_to=A + 2 * GB, to_pitch=300,
            kept=A + 3 * GB, lens_to=A + 4 * GB, status=None, dst=None):
    return sz._lib.sz_evict_pages_pitched(w, wh, pitch, at(cache()), lens, n, 0, budget, 4, 64,
                                          at(dst or cache()), w_to, to_pitch, kept, lens_to,
                                          status, None)


def test_pitched_refuses(host_sz):
    for kw in (dict(to_pitch=255), dict(to_pitch=0), dict(to_pitch=1 << 31),
               dict(to_pitch=(1 << 64) - 1), dict(budget=0, to_pitch=0), dict(wh=2),
               dict(w_to=None), dict(w_to=A + 2 * GB + 2), dict(kept=None),
               # the last row's weights, at 23 rows of 300, reach what is behind them
               dict(kept=A + 2 * GB + 4 * (23 * 300 + 255)),
               dict(lens_to=A + 2 * GB + 4 * (23 * 300 + 255)),
               dict(status=A + 2 * GB + 4 * (23 * 300 + 255)), dict(w_to=A),
               dict(w_to=A - 4 * (23 * 300 + 255)), dict(w_to=A + GB),
               dict(n=65536), dict(dst=cache(kv_heads=4))):
        assert pitched(host_sz, **kw) == 1, kw
    assert pitched(host_sz, n=0) == 0
    assert evict(host_sz, n=0) == 0


def test_python_layer_refuses(host_sz):
    import torch
    with pytest.raises(ValueError):
        host_sz.sz_evict_pages_pitched(torch.zeros(2, 2), None, 1, None, None, None, None, 0, 1, 0,
                                       0, None)
    for pitch in (-1, 1 << 64):
        with pytest.raises(ValueError):
            host_sz.sz_evict_pages_pitched(torch.zeros(2, 2, 4), None, pitch, None, None, None,
                                           None, 0, 1, 0, 0, None)
    with pytest.raises(ValueError):
        host_sz.evict_pages(torch.zeros(2, 2, 4), None, None, torch.zeros(2), 3, room=2)


# ---- on the GPU -----------------------------------------------------------------

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


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [1, 3])
def test_rows_between_are_left(torch, sz, heads):
    """Rows of weights some entries apart, all else around them as it was; the
    same tokens and weights as without."""
    lens, budget = [0, 5, 40, 300, 131], 40
    S = Setup(torch, sz, [(0, n) for n in lens], 3, 3, 64, 16, seed=3)
    g = torch.Generator().manual_seed(4)
    w = torch.rand(len(lens), heads, 310, generator=g).cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    results = []
    for pitch in (40, 41, 64, 777):
        D = Setup(torch, sz, [(0, min(x, budget)) for x in lens], 3, 3, 64, 16, seed=5,
                  fill=SENTINEL)
        out = torch.full((len(lens), heads, pitch), SENTINEL, device="cuda")
        kept = torch.full((len(lens), heads, budget), 99, dtype=torch.int32, device="cuda")
        lens_to, status = torch.zeros_like(n), torch.full_like(n, -1)
        sz.sz_evict_pages_pitched(w, out, pitch, S.cache, D.cache, n, lens_to, 304, budget, 2, 8,
                                  kept, status)
        torch.cuda.synchronize()
        assert status.tolist() == [0] * len(lens) and lens_to.tolist() == [0, 5, 40, 40, 40]
        for s, stay in enumerate(lens_to.tolist()):
            assert bool((out[s, :, stay:] == SENTINEL).all()), (pitch, s)
            for h in range(heads):
                want = pick(w[s, h, :lens[s]].tolist(), lens[s], budget, 2, 8)
                assert kept[s, h, :stay].tolist() == want
                assert torch.equal(out[s, h, :stay], w[s, h, want])
        results.append((out[..., :budget].clone(), kept, D.kd, D.vd))
    for x in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(x, results[0]))
    with pytest.raises(ValueError):                   # one entry short
        sz.sz_evict_pages_pitched(w, out.flatten()[:(len(lens) * heads - 1) * 64 + 39], 64,
                                  S.cache, D.cache, n, lens_to, 304, budget, 2, 8, kept)


def expect(S, starts, lens, q, lse, keys, before, keep):
    """What weigh_pages should leave: per sequence [KH, length] and bound."""
    for s, length in enumerate(lens):
        a, b = starts[s], starts[s + 1]
        want, tol = weights_of(q[a:b], lse[a:b], keys[s], length, S.dim ** -0.5)
        if before is not None:
            old = length - (b - a)
            part = before[s, :, :old].double() * keep
            want[:, :old] += part
            tol[:, :old] += 2 * ref.U32 * (part.abs() + want[:, :old])
        yield s, length, want, tol


@pytest.mark.gpu
def test_heads_with_tokens_of_their_own(torch, sz):
    """A prompt, cut; five tokens, each weighed on top of what stayed; cut
    again, into the first pages."""
    H, KH, D, page, budget, keep = 8, 2, 64, 16, 96, 0.9
    pairs = [(3, 300), (1, 90), (40, 150)]
    S = Setup(torch, sz, pairs, H, KH, D, page, seed=40)
    T = Setup(torch, sz, [(1, min(n, budget) + 5) for _, n in pairs], H, KH, D, page, seed=41,
              fill=0.0)
    g = torch.Generator().manual_seed(42)
    i32 = dict(dtype=torch.int32, device="cuda")
    room = T.cache.pages_per_seq * page
    _, lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch)
    weights = sz.weigh_pages(S.q.cuda(), lse, S.cache, S.batch)
    keys = [S.rows(S.k, s) for s in range(3)]
    for s, n, want, tol in expect(S, S.starts, [n for _, n in pairs], S.q, lse.cpu(), keys, None,
                                  1.0):
        assert bool(((weights[s, :, :n].cpu().double() - want).abs() <= tol).all()), s
    full = weights
    kept, weights, lens = sz.evict_pages(weights, S.cache, T.cache,
                                         torch.tensor([n for _, n in pairs], **i32), budget, 2, 8,
                                         room=room)
    assert weights.shape == (3, KH, room) and lens.tolist() == [96, 90, 96]
    for s, (_, n) in enumerate(pairs):
        for h in range(KH):
            want = pick(full[s, h, :n].tolist(), n, budget, 2, 8)
            assert kept[s, h].tolist() == want + [-1] * (budget - len(want))
            assert torch.equal(weights[s, h, :len(want)], full[s, h, want])
            assert bool((weights[s, h, len(want):] == 0).all())
    rope = sz.rope(D)
    for step in range(5):
        k, v, q = (torch.randn(3, h, D, generator=g).bfloat16() for h in (KH, KH, H))
        lens = lens + 1
        batch = sz.Batch(torch.arange(4, **i32), lens, 3)
        places = torch.tensor([n + step for _, n in pairs], **i32)
        q = sz.kv_append(k.cuda(), v.cuda(), T.cache, batch, rope, q.cuda(), positions=places)
        _, lse = sz.attend_pages(q, T.cache, batch)
        before = weights.cpu()
        again = sz.weigh_pages(q, lse, T.cache, batch, weights, keep)
        assert again.data_ptr() == weights.data_ptr()          # in place: there is room
        T.pairs = [(1, n) for n in lens.tolist()]
        keys = [T.rows(T.kd.cpu(), s) for s in range(3)]
        for s, n, want, tol in expect(T, range(4), lens.tolist(), q.cpu(), lse.cpu(), keys, before,
                                      keep):
            assert bool(((weights[s, :, :n].cpu().double() - want).abs() <= tol).all()), (step, s)
            assert bool((weights[s, :, n:] == 0).all()), (step, s)
        say("own tokens", step)
    full = weights.clone()
    kept, weights, lens_to = sz.evict_pages(weights, T.cache, S.cache, lens, 64, 2, 8, room=100)
    assert weights.shape == (3, KH, 100) and lens_to.tolist() == [64, 64, 64]
    for s, n in enumerate(lens.tolist()):
        for h in range(KH):
            want = pick(full[s, h, :n].tolist(), n, 64, 2, 8)
            assert kept[s, h].tolist() == want
            assert torch.equal(weights[s, h, :64], full[s, h, want])


@pytest.mark.gpu
def test_one_choice_for_all_heads(torch, sz):
    """The same with one choice by the heads' sum: what stays stands in the
    first head's row, so that the heads' sum goes on."""
    H, KH, D, page, budget, keep = 6, 3, 64, 16, 50, 0.75
    pairs = [(2, 200), (1, 40), (30, 131)]
    S = Setup(torch, sz, pairs, H, KH, D, page, seed=50)
    T = Setup(torch, sz, [(1, min(n, budget) + 3) for _, n in pairs], H, KH, D, page, seed=51,
              fill=0.0)
    i32 = dict(dtype=torch.int32, device="cuda")
    room = T.cache.pages_per_seq * page
    _, lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch)
    weights = sz.weigh_pages(S.q.cuda(), lse, S.cache, S.batch)
    full = weights.sum(1, keepdim=True)
    lens = torch.tensor([n for _, n in pairs], **i32)
    kept, weights, lens = sz.evict_pages(full, S.cache, T.cache, lens, budget, 2, 8, room=room)
    assert kept.shape == (3, 1, budget) and weights.shape == (3, KH, room)
    for s, (_, n) in enumerate(pairs):
        want = pick(full[s, 0, :n].tolist(), n, budget, 2, 8)
        assert kept[s, 0].tolist() == want + [-1] * (budget - len(want))
        assert torch.equal(weights[s, 0, :len(want)], full[s, 0, want])
        assert bool((weights[s, 0, len(want):] == 0).all())
    assert bool((weights[:, 1:] == 0).all())
    g = torch.Generator().manual_seed(52)
    rope = sz.rope(D)
    total = torch.zeros(3, room, dtype=torch.float64)     # over the heads, in 64 bits
    slack = torch.zeros_like(total)
    total[:] = weights[:, 0].cpu()
    for step in range(3):
        k, v, q = (torch.randn(3, h, D, generator=g).bfloat16() for h in (KH, KH, H))
        lens = lens + 1
        batch = sz.Batch(torch.arange(4, **i32), lens, 3)
        places = torch.tensor([n + step for _, n in pairs], **i32)
        q = sz.kv_append(k.cuda(), v.cuda(), T.cache, batch, rope, q.cuda(), positions=places)
        _, lse = sz.attend_pages(q, T.cache, batch)
        weights = sz.weigh_pages(q, lse, T.cache, batch, weights, keep)
        T.pairs = [(1, n) for n in lens.tolist()]
        for s, n in enumerate(lens.tolist()):
            want, tol = weights_of(q[s:s + 1].cpu(), lse[s:s + 1].cpu(),
                                   T.rows(T.kd.cpu(), s), n, D ** -0.5)
            total[s, :n - 1] *= keep
            # (each step's product and sum round once)
            slack[s] = slack[s] * keep + 2 * ref.U32 * total[s]
            total[s, :n] += want.sum(0)
            slack[s, :n] += tol.sum(0) + 2 * ref.U32 * total[s, :n]
        got = weights.cpu().double().sum(1)
        assert bool(((got - total).abs() <= slack).all()), step
        say("one choice", step)
    full = weights.sum(1, keepdim=True)
    kept, weights, lens_to = sz.evict_pages(full, T.cache, S.cache, lens, 30, 2, 8)
    assert weights.shape == (3, 1, 30)                # as ever without room
    for s, n in enumerate(lens.tolist()):
        want = pick(full[s, 0, :n].tolist(), n, 30, 2, 8)
        assert kept[s, 0].tolist() == want
        assert torch.equal(weights[s, 0], full[s, 0, want])
