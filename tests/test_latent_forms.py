"""Latent attention from end to end: a prompt's latents are appended, normed
and rotated, to pages; keys and values expanded from what the pages hold are
attended to; single tokens go on in the absorbed form, and their outputs,
projected back, are those of attention in the heads.  Each stage is compared
with 64 bits on what the stage before it left, within bounds that zeros, another
sequence's keys, keys without their rotary part and another head's do not meet
(the CPU tests below plant them)."""
import math
import sys

import pytest
import torch

import kv_reference as ref

H, L, R, D, V, PAGE = 6, 256, 32, 64, 64, 16
SCALE = (D + R) ** -0.5
LENS, FIRST = [150, 61], [100, 40]        # tokens after the prompt, and of its first chunk
FREQ = [10000.0 ** (-2.0 * i / R) for i in range(R // 2)]


def say(*a):
    print("[latent-forms]", *a, flush=True)
    sys.stdout.flush()


class Model:
    """Projections of keys and values from a latent, as BF16 has them."""

    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.up_k = (self.randn(H, D, L) * L ** -0.5).bfloat16().double()
        self.up_v = (self.randn(H, V, L) * L ** -0.5).bfloat16().double()
        self.weight = 1 + 0.2 * self.randn(L)

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g)

    def expand(self, c):
        """Keys and values [length, H, ..] of latents [length, L], 64 bits."""
        c = c.double()
        return (torch.matmul(self.up_k, c.t()).permute(2, 0, 1),
                torch.matmul(self.up_v, c.t()).permute(2, 0, 1))

    def absorb(self, q):
        """q [new, H, D] in 64 bits as queries of latents [new, H, L]."""
        return torch.matmul(q.transpose(0, 1), self.up_k).transpose(0, 1)

    def project(self, o):
        """Outputs [new, H, L] (or their error) to [new, H, V]."""
        return torch.matmul(o.transpose(0, 1), self.up_v.transpose(1, 2)).transpose(0, 1)


def with_rotary(k, r):
    """Keys [length, H, D] with the rotary part [length, R] that all share."""
    return torch.cat([k, r[:, None].expand(-1, k.shape[1], -1)], -1)


def within(got, want, tol):
    return bool(((got.double() - want).abs() <= tol).all())


# ---- the expanded form --------------------------------------------------------

def expanded_want(q, kv, r):
    """q [new, H, D + R] and the tensors that the call takes, kv [length, H,
    D + V] and r [length, R], all BF16: output, log-sums and their bounds."""
    K = with_rotary(kv[..., :D].double(), r.double())
    return ref.attend(q, K, kv[..., D:], kv.shape[0], SCALE)


# ---- the absorbed form ----------------------------------------------------------

def heads_want(m, q_nope, q_rot, q_latent, rows):
    """Attention in the heads, 64 bits: q_nope [new, H, D], q_rot [new, H, R],
    rows [length, L + R] as the pages hold them; and a bound for what the
    absorbed form projects back.  Its queries are q_latent, the absorbed ones
    rounded to BF16, whose scores are off from the heads' by what is computed
    here for each key: all weights change by at most twice the largest of these.
    What else changes a weight (its rounding, its score's) changes it for all
    elements of a key's latent, and so for the value that these project to:
    ref.attend's bound with the projected values.  Only the sums over the keys
    are off element by element, by (2 n + 64) U32, and that is projected by
    absolute values."""
    new, n = q_nope.shape[0], rows.shape[0]
    k, v = m.expand(rows[:, :L])
    c, r = rows[:, :L].double(), rows[:, L:].double()
    q, K = torch.cat([q_nope, q_rot], -1), with_rotary(k, r)
    want, _, _, _ = ref.attend(q, K, v, n, SCALE)
    size, _, _, _ = ref.attend(q, K, v.abs(), n, SCALE)
    off = (q_latent.double() - m.absorb(q_nope)) @ c.t() * SCALE              # [new, H, n]
    tol = torch.expm1(2 * off.abs().amax(-1, keepdim=True)) * size
    q, K = torch.cat([q_latent.double(), q_rot], -1), rows[:, None].double().expand(-1, H, -1)
    tol = tol + ref.attend(q, K, v, n, SCALE, f32_out=True)[2]
    size = ref.attend(q, K, c[:, None].abs().expand(-1, H, -1), n, SCALE)[0]
    tol = tol + (2 * n + 64) * ref.U32 * torch.matmul(
        size.transpose(0, 1), m.up_v.abs().transpose(1, 2)).transpose(0, 1)
    assert want.shape == (new, H, V) == tol.shape
    return want, tol


def planted(m, q_nope, q_rot, rows, others):
    """What must not pass for heads_want's: by name."""
    n = rows.shape[0]
    k, v = m.expand(rows[:, :L])
    r = rows[:, L:].double()
    q = torch.cat([q_nope, q_rot], -1)
    k2, v2 = m.expand(others[:n, :L])
    yield "zeros", torch.zeros_like(q_nope)
    yield "no rotary part", ref.attend(q_nope, k, v, n, SCALE)[0]
    yield "another sequence", ref.attend(q, with_rotary(k2, others[:n, L:].double()), v2,
                                         n, SCALE)[0]
    yield "another head's keys", ref.attend(q, with_rotary(k.roll(1, 1), r), v, n, SCALE)[0]
    yield "another head's values", ref.attend(q, with_rotary(k, r), v.roll(1, 1), n, SCALE)[0]


def planted_expanded(q, kv, r, other_kv, other_r):
    n = kv.shape[0]
    k, v = kv[..., :D].double(), kv[..., D:].double()
    K = with_rotary(k, r.double())
    yield "zeros", torch.zeros(q.shape[0], H, V, dtype=torch.float64)
    yield "no rotary part", ref.attend(q[..., :D], k, v, n, SCALE)[0]
    yield "another sequence", ref.attend(q, with_rotary(other_kv[:n, :, :D].double(),
                                                        other_r[:n].double()),
                                         other_kv[:n, :, D:], n, SCALE)[0]
    yield "another head's keys", ref.attend(q, K.roll(1, 1), v, n, SCALE)[0]
    yield "another head's values", ref.attend(q, K, v.roll(1, 1), n, SCALE)[0]
    yield "not causal", ref.attend(q, K, v, n, SCALE, causal=False)[0]


def test_bounds_of_the_expanded_form_reject():
    m = Model(1)
    rows = [m.randn(n, L + R).bfloat16() for n in (LENS[0], LENS[0])]
    kv = [torch.cat(m.expand(x[:, :L]), -1).bfloat16() for x in rows]
    q = m.randn(30, H, D + R).bfloat16()
    want, lse, tol, tol_lse = expanded_want(q, kv[0], rows[0][:, L:])
    # within: the form that the kernel computes, FP32 sums of BF16 weights
    K = with_rotary(kv[0][..., :D].float(), rows[0][:, L:].float())
    s = torch.matmul(q.float().transpose(0, 1), K.permute(1, 2, 0)) * SCALE
    at = torch.arange(30)[:, None] + LENS[0] - 30
    s.masked_fill_(torch.arange(LENS[0])[None] > at, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    out = torch.matmul(p.bfloat16().float(), kv[0][..., D:].float().transpose(0, 1)) / \
        p.sum(-1, keepdim=True)
    assert within(out.transpose(0, 1).bfloat16(), want, tol)
    assert within((p.sum(-1).log() + top[..., 0]).t(), lse, tol_lse)
    for name, wrong in planted_expanded(q, kv[0], rows[0][:, L:], kv[1], rows[1][:, L:]):
        assert not within(wrong, want, tol), name


def test_bounds_of_the_absorbed_form_reject():
    m = Model(2)
    rows, others = (m.randn(LENS[0] + 1, L + R).bfloat16() for _ in range(2))
    q_nope, q_rot = m.randn(1, H, D).bfloat16().double(), m.randn(1, H, R).bfloat16().double()
    q_latent = m.absorb(q_nope).bfloat16()
    want, tol = heads_want(m, q_nope, q_rot, q_latent, rows)
    q = torch.cat([q_latent.float(), q_rot.float()], -1)
    s = torch.matmul(q, rows.float().t()) * SCALE
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(p.bfloat16().float(), rows[:, :L].float()) / p.sum(-1, keepdim=True)
    assert within(m.project(o.double()), want, tol)
    for name, wrong in planted(m, q_nope, q_rot, rows, others):
        assert not within(wrong, want, tol), name
    k, v = m.expand(rows[:, :L])
    K = with_rotary(k, rows[:, L:].double())[:-1]
    one_less = ref.attend(torch.cat([q_nope, q_rot], -1), K, v[:-1], K.shape[0], SCALE)[0]
    assert not within(one_less, want, tol)


# ---- on the GPU -----------------------------------------------------------------

@pytest.fixture(scope="module")
def sz():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    torch.cuda.set_device(0)
    import lossless_bf16_kv_split_amd as m
    return m


class Cached:
    """Two sequences in pages in shuffled order; what each has been given."""

    def __init__(self, sz, m):
        self.sz, self.m = sz, m
        order = torch.randperm(24, generator=m.g)
        self.ids = order[:22].view(2, 11)
        self.pool = torch.zeros(24, PAGE, L + R, dtype=torch.bfloat16, device="cuda")
        self.cache = sz.latent_cache(self.pool, self.ids.cuda(), L)
        self.rope = sz.rope(R, interleaved=True)
        self.given = [torch.zeros(0, 1, L + R, dtype=torch.bfloat16) for _ in range(2)]

    def batch(self, news, lens):
        i32 = dict(dtype=torch.int32, device="cuda")
        return self.sz.Batch(torch.tensor([0, news[0], sum(news)], **i32),
                             torch.tensor(lens, **i32), sum(news))

    def append(self, lens, q=None):
        """New tokens up to lens; returns the batch and the turned queries."""
        news = [n - x.shape[0] for n, x in zip(lens, self.given)]
        x = self.m.randn(sum(news), 1, L + R).bfloat16()
        self.given = [torch.cat([y, x[a:b]]) for y, a, b in
                      zip(self.given, (0, news[0]), (news[0], sum(news)))]
        batch, x = self.batch(news, lens), x.cuda()
        return batch, self.sz.latent_append(x[..., :L], self.cache, batch, x[..., L:], self.rope,
                                            q, self.m.weight.cuda())

    def rows(self, s):
        return self.pool[self.ids[s].cuda()].reshape(-1, L + R)[:self.given[s].shape[0]]

    def check_rows(self):
        for s in range(2):
            n, got = self.given[s].shape[0], self.rows(s).cpu()
            x = self.given[s]
            want, tol = ref.turn(x[..., :L], self.m.weight, 1e-6, torch.arange(n), FREQ, 0,
                                 True, 1.0)
            assert within(got[:, None, :L], want, tol), s
            want, tol = ref.turn(x[..., L:], None, 0, torch.arange(n), FREQ, R, True, 1.0)
            assert within(got[:, None, L:], want, tol), s
        spare = torch.tensor([i for i in range(24) if i not in self.ids.flatten().tolist()])
        assert bool((self.pool[spare.cuda()] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("seed", [20, 21])
def test_prompt_then_single_tokens(sz, seed):
    m = Model(seed)
    C = Cached(sz, m)
    C.append(FIRST)
    news = [a - b for a, b in zip(LENS, FIRST)]
    q = m.randn(sum(news), H, D + R).bfloat16()
    before = q[..., D:].clone()
    batch, turned = C.append(LENS, q[..., D:].contiguous().cuda())
    q[..., D:] = turned.cpu()
    C.check_rows()
    at = torch.cat([torch.arange(a, b) for a, b in zip(FIRST, LENS)])
    want, tol = ref.turn(before, None, 0, at, FREQ, R, True, 1.0)
    assert within(q[..., D:], want, tol)
    say("appended", seed)

    c = torch.cat([C.rows(s) for s in range(2)])
    up = torch.cat([m.up_k, m.up_v], 1).float().cuda()
    kv = (c[:, :L].float() @ up.view(-1, L).t()).bfloat16().view(-1, H, D + V)
    starts = torch.tensor([0, LENS[0]], dtype=torch.int32, device="cuda")
    out, lse = sz.attend_expanded(q.cuda(), kv[..., :D], kv[..., D:], starts, batch, SCALE,
                                  c[:, None, L:])
    out, lse, kv, r = out.cpu(), lse.cpu(), kv.cpu(), c[:, L:].cpu()
    rows = [slice(0, LENS[0]), slice(LENS[0], sum(LENS))]
    for s in range(2):
        a, b = sum(news[:s]), sum(news[:s + 1])
        want, want_lse, tol, tol_lse = expanded_want(q[a:b], kv[rows[s]], r[rows[s]])
        assert within(out[a:b], want, tol) and within(lse[a:b], want_lse, tol_lse), s
        if s == 1:                       # (the other sequence has at least as many keys)
            for name, wrong in planted_expanded(q[a:b], kv[rows[1]], r[rows[1]], kv[rows[0]],
                                                r[rows[0]]):
                assert not within(out[a:b], wrong, tol), name
    say("expanded", seed)

    for step in range(3):
        q_nope = m.randn(2, H, D).bfloat16().double()
        q_latent = m.absorb(q_nope).bfloat16()
        q_rot = m.randn(2, H, R).bfloat16()
        lens = [n + 1 + step for n in LENS]
        batch, turned = C.append(lens, q_rot.cuda())
        C.check_rows()
        o, _ = sz.attend_latent(torch.cat([q_latent.cuda(), turned], -1), C.cache, batch, SCALE,
                                max(lens), out_dtype=torch.float32)
        back, turned = m.project(o.cpu().double()), turned.cpu().double()
        for s in range(2):
            one = slice(s, s + 1)
            mine, other = C.rows(s).cpu(), C.rows(1 - s).cpu()
            want, tol = heads_want(m, q_nope[one], turned[one], q_latent[one], mine)
            assert within(back[one], want, tol), (step, s)
            if s == 1:
                for name, wrong in planted(m, q_nope[one], turned[one], mine, other):
                    assert not within(back[one], wrong, tol), (name, step)
        say("absorbed", seed, step)
