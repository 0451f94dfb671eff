"""Attention weights of batches whose sequences have few new rows on average and
some of which have many: a chunk of a prompt beside single tokens, beside idle
sequences, at every size of a workgroup's keys."""
import math

import pytest

from test_gpu_evict import SENTINEL, check_weigh, sz, torch, weigh  # noqa: F401
from test_gpu_kv import Setup

pytestmark = pytest.mark.gpu

# (new, cached) of sequences; heads, KV heads, elements, page; the mean stays within 32 rows
# of a KV head's heads
SHAPES = [(8, 2, 64, 16), (4, 4, 128, 16), (3, 1, 256, 32), (12, 4, 96, 64)]


def mixed(chunks, singles, longest, idle=0):
    pairs = [(1, 1 + 37 * i % longest) for i in range(singles)]
    pairs += [(0, 1 + 53 * i % longest) for i in range(idle)]
    for i, c in enumerate(chunks):
        pairs.insert(7 * i + 3, c)
    return pairs


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("chunk", [(129, 129), (130, 700), (257, 300), (200, 3001)], ids=str)
def test_a_chunk_beside_single_tokens(torch, sz, shape, chunk):
    group = shape[0] // shape[1]
    pairs = mixed([chunk], -(-chunk[0] * group // 20), 300)
    S = Setup(torch, sz, pairs, *shape, seed=60, before=3, behind=2)
    assert S.n * group <= 32 * len(pairs)
    assert check_weigh(torch, sz, S, f"chunk {shape} {chunk}", keep=0.5) == 0


@pytest.mark.parametrize("kw", [dict(causal=False), dict(window=1), dict(window=40),
                                dict(window=300), dict(softcap=5.0)], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_masks(torch, sz, shape, kw):
    pairs = mixed([(150, 150), (131, 600)], 70, 200, idle=10)
    S = Setup(torch, sz, pairs, *shape, seed=61)
    check_weigh(torch, sz, S, f"masks {shape} {kw}", keep=0.9, **kw)


@pytest.mark.parametrize("tokens", [32, 33, 43, 65, 128, 129])
def test_at_the_border(torch, sz, tokens):
    """Rows of one sequence around what one form takes."""
    for shape in ((4, 1, 64, 16), (3, 1, 128, 16), (2, 2, 64, 16)):
        S = Setup(torch, sz, mixed([(tokens, 200)], 40, 150), *shape, seed=62)
        check_weigh(torch, sz, S, f"border {tokens} {shape}", keep=1.0)


def test_beside_idle_sequences(torch, sz):
    """One sequence goes on, the others keep what they have; as many new tokens
    as sequences, and fewer."""
    for idle in (40, 149, 160):
        S = Setup(torch, sz, mixed([(150, 260)], 0, 220, idle=idle), 4, 2, 64, 16, seed=63)
        check_weigh(torch, sz, S, f"idle {idle}", keep=0.25)


def test_many_keys_and_short_bounds(torch, sz):
    """Workgroups of 128, 256 and 512 keys, by the bound of the lengths."""
    for longest, singles in ((600, 14), (2500, 40), (2500, 300)):
        pairs = mixed([(140, longest), (200, 201)], singles, longest)
        S = Setup(torch, sz, pairs, 2, 2, 64, 64, seed=64)
        check_weigh(torch, sz, S, f"keys {longest} {singles}", keep=0.75, max_len=longest)
        check_weigh(torch, sz, S, f"keys {longest} {singles}", with_before=False)


def test_more_new_tokens_than_cached(torch, sz):
    """Rows that see nothing: positions before the first key."""
    pairs = mixed([(150, 20), (140, 0), (160, 159)], 60, 100)
    S = Setup(torch, sz, pairs, 4, 2, 64, 16, seed=65)
    check_weigh(torch, sz, S, "more new than cached", keep=1.0)


def test_in_place_and_log_sums_of_nothing(torch, sz):
    pairs = mixed([(140, 400)], 60, 300)
    S = Setup(torch, sz, pairs, 4, 2, 128, 16, seed=66)
    _, lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch)
    lse[S.starts[3] + 5:S.starts[3] + 70] = -math.inf      # (rows of the chunk)
    check_weigh(torch, sz, S, "log-sums of nothing", lse=lse)
    pitch = S.width * S.page
    before = S.rand(len(pairs), 2, pitch).abs().cuda()
    out = torch.full_like(before, SENTINEL)
    same = before.clone()
    for at, to in ((before, out), (same, same)):
        sz.sz_weigh_pages(S.q.cuda(), lse, at, to, pitch, 0.5, S.cache, S.batch, 0, 0.1)
    torch.cuda.synchronize()
    for s, (_, n) in enumerate(pairs):
        assert torch.equal(out[s, :, :n], same[s, :, :n]), s
        assert torch.equal(same[s, :, n:], before[s, :, n:]), s


def test_unseen_content_and_bad_sequences(torch, sz):
    """What a chunk's rows do not see, and sequences at fault, change nothing
    for the others."""
    pairs = mixed([(140, 400)], 60, 300)
    S = Setup(torch, sz, pairs, 4, 2, 64, 16, seed=67)
    _, lse = sz.attend_pages(S.q.cuda(), S.cache, S.batch)
    want, status, _ = weigh(torch, sz, S, lse, None)
    assert status == [0] * len(pairs)
    own = torch.zeros(S.kd.shape[0], dtype=torch.bool)
    own[S.ids[3, :25]] = True
    page, kv, dim = S.shape
    pool = S.kd.view(-1, page, kv * dim)
    pool[(~own).cuda()] = math.nan                         # every other sequence's keys
    got, status, _ = weigh(torch, sz, S, lse, None)
    assert status == [0] * len(pairs)
    assert torch.equal(got[3, :, :400], want[3, :, :400])
    S.upload()
    lens = torch.tensor([n for _, n in pairs], dtype=torch.int32, device="cuda")
    for s, bad in ((3, -1), (3, 2 ** 31 - 1), (9, 2 ** 31 - 1), (9, -7)):
        x = lens.clone()
        x[s] = bad
        starts = torch.tensor(S.starts, dtype=torch.int32, device="cuda")
        got, status, _ = weigh(torch, sz, S, lse, None, batch=sz.Batch(starts, x, S.n))
        assert [i for i, v in enumerate(status) if v] == [s]
        keep = [i for i in range(len(pairs)) if i != s]
        assert torch.equal(got[keep], want[keep]) and bool((got[s] == SENTINEL).all())


def test_captured(torch, sz):
    """A graph of the call, replayed with other lengths: the long sequence's
    place changes from replay to replay."""
    pairs = mixed([(140, 400)], 60, 300)
    S = Setup(torch, sz, pairs, 4, 2, 64, 16, seed=68)
    pitch = S.width * S.page
    q, lse = S.q.cuda(), torch.full((S.n, 4), 6.0, device="cuda")
    out = torch.zeros(len(pairs), 2, pitch, device="cuda")
    starts = torch.tensor(S.starts, dtype=torch.int32, device="cuda")
    lens = torch.tensor([n for _, n in pairs], dtype=torch.int32, device="cuda")
    batch = sz.Batch(starts, lens, S.n)

    def step():
        sz.sz_weigh_pages(q, lse, None, out, pitch, 0.0, S.cache, batch, 0, 0.125)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for at in (3, 0, 30, 60):
        news = [1] * len(pairs)
        news[at] = 140
        bounds = [0]
        for x in news:
            bounds.append(bounds[-1] + x)
        starts.copy_(torch.tensor(bounds, dtype=torch.int32))
        # (lengths within each sequence's own pages)
        lens.copy_(torch.tensor([n for _, n in pairs], dtype=torch.int32))
        out.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.fill_(SENTINEL)
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and bool((out != SENTINEL).any()), at
