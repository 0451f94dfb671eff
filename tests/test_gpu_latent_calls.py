"""How the operators on latents, the expanded form, attention weights and
eviction are called: on other streams, two at once, captured into graphs that
share a workspace, again with the same result to the bit, over pages that stand
in a table more than once, without new tokens.  What they compute is checked in
test_gpu_latent.py, test_gpu_expanded.py and test_gpu_evict.py."""
import math
import sys

import pytest

import kv_reference as ref
import test_gpu_evict as evict
import test_gpu_latent as latent

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-calls]", *a, flush=True)
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


class Call:
    """An operator with its inputs, outputs and workspace.  words(i) puts other
    inputs in place, by copies alone; run() computes; results() clones."""

    def __init__(self, torch, inputs, outputs, size, run):
        self.torch, self.inputs, self.outputs, self.size = torch, inputs, outputs, size
        self.ws = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
        self._run = run
        g = torch.Generator().manual_seed(5)
        self.values = [[torch.randn(t.shape, generator=g).to(t.dtype).cuda() for t in inputs]
                       for _ in range(3)]

    def words(self, i):
        for t, v in zip(self.inputs, self.values[i]):
            t.copy_(v)

    def run(self, ws=None):
        self._run(self.ws if ws is None else ws)

    def clear(self):
        for t in self.outputs:
            t.zero_()

    def results(self):
        return [t.clone() for t in self.outputs]


def make(torch, sz, name):
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    if name in ("append", "absorbed"):
        S = latent.Setup(torch, sz, [(3, 900), (1, 40), (5, 2000)], 16, 512, 64, 16, seed=3)
        if name == "append":
            x, k = torch.zeros(S.n, 1, 512, **bf16), torch.zeros(S.n, 1, 64, **bf16)
            q, out = torch.zeros(S.n, 16, 64, **bf16), torch.zeros(S.n, 16, 64, **bf16)
            rope = sz.rope(64)
            return Call(torch, [x, k, q], [out, S.dev], 0, lambda ws: sz.sz_latent_append(
                x, None, 0.0, k, q, out, rope, None, S.cache, S.batch))
        q = torch.zeros(S.n, 16, 576, **bf16)
        out, lse = torch.zeros(S.n, 16, 512, **bf16), torch.zeros(S.n, 16, device="cuda")
        size = sz.sz_attend_latent_workspace_size(16, S.cache, S.batch, 2000)
        assert size > 0
        return Call(torch, [q, S.dev], [out, lse], size, lambda ws: sz.sz_attend_latent(
            q, out, lse, S.cache, S.batch, 2000, 0.1, True, ws, size))
    if name == "expanded":
        n, keys, H = 200, 3000, 4
        q, out = torch.zeros(n, H, 192, **bf16), torch.zeros(n, H, 128, **bf16)
        k, v = torch.zeros(keys, H, 128, **bf16), torch.zeros(keys, H, 128, **bf16)
        r, lse = torch.zeros(keys, 1, 64, **bf16), torch.zeros(n, H, device="cuda")
        batch = sz.Batch(torch.tensor([0, 150, n], **i32), torch.tensor([2100, 900], **i32), n)
        starts = torch.tensor([0, 2100], **i32)
        size = sz.sz_attend_expanded_workspace_size(H, 128, batch, 2100)
        assert size > 0
        return Call(torch, [q, k, v, r], [out, lse], size, lambda ws: sz.sz_attend_expanded(
            q, out, lse, k, r, v, starts, batch, 2100, 0.1, True, ws, size))
    S = evict.Setup(torch, sz, [(300, 2500), (1, 700)], 8, 2, 64, 16, seed=4)
    if name == "weigh":
        q, lse = torch.zeros(S.n, 8, 64, **bf16), torch.zeros(S.n, 8, device="cuda")
        w = torch.zeros(2, 2, 2500, device="cuda")
        size = sz.sz_weigh_workspace_size(8, S.cache, S.batch, 2500)
        assert size > 0
        return Call(torch, [q, S.kd, lse], [w], size, lambda ws: sz.sz_weigh_pages(
            q, lse, None, w, 2500, 0.0, S.cache, S.batch, 2500, 0.1, workspace=ws,
            workspace_bytes=size))
    T = evict.Setup(torch, sz, [(1, 600), (1, 600)], 8, 2, 64, 32, seed=6, fill=0.0)
    w, w_to = torch.zeros(2, 2, 2500, device="cuda"), torch.zeros(2, 2, 600, device="cuda")
    kept, lens_to = torch.zeros(2, 2, 600, **i32), torch.zeros(2, **i32)
    lens = torch.tensor([2500, 700], **i32)
    return Call(torch, [w, S.kd, S.vd], [w_to, kept, lens_to, T.kd, T.vd], 0,
                lambda ws: sz.sz_evict_pages(w, w_to, S.cache, T.cache, lens, lens_to, 2500, 600,
                                             4, 64, kept))


NAMES = ["append", "absorbed", "expanded", "weigh", "evict"]


def same(torch, a, b, label):
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), (label, i)


def expected(torch, call, i):
    call.words(i)
    call.clear()
    call.run()
    torch.cuda.synchronize()
    return call.results()


@pytest.mark.parametrize("name", NAMES)
def test_again_and_on_another_stream(torch, sz, name):
    """The same words give the same bits: again, with a workspace of other
    content, and on a stream where they have only just been put in place."""
    call = make(torch, sz, name)
    want = [expected(torch, call, i) for i in range(3)]
    assert not all(torch.equal(a, b) for a, b in zip(want[0], want[1]))
    call.ws.fill_(0xFF)
    same(torch, expected(torch, call, 0), want[0], "again")
    side = torch.cuda.Stream()
    for i in (1, 2, 0):
        say(name, "stream", i)
        with torch.cuda.stream(side):
            call.words(i)
            call.clear()
            call.run()
            got = call.results()
        side.synchronize()
        same(torch, got, want[i], i)


@pytest.mark.parametrize("pair", [("absorbed", "weigh"), ("expanded", "evict"),
                                  ("append", "absorbed"), ("weigh", "weigh")], ids=str)
def test_two_at_once(torch, sz, pair):
    """Two calls under way at the same time on two streams, each with its own
    workspace."""
    calls = [make(torch, sz, name) for name in pair]
    want = [expected(torch, c, i) for i, c in enumerate(calls)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    say(pair)
    for c in calls:
        c.clear()
    torch.cuda.synchronize()
    for _ in range(5):
        for c, stream in zip(calls, streams):
            with torch.cuda.stream(stream):
                c.run()
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        same(torch, c.results(), w, pair)


def test_graphs_that_share_a_workspace(torch, sz):
    """Graphs of the five operators over one workspace, replayed in turn and in
    other orders with other words, eager work and synchronizations between."""
    calls = {name: make(torch, sz, name) for name in NAMES}
    want = {name: [expected(torch, c, i) for i in range(3)] for name, c in calls.items()}
    ws = torch.empty(max(c.size for c in calls.values()), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c in calls.values():
            c.run(ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs = {}
    for name, c in calls.items():
        graphs[name] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[name]):
            c.run(ws)
    for replay, order in enumerate([NAMES, NAMES[::-1], NAMES[2:] + NAMES[:2], NAMES]):
        say("replay", replay)
        i = replay % 3
        for name in order:
            calls[name].words(i)
            calls[name].clear()
        for name in order:
            graphs[name].replay()
        torch.cuda.synchronize()
        for name in order:
            same(torch, calls[name].results(), want[name][i], (replay, name))
        calls[order[0]].run(ws)        # eager work over the same workspace
        torch.cuda.synchronize()
        same(torch, calls[order[0]].results(), want[order[0]][i], replay)


def test_pages_that_stand_twice_in_a_table(torch, sz):
    """Sequences with the same first pages, and one page at several places of a
    sequence: attended to, weighed and given up as separate tokens."""
    S = latent.Setup(torch, sz, [(1, 200), (2, 150), (1, 90)], 16, 128, 64, 16, seed=7)
    S.ids[1, :5] = S.ids[0, :5]
    S.ids[2, 1] = S.ids[2, 3] = S.ids[2, 0]
    S.upload()
    latent.check(torch, sz, S, "latents")
    W = evict.Setup(torch, sz, [(1, 200), (2, 150), (1, 90)], 8, 2, 64, 16, seed=8)
    W.ids[1, :5] = W.ids[0, :5]
    W.ids[2, 1] = W.ids[2, 3] = W.ids[2, 0]
    table = W.ids.cuda()
    view = lambda x: ref.page_view(x, W.shape, True)
    W.cache = sz.paged_cache(view(W.kd), view(W.vd), table)
    evict.check_weigh(torch, sz, W, "weights")
    T = evict.Setup(torch, sz, [(1, 40)] * 3, 8, 2, 64, 16, seed=9, fill=0.0)
    weights = W.rand(3, 2, 200).abs().cuda()
    lens = torch.tensor([n for _, n in W.pairs], dtype=torch.int32, device="cuda")
    kept, w_to, lens_to = sz.evict_pages(weights, W.cache, T.cache, lens, 40, 2, 8, max_len=200)
    assert lens_to.tolist() == [40] * 3
    K, V = view(W.kd).cpu(), view(W.vd).cpu()
    K1, V1 = view(T.kd).cpu(), view(T.vd).cpu()
    for s in range(3):
        for h in range(2):
            for d, j in enumerate(kept[s, h].tolist()):
                for a, b in ((K, K1), (V, V1)):
                    assert torch.equal(a[W.ids[s, j // 16], j % 16, h],
                                       b[T.ids[s, d // 16], d % 16, h]), (s, h, d)
                assert w_to[s, h, d] == weights[s, h, j]


def test_weights_without_new_tokens(torch, sz):
    """A batch of no new tokens, and a sequence of none beside others: the
    weights are multiplied by keep."""
    S = evict.Setup(torch, sz, [(0, 300), (0, 0), (0, 17)], 8, 2, 64, 16, seed=10)
    before = S.rand(3, 2, 304).abs().cuda()
    for in_place in (False, True):
        w = before.clone() if in_place else torch.full_like(before, math.inf)
        status = torch.full((3,), -1, dtype=torch.int32, device="cuda")
        q = torch.zeros(0, 8, 64, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(0, 8, device="cuda")
        sz.sz_weigh_pages(q, lse, w if in_place else before, w, 304, 0.25, S.cache, S.batch, 304,
                          0.1, d_status=status)
        torch.cuda.synchronize()
        assert status.tolist() == [0, 0, 0]
        for s, (_, n) in enumerate(S.pairs):
            assert torch.equal(w[s, :, :n], 0.25 * before[s, :, :n]), s
            assert torch.equal(w[s, :, n:], before[s, :, n:] if in_place else
                               torch.full_like(before[s, :, n:], math.inf)), s
