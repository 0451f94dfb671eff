"""Attention of chunks over a paged cache (sz_attend_pages) where tiles have
128 and 256 rows: sampled rows of long calls against the plain 64-bit form,
with the bounds of kv_reference.py."""
import math

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
    picked |= set(torch.randint(0, n, (count,), generator=g).tolist()) if n else set()
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


def check(torch, sz, S, label, count=24, out_type=None, max_len=0, **kw):  # noqa: F811
    say(label)
    out, lse = run(torch, sz, S, out_type, max_len, **kw)
    covered = torch.zeros(S.n, dtype=torch.bool)
    for s, (new, length) in enumerate(S.pairs):
        a, b = S.starts[s], S.starts[s + 1]
        covered[a:b] = True
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
