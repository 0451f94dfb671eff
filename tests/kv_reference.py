"""Plain 64-bit forms of the operators on a paged cache (torch, on the CPU),
with the error that FP32 arithmetic and BF16 roundings may bring.

U16 is half a step of BF16 (relative to the value), U32 of FP32."""
import math

import torch

U16 = torch.finfo(torch.bfloat16).eps / 2
U32 = torch.finfo(torch.float32).eps / 2


def attend(q, keys, values, length, scale, causal=True, window=0, softcap=0.0, f32_out=False):
    """q [new, H, D], keys and values [length, KH, D] (any type); returns
    out, lse, and bounds of their errors.

    A score is an FP32 sum of D products that are exact in FP32 (BF16 x
    BF16), in any order: off by at most D U32 sum|q k|, and a few roundings
    of the result (scale, cap, the exponent's argument, whose size is the
    score's): together ds.  A weight exp(s - m) is then off by a factor
    within 2 ds (score and maximum) + 2^-20 (the exponential) and, before it
    multiplies the values, U16 (its rounding to BF16).  The sums over the
    keys add n U32.  A common factor 2^k of the weights is exact.  Output
    and weights' sum are divided: the factors add up.  The maximum may lag
    behind by a bounded factor, which changes no relative error."""
    new, H, D = q.shape
    G = H // keys.shape[1]
    q = q.double().transpose(0, 1)                                      # [H, new, D]
    K = keys.double().transpose(0, 1).repeat_interleave(G, 0)           # [H, length, D]
    V = values.double().transpose(0, 1).repeat_interleave(G, 0)
    c = (length - new + torch.arange(new))[:, None]
    j = torch.arange(length)[None]
    seen = (j <= c) if causal else (j < length).expand(new, length)
    if window:
        seen = seen & (j > c - window)
    n = seen.sum(1)[None, :, None]                                      # [1, new, 1]
    if length == 0:
        zero = torch.zeros(new, H, D, dtype=torch.float64)
        return zero, zero[..., 0] - math.inf, zero, zero[..., 0]

    def most(x):
        return x.masked_fill(~seen, 0).amax(-1, keepdim=True)

    s = (q @ K.transpose(1, 2)) * scale
    size = most((q.abs() @ K.abs().transpose(1, 2)) * scale)
    bound = size
    if softcap:
        s = softcap * torch.tanh(s / softcap)
        bound = size.clamp(max=softcap)
    top = most(s.abs())
    ds = D * U32 * size + 8 * U32 * torch.maximum(bound, top)
    if softcap:
        ds = ds + 8 * U32 * softcap      # 1 - 2 / (1 + e^2x): absolute, scaled by the cap
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    p = torch.exp(s - lse.clamp(min=-1e300))
    out = p @ V
    rel = 4 * ds + (2 * n + 64) * U32 + 2.0 ** -19
    tol = (U16 + rel) * (p @ V.abs()) * (1 + U16) + (0 if f32_out else U16) * out.abs()
    tol_lse = rel + 8 * U32 * lse.abs() + 8 * U32 * top
    out, lse, tol, tol_lse = (x.transpose(0, 1) for x in (out, lse[..., 0], tol, tol_lse[..., 0]))
    return out, lse, tol, tol_lse


def turn(x, weight, eps, positions, freq, rotary, interleaved, magnitude):
    """x [tokens, heads, D]; returns the normed and rotated rows and a bound
    of the error of FP32 arithmetic (norm: the sum of squares off by D U32,
    halved by the root, and a few roundings; angles within 2^-32 turns plus
    2^-32 for the fraction's cut; cos and sin within 2^-22; the pair's two
    products) with one rounding to BF16."""
    x = x.double().clone()
    D = x.shape[-1]
    rel = 4 * U32
    if weight is not None:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * weight.double()
        rel += (D / 2 + 8) * U32
    tol = rel * x.abs()
    R = rotary
    if R:
        i = torch.arange(R // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        t = positions.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64)
        u, v = x[..., a], x[..., b]
        tol_ab = (u.abs() + v.abs()) * magnitude * (rel + 2.0 ** -22 + 4 * U32)
        x[..., a] = magnitude * (u * t.cos() - v * t.sin())
        x[..., b] = magnitude * (v * t.cos() + u * t.sin())
        tol[..., a], tol[..., b] = tol_ab, tol_ab
    # the rounding, of the value as computed; below the normal range BF16's
    # step is 2^-133
    return x, tol + U16 * (x.abs() + tol) + 2.0 ** -134


def page_view(pool, cache_shape, tokens_first):
    """A pool [pages, words] as [pages, token, head, dim]."""
    page, KH, D = cache_shape
    if tokens_first:
        return pool.view(-1, page, KH, D)
    return pool.view(-1, KH, page, D).transpose(1, 2)


def attend_rows(q, positions, keys, values, length, scale, causal=True, window=0, softcap=0.0,
                f32_out=False):
    """attend() for some rows of a sequence only: q [rows, H, D], at cache
    positions [rows]; keys and values of the whole sequence, used a KV head
    at a time.  The same bounds, but for a cap: its score is off by at most
    16 U32 of its own size (below |x| = 1/2 a polynomial off by 3e-8, of an
    argument off by 4 roundings, with 3 more; above, where |tanh x| > 0.46,
    an exponent's argument off by 4 U32 of x sech^2 x <= 0.45, two units each
    for the exponential and the reciprocal and one for the difference: less
    than 6 U32, 13 relative; and two roundings of the cap), and for caps of
    64 and less, where steps that every row sees may leave out the
    polynomial, by 8 U32 of the cap."""
    n, H, D = q.shape
    KH = keys.shape[1]
    G = H // KH
    out, tol = (torch.zeros(n, H, D, dtype=torch.float64) for _ in range(2))
    lse, tol_lse = (torch.zeros(n, H, dtype=torch.float64) for _ in range(2))
    j = torch.arange(length)[None]
    c = positions[:, None]
    seen = (j <= c) if causal else (j < length).expand(n, length)
    if window:
        seen = seen & (j > c - window)
    count = seen.sum(1)[:, None, None]
    seen = seen[:, None]
    for kv in range(KH):
        at = slice(kv * G, (kv + 1) * G)
        x, K, V = q[:, at].double(), keys[:, kv].double(), values[:, kv].double()
        s = (x @ K.t()) * scale
        size = ((x.abs() @ K.abs().t()) * scale).masked_fill(~seen, 0).amax(-1, keepdim=True)
        bound = size
        if softcap:
            s = softcap * torch.tanh(s / softcap)
            bound = size.clamp(max=softcap)
        top = s.abs().masked_fill(~seen, 0).amax(-1, keepdim=True)
        ds = D * U32 * size + 8 * U32 * torch.maximum(bound, top)
        if softcap:
            ds = ds + 16 * U32 * top + (8 * U32 * softcap if softcap <= 64 else 0)
        s = s.masked_fill(~seen, -math.inf)
        z = torch.logsumexp(s, -1, keepdim=True)
        p = torch.exp(s - z.clamp(min=-1e300))
        o = p @ V
        rel = 4 * ds + (2 * count + 64) * U32 + 2.0 ** -19
        out[:, at], lse[:, at] = o, z[..., 0]
        tol[:, at] = (U16 + rel) * (p @ V.abs()) * (1 + U16) + (0 if f32_out else U16) * o.abs()
        tol_lse[:, at] = (rel + 8 * U32 * z.abs() + 8 * U32 * top)[..., 0]
    return out, lse, tol, tol_lse
