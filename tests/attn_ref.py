"""Plain 64-bit attention and cache quantisation for the attention tests, on the CPU, with the
elementwise error bound each result may have.

Bounds. With p_j the softmax weights and A = sum_j p_j |v_j| (so |o| <= A), a kernel that keeps
scores, statistics and sums in fp32 is off by at most A times
  2 ds + (keys + 32) 2^-24    ds: error of a score: the fp32 dot product's (d + 4) 2^-24 sum |q k|
                              scale, and 2^-20 for the exponential (in its argument's units)
and, with bf16 inputs, 2^-8 (half a unit in the last place of 8 significant bits, relative to
the smallest mantissa) for each weight's rounding and 2^-8 for the output's. lse is off by
at most ds + (keys + 32) 2^-24 plus its own rounding.
"""
import math

import torch

U32 = 2.0 ** -24


def attend(q, k, v, scale, allowed):
    """q [m, d], k, v [l, d] (any float type), allowed bool [m, l]. Returns o [m, d], lse [m], the
    bound's A [m, d] and the relative bounds of o without and with bf16 roundings, [m, 1]."""
    q, k, v = q.double(), k.double(), v.double()
    m, l = allowed.shape
    seen = allowed.any(1, keepdim=True)
    # a masked key contributes nothing, whatever it holds
    s = torch.full((m, l), -math.inf, dtype=torch.float64)
    a = torch.zeros(m, v.shape[1], dtype=torch.float64)
    o = torch.zeros_like(a)
    raw = q @ k.t() * scale
    s = torch.where(allowed, raw, s)
    lse = torch.where(seen[:, 0], torch.logsumexp(s, 1), torch.full((m,), -math.inf, dtype=torch.float64))
    p = torch.where(allowed, torch.exp(s - torch.where(seen, lse[:, None], 0.0)), 0.0)
    if bool(torch.isfinite(v).all()):
        o, a = p @ v, p @ v.abs()
    else:
        for i in range(m):
            at = allowed[i]
            o[i] = p[i, at] @ v[at]
            a[i] = p[i, at] @ v[at].abs()
    size = torch.where(allowed, (q.abs() @ k.abs().t()) * abs(scale), 0.0)
    ds = (q.shape[1] + 4) * U32 * size.amax(1, keepdim=True) + 2.0 ** -20 if l else torch.zeros(m, 1).double()
    f32 = 2 * ds + (l + 32) * U32
    return o, lse, a, f32, f32 + 2.0 ** -7


def causal_mask(lq, lk, causal):
    i, j = torch.arange(lq)[:, None], torch.arange(lk)[None]
    return (j <= i + lk - lq) if causal else torch.ones(lq, lk, dtype=torch.bool)


def check(out, lse, o, lse_ref, a, f32, bf16, what=""):
    """Compare one (sequence, head)'s rows with attend()'s answer."""
    rel = bf16 if out.dtype == torch.bfloat16 else f32
    got = out.double().cpu()
    nan = torch.isnan(o)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(o)
    assert torch.equal(got[inf], o[inf]), f"{what}: infinities"
    fine = ~nan & ~inf & torch.isfinite(a)
    # the smallest normal number covers roundings to zero
    tol = rel * a + 2.0 ** -126
    err = (got - o).abs()
    worst = ((err / tol)[fine]).max().item() if bool(fine.any()) else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3f} times its bound"
    if lse is not None:
        g = lse.double().cpu()
        empty = torch.isinf(lse_ref)
        assert torch.equal(g[empty], lse_ref[empty]), f"{what}: lse of rows that see nothing"
        ok = torch.isfinite(lse_ref)
        bound = f32[:, 0] + lse_ref.abs() * 2.0 ** -22 + 2.0 ** -20
        assert bool(((g - lse_ref).abs()[ok] <= bound[ok]).all()), f"{what}: lse"


def quantise(x):
    """fp8 rows as the cache keeps them: (values, scale bytes). x [..., d]."""
    x = x.double()
    fin = torch.isfinite(x)
    top = torch.where(fin, x.abs(), 0.0).amax(-1, keepdim=True)
    m, e = torch.frexp(top)
    e = torch.where(top > 0, (e - 9 + (m > 0.875)).clamp(min=-126), 0)
    unit = torch.ldexp(torch.ones_like(top), e)
    y = x / unit
    step = torch.ldexp(torch.ones_like(y), torch.frexp(y.abs().clamp(min=2.0 ** -6).nan_to_num(1.0, 1.0))[1] - 4)
    q = torch.where(fin, torch.round(y / step) * step * unit, math.nan)
    return q, (e[..., 0] + 127).to(torch.uint8)
