"""Plain 64-bit norms and rotary positions for the tests, on the CPU, with the elementwise error
bound each result may have.

Bounds, in units of u = 2^-24. The norm's sum of d squares is taken 8 or 16 to a lane, then over at
most 32 lanes by halves: each term meets at most 1 + 16 + 5 roundings, its square root half of that,
and the mean, eps, square root, division, bias and two products 7 more: less than 2^-19 of the
normed element y. A cosine or sine in fp32 is good to 2^-21 (the library's 2 ulp of numbers up to 1,
2^-23 each, the rest of the reduced angle, and scaling), and the rotation's two products and sum
round three times: for a pair (a, b), (|a| + |b|) (2^-21 + 3 u) of each element. Angles are exact to
three roundings of 64 bits. The result is rounded once to its type, by at most eps / 2 of itself.
"""
import torch

U32 = 2.0 ** -24


def norm_rope(x, weight, bias, eps, freq, pos, interleaved, scale):
    """x [total, h, d]; weight [d] or None; freq [half] or None; pos [total, half] (each pair's position,
    int). Returns the rows in 64 bits and the absolute error that fp32 may have, both [total, h, d]."""
    y = x.double()
    size = y.abs()
    err = torch.zeros_like(y)
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * (bias + weight.double())
        size = y.abs()
        # a sum of bias and weight may cancel: its rounding is relative to what it is of
        part = y / torch.where(bias + weight.double() == 0, 1.0, bias + weight.double())
        err = 2.0 ** -19 * size + part.abs() * U32 * (abs(bias) + weight.double().abs())
    if freq is None:
        return y, err
    half = freq.shape[0]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    angle = (pos.double() * freq.double())[:, None]
    cos, sin = torch.cos(angle) * scale, torch.sin(angle) * scale
    out, bound = y.clone(), err.clone()
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., b] * cos + y[..., a] * sin
    both = (size[..., a] + size[..., b]) * abs(scale)
    far = both * (2.0 ** -21 + 3 * U32 + angle.abs() * 2.0 ** -50) + (err[..., a] + err[..., b]) * abs(scale)
    bound[..., a] = bound[..., b] = far
    return out, bound


def check(got, want, bound, what=""):
    """Compare what a call wrote (bfloat16 or float32) with norm_rope()'s answer."""
    g = got.double().cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(g), nan), f"{what}: NaN in other places"
    tol = bound + torch.finfo(got.dtype).eps / 2 * want.abs() + 2.0 ** -126
    fine = ~nan & torch.isfinite(want)
    worst = ((g - want).abs() / tol)[fine].max().item() if bool(fine.any()) else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3f} times its bound"
