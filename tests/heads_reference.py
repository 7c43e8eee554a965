"""The per-head norm, rotation and FP8 cache in float64, for the tests.

Tensors are torch CPU tensors.  U is half a step of fp32 (2^-24), H of bf16.
"""
import torch

U = 2.0 ** -24
H = 2.0 ** -8


def norm_rope(x, gamma, eps, weight_offset, cos_sin, positions, interleaved):
    """(y, mag) of [tokens, heads, dim]: the exact values, and for each the sum
    of the magnitudes of the terms it is made of."""
    x = x.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y = x * r * (gamma.double() + weight_offset)
    mag = (x * r).abs() * (gamma.double().abs() + abs(weight_offset))
    if cos_sin is None:
        return y, mag
    rot = cos_sin.shape[1]
    half = rot // 2
    row = cos_sin.double()[positions]
    out, omag = y.clone(), mag.clone()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = row[:, i, None], row[:, half + i, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        omag[..., a] = mag[..., a] * c.abs() + mag[..., b] * s.abs()
        omag[..., b] = mag[..., b] * c.abs() + mag[..., a] * s.abs()
    return out, omag


def norm_error(mag):
    """Bound of the fp32 error of norm_rope's values.  In units of U: the sum
    of squares is a tree of at most 10 additions over products of one rounding
    (11), times 1 / dim rounded (2), plus eps (1); its root halves that (7);
    the hardware reciprocal root adds 2 ulp (4); x * r, gamma + offset and
    their product one each (3); the rotation a product and a sum (2)."""
    return 17 * U * mag


def check_bf16(got, y, err, label):
    """|got - y| is at most the fp32 error, half a bf16 step, and half the
    smallest bf16 subnormal step."""
    tol = err + H * (y.abs() + err) + 2.0 ** -134
    d = (got.double() - y).abs()
    assert bool((d <= tol).all()), f"{label}: {float((d / tol).max()):.3f} of the bound"


E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def e4m3(y):
    """y rounded to the nearest e4m3 value, ties to even, saturating."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448)


def row_scale(x, scale_ub):
    return x.double().abs().amax(-1).clamp(max=scale_ub).clamp(min=1e-12) / 448


def exact_codes(x, scale_ub):
    """The nearest codes of bf16 rows.  x / scale is 448 x / amax, taken with
    one rounding of float64: 448 x is exact, and a quotient that is an e4m3
    midpoint (a bf16 x over a bf16 amax often is) comes out exact, where x over
    a rounded scale would land on either side of it."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True).clamp(max=scale_ub).clamp(min=1e-12)
    return e4m3(448 * x / amax)


def check_codes(codes, scales, x, err, scale_ub, label):
    """codes (as values) and scales of rows x (float64) that the kernel held
    with an error of at most err.  The maximum is off by at most the largest
    err, the division rounds once; a code is the nearest to a quotient that is
    off by err / scale and a few fp32 roundings (4 U)."""
    scale = row_scale(x, scale_ub)
    serr = err.amax(-1) / 448 + 1.01 * U * scale
    assert bool(((scales.double() - scale).abs() <= serr).all()), f"{label}: scales"
    y = x / scale[..., None]
    yerr = err / scale[..., None] + y.abs() * (serr / scale)[..., None] + 4 * U * y.abs()
    y = y.clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2((y.abs() + yerr).clamp(min=2.0 ** -6))) - 3)
    d = (codes.double() - y).abs()
    assert bool((d <= step / 2 + yerr).all()), f"{label}: codes"


def place_of(slots, page_size):
    return slots // page_size, slots % page_size
