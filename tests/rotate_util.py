"""Plain 64-bit rotation by position, with a bound on a kernel's error derived from its arithmetic."""
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def rotate_reference(x, pos, freqs, magnitude, begin, pairs, out_dtype, inverse=False):
    """Rows x [n][h][d] turned by pos [n] in double, and a bound on each element's error.

    Bound.  A cosine or sine is off by 2^-22 at most (the fraction of a turn rounded to fp32, at most an
    eighth: pi / 4 2^-24; sincospif: two steps of a value of at most 1, 2^-22) and by the frequency's own
    rounding, pos f 2^-50 radians (f / 2 pi and the reference's angle, both double).  The magnitude's
    product, the two products and their sum in fp32 add less than 4 2^-24 of (|u| + |v|) magnitude.  Last
    the result's rounding, half a step.  Dims that do not turn are exact but for that rounding."""
    n_rot = 2 * len(freqs)
    x = x.double().cpu()
    y, tol = x.clone(), torch.zeros_like(x)
    j = torch.arange(n_rot // 2)
    a, b = (2 * j, 2 * j + 1) if pairs else (j, j + n_rot // 2)
    angle = torch.outer(pos.double().cpu(), torch.tensor(freqs, dtype=torch.float64)) * (-1 if inverse else 1)
    c, s = (angle.cos() * magnitude)[:, None], (angle.sin() * magnitude)[:, None]
    u, v = x[..., begin + a], x[..., begin + b]
    y[..., begin + a], y[..., begin + b] = u * c - v * s, u * s + v * c
    delta = (2.0 ** -21 + angle.abs()[:, None] * 2.0 ** -50) * abs(magnitude) * (u.abs() + v.abs())
    tol[..., begin + a] = delta
    tol[..., begin + b] = delta
    return y, tol * (1 + HALF_STEP[out_dtype]) + HALF_STEP[out_dtype] * y.abs() + 1e-40
