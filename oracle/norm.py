"""Root-mean-square norm with the residual's addition, its gradient, and the
gradient of SwiGLU: float64 NumPy from the definitions.  Test infrastructure.

    s = BF16(x + r),  rstd = 1 / sqrt(mean_k s^2 + eps),  y = s rstd w
    dx = rstd (dy w - s rstd c) + ds,  c = mean_k(dy w s rstd),  dw = sum_m dy s rstd
    h = silu(g) u:  dg = dh u sg (1 + g (1 - sg)),  du = dh g sg,  sg = 1 / (1 + e^-g)

The sum's rounding is the only one here (the norm is of the stream as it is
stored): x + r is formed in FP32 and rounded to BF16, as every addition of
two BF16 values is.
"""

import numpy as np

from .codec import bf16_bits_to_f64, bf16_round


def residual_sum(x_bits, r_bits):
    """BF16(x + r) as float64."""
    a = bf16_bits_to_f64(x_bits).astype(np.float32) + bf16_bits_to_f64(r_bits).astype(np.float32)
    return bf16_round(a.astype(np.float64))


def rms_norm(s, w, eps):
    """(rstd [M], y [M, K]) of the stream s."""
    rstd = 1.0 / np.sqrt((s * s).mean(axis=1) + np.float64(np.float32(eps)))
    return rstd, s * rstd[:, None] * w


def rms_norm_backward(dy, s, rstd, w, ds=None):
    """(dx, dw) with the rstd that the forward pass left."""
    g, xh = dy * w, s * rstd[:, None]
    dx = rstd[:, None] * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    return dx if ds is None else dx + ds, (dy * xh).sum(axis=0)


def swiglu_backward(dh, g, u):
    """(dg, du) of h = silu(g) u."""
    with np.errstate(over="ignore"):
        sg = 1.0 / (1.0 + np.exp(-g))
    return dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg
