"""Plain 64-bit definitions of the norm, the activations and the products' epilogue, in numpy, and the errors that
FP32 arithmetic in the kernels' order may have. U is half a step of FP32, relative to the value; a division, a square
root and an addition are off by one U at most, the hardware's reciprocal and power of two by two."""
from __future__ import annotations

import numpy as np
import torch
from scipy import special

from tests import _fp8 as R

U = 2.0 ** -24
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def plain(x):
    return x.double().cpu().numpy()


def activation(p, name, short=False):
    """(value, slope, error of the value, error of the slope), the errors in U; short: as for results of 16 bits.

    A sigmoid is off by 4 (exp_below: power of two 2, its correction 1, products 1) + 1 (sum) + 2 (reciprocal) + 1
    (product) = 8, and by what the rounding of its argument x changes it, (1 - s) |x| times x's relative error. The
    short one's exponential has no correction: its argument is off by 2 (silu: a product and its constant) or 4 (tanh: a
    square, a fused product, a product, constants), and 1 - s is a difference, off by s's error and half a step of 1.
    The normal integral's tail: 2 of the power of two, p^2/2 times its argument's 2, a reciprocal of a rounded sum (3)
    that changes the polynomial by 4 times as much at most, nine steps of a polynomial whose terms add up to 2.2 times
    its value (20 at most), 1 of the fit (144 of the short one, 8.6e-6), 2 of products: 37 (180). A power of two under
    2^-126 is zero in the hardware's instruction: the sigmoid or the integral loses less than that (gelu at p = -13.4375,
    u = 4.375: exp(-p^2/2) = 6.2e-40 and z = -1.07e-39 come out as 0).
    """
    lost = 2.0 ** -126 / U
    with np.errstate(over="ignore", invalid="ignore"):
        if name == "none":
            return p, np.ones_like(p), 0 * p, 0 * p
        if name == "relu":
            return np.where(p <= 0, 0.0, p), np.where(p <= 0, 0.0, np.where(p > 0, 1.0, p)), 0 * p, 0 * p
        q = np.clip(p, -1e4, 1e4)
        if name == "gelu":
            below, above, density = special.ndtr(q), special.ndtr(-q), np.exp(-0.5 * q * q) / np.sqrt(2 * np.pi)
            value, slope = np.where(p > 1e4, p, q * below), below + q * density
            tail = ((180 if short else 37) + q * q) * np.minimum(below, above)
            return (value, slope, np.abs(q) * (tail + lost) + 2 * np.abs(value),
                    tail + 2 * below + (8 + q * q) * np.abs(q) * density + (1 + np.abs(q)) * lost)
        if name == "silu":
            a, b, off = q, np.ones_like(q), 2.0 if short else 0.0
        else:
            k = np.sqrt(2 / np.pi)
            a, b, off = 2 * k * (q + 0.044715 * q ** 3), 2 * k * (1 + 3 * 0.044715 * q ** 2), 4.0 if short else 6.0
        s, c = special.expit(a), special.expit(-a)
        rel = 8 + off * np.minimum(np.abs(a), 200) * c  # of s
        value, slope = np.where(p > 1e4, p, q * s), s + q * b * s * c
        # 1 - s: relative in the long form, the difference's half step and s's own error in the short one
        rest = s * c * (rel + 12 + off * np.minimum(np.abs(a), 200)) if not short else s * (1 + rel * s) + s * c * (rel + 12)
        return (value, slope, (rel + 2) * np.abs(value) + np.abs(q) * lost,
                (rel + 2) * s + np.abs(q) * b * rest + (1 + np.abs(q) * b) * lost)


def quantised(Q, S, want, error):
    """Asserts that Q, S are `want`'s rows in e4m3 with scales for blocks of 128, `error` the absolute error that the
    kernel's FP32 values may have before the rounding."""
    q, s = R.bytes_of(Q), S.cpu().numpy().astype(np.float64)
    n, k = want.shape
    assert Q.shape == (n, k) and Q.stride(0) % 16 == 0 and s.shape == (n, -(-k // 128))
    for b in range(s.shape[1]):
        at = slice(b * 128, b * 128 + 128)
        size, slack = np.abs(want[:, at]).max(1), error[:, at].max(1)
        scale = np.maximum(size, 2.0 ** -64) / 448
        np.testing.assert_array_less(np.abs(s[:, b] - scale), slack / 448 + 3 * U * scale + 1e-300)
        # half a step of e4m3 (2^-4 of the value, 2^-10 below the normal numbers), at a quotient that is off itself
        quotient = want[:, at] / s[:, b:b + 1]
        moved = error[:, at] / s[:, b:b + 1] + 3 * U * np.abs(quotient)
        off = np.abs(q[:, at] - quotient)
        assert (off <= np.maximum(2.0 ** -4 * np.abs(quotient), 2.0 ** -10) + 2 * moved).all(), off.max()


def near(got, want, error, kind):
    """Asserts a result of type `kind` whose FP32 value may be off by `error`."""
    rel, least = R.half_step(kind)
    got = plain(got)
    bound = error + rel * (np.abs(want) + error) + least
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - want) / bound)[bad].max()))


def norm(h, w, eps):
    """(rstd, y) of rows h."""
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    return rstd, h * rstd[:, None] * w


def norm_backward(dy, h, rstd, w, dh):
    """(dx, dw, error of dx, error of dw / U without the rows' sum) for the rows' FP32 rstd."""
    n, g = h * rstd[:, None], w * dy
    mean, size = (g * n).mean(1, keepdims=True), np.abs(g * n).mean(1, keepdims=True)
    dx = rstd[:, None] * (g - n * mean) + dh
    # n, g: one rounding each; the mean of g n: 16 additions of a thread, 6 of a wave, 16 of waves, with the products'
    # and the division's roundings 44; then two products, two sums
    error = U * (rstd[:, None] * (4 * np.abs(g) + (48 + 4) * np.abs(n) * size) + 2 * np.abs(dx) + np.abs(dh))
    return dx, (dy * n).sum(0), error, np.abs(dy * n).sum(0)
