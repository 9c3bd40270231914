"""Data and float64 references shared by the CPU and GPU tests of linear layers
and layer norms, a ciphertext a feature."""
from __future__ import annotations

import numpy as np


def rsqrt_poly(half_width, degree=7):
    """Power-basis coefficients of a fit of (1 + u)^-1/2 on |u| <= half_width, and its largest relative error."""
    c = np.polynomial.chebyshev.Chebyshev.interpolate(lambda u: (1 + u) ** -0.5, degree, [-half_width, half_width])
    coeffs = c.convert(kind=np.polynomial.Polynomial).coef
    u = np.linspace(-half_width, half_width, 2001)
    return coeffs, float(np.max(np.abs(np.polynomial.polynomial.polyval(u, coeffs) * (1 + u) ** 0.5 - 1)))


def features(rng, F, n, pad, half_width, eps):
    """x [F][n] with every token's variance + eps in 1 +- half_width, the last `pad` tokens zero."""
    x = rng.normal(0, 1, (F, n))
    x -= x.mean(0)
    x *= np.sqrt((rng.uniform(1 - half_width, 1 + half_width, n) - eps) / (x ** 2).mean(0))
    x += rng.uniform(-1, 1, n)  # a mean of its own
    if pad:
        x[:, n - pad:] = 0
    return x


def norm_forward(x, r):
    """Normalised x [F][n] with the given rstd [n]."""
    return (x - x.mean(0)) * r


def norm_backward(dy, xhat, r, gamma):
    """(dx, the terms' largest size): rstd (g - mean g - xhat mean(g xhat)), g = gamma dy."""
    g = gamma[:, None] * dy
    m1, m2 = g.mean(0), (g * xhat).mean(0)
    return r * (g - m1 - xhat * m2), float(np.max(np.abs(r) * (np.abs(g) + np.abs(m1) + np.abs(xhat * m2))))


def norm_loss(x, dy, gamma, beta, eps):
    """sum dy (layer norm of x), per token."""
    d = x - x.mean(0)
    return (dy * (gamma[:, None] * d / np.sqrt((d ** 2).mean(0) + eps) + beta[:, None])).sum(0)


def differences(x, dy, gamma, beta, eps, h=1e-5):
    """Central differences of norm_loss in every feature."""
    out = np.empty_like(x)
    for i in range(len(x)):
        e = np.zeros_like(x)
        e[i] = h
        out[i] = (norm_loss(x + e, dy, gamma, beta, eps) - norm_loss(x - e, dy, gamma, beta, eps)) / (2 * h)
    return out
