"""Newton-Schulz orthogonalisation and the Muon step in numpy (test infrastructure only).

``newton_schulz`` is the definition in binary64.  ``rounded`` is the same with every value that the
kernels store rounded to so many bits, along the way that they take (groups of at most three
iterations on A = X X^T, then their polynomial times X): its distance from the definition says how
far rounding of that kind moves a given matrix.  ``momentum`` is the step's element-wise part in
binary32, one rounding per operation.
"""

import numpy as np

COEFFICIENTS = (3.4445, -4.775, 2.0315)
F = np.float32


def newton_schulz(u, steps=5, eps=1e-7):
    a, b, c = COEFFICIENTS
    x = np.asarray(u, np.float64)
    x = x / max(np.linalg.norm(x), eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(steps):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if tall else x


def _round(x, bits):
    """Nearest value of ``bits`` significant bits, of at least 2^-36 apart."""
    f, e = np.frexp(x)
    step = np.exp2(np.maximum(e - bits, -36))
    return np.round(x / step) * step


def rounded(u, steps=5, eps=1e-7, bf16=False):
    """``newton_schulz`` with stored values of 22 bits; for a bf16 destination of 15, and the last group, if it
    is not the first and has at most two iterations, with 11."""
    a, b, c = COEFFICIENTS
    x = np.asarray(u, np.float64)
    x = x / max(np.linalg.norm(x), eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    one = np.eye(x.shape[0])
    done = 0
    x = _round(x, 15 if bf16 else 22)
    while done < steps:
        length = min(3, steps - done)
        bits = 22 if not bf16 else 11 if done and steps - done <= 2 else 15
        r = lambda v: _round(v, bits)  # noqa: E731,B023
        x = r(x)
        g, q = r(x @ x.T), None
        for i in range(length):
            p = r(a * one + b * g + c * (g @ g))
            q = p if q is None else r(p @ q)
            if i + 1 < length:
                g = r(r(p @ g) @ p)
        x = q @ x
        done += length
        if done < steps:
            x = _round(x, 15 if bf16 else 22)
    return x.T if tall else x


def momentum(g, m, mu, nesterov=True, scale=None):
    """(new momentum, update) in binary32."""
    g, m, mu = np.asarray(g, F), np.asarray(m, F), F(mu)
    if scale is not None:
        g = g * F(scale)
    t = g * (F(1) - mu)
    m = m * mu + t
    return m, (m * mu + t if nesterov else m)


def rate(lr, rows, cols, adjust):
    """The rate of a matrix, rounded to binary32 once."""
    size = np.sqrt(max(1.0, rows / cols)) if adjust == "original" else 0.2 * np.sqrt(max(rows, cols))
    return F(float(F(lr)) * size)


def decay(lr, weight_decay):
    return F(1.0 - float(F(lr)) * float(F(weight_decay)))
