"""Newton-Schulz orthogonalisation and the Muon step in numpy (test infrastructure only).

``newton_schulz`` is the definition in binary64.  ``rounded`` is the same with every value that the
kernels store rounded to so many bits, along the way that they take (groups of at most three
iterations on A = X X^T, then their polynomial times X): its distance from the definition says how
far rounding of that kind moves a given matrix, and ``result_bound`` how far a kernel's result may be
off before it is rounded to its destination.  ``momentum`` is the step's element-wise part in
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
    """Nearest value of ``bits`` significant bits, of at least 2^-36 apart where that is a pair of binary16
    numbers' precision or less."""
    f, e = np.frexp(x)
    step = np.exp2(np.maximum(e - bits, -36 if bits <= 22 else -1074))
    return np.round(x / step) * step


def rounded(u, steps=5, eps=1e-7, bf16=False, bits=22):
    """``newton_schulz`` with stored values of ``bits`` bits.  What is stored does not depend on whether the
    destination is ``bf16``; its own rounding is not part of this."""
    a, b, c = COEFFICIENTS
    x = np.asarray(u, np.float64)
    x = x / max(np.linalg.norm(x), eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    one = np.eye(x.shape[0])
    r = lambda v: _round(v, bits)  # noqa: E731
    done = 0
    x = r(x)
    while done < steps:
        length = min(3, steps - done)
        g, q = r(x @ x.T), None
        for i in range(length):
            p = r(a * one + b * g + c * (g @ g))
            q = p if q is None else r(p @ q)
            if i + 1 < length:
                g = r(r(p @ g) @ p)
        x = q @ x
        done += length
        if done < steps:
            x = r(x)
    return x.T if tall else x


def result_bound(u, steps=5, eps=1e-7):
    """(exact result, how far another may be off it in the Frobenius norm before it is rounded to its
    destination): 8 times what the stored values' rounding moves this matrix by, and as much again for
    binary32 sums of k terms, whose average error of sqrt(k) / 2 roundings of 2^-24 is sqrt(k) / 8 of a stored
    value's 2^-22."""
    want = newton_schulz(u, steps, eps)
    model = np.linalg.norm(rounded(u, steps, eps) - want)
    return want, 8 * model * (1 + np.sqrt(max(u.shape)) / 8) + 2.0 ** -22


def to_bf16(x):
    """Nearest bfloat16 numbers (8 bits), of magnitudes from 2^-126 on."""
    f, e = np.frexp(x)
    return np.ldexp(np.round(np.ldexp(f, 8)), e - 8)


def beyond_half(y, want):
    """By how much |y - want| exceeds half of the spacing of bfloat16 numbers at y, 0 where it does not."""
    e = np.frexp(y)[1]  # |y| in [2^(e - 1), 2^e): 2^(e - 8) apart
    return np.maximum(abs(y - want) - np.ldexp(0.5, e - 8) * (y != 0), 0.0)


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
