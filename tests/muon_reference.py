"""The Newton-Schulz steps of the Muon update in 64 bits, and how far an evaluation with products of two f16 parts and
sums in f32 may be off in the Frobenius norm (any device)."""
import math

import torch

A, B, C = 3.4445, -4.7750, 2.0315
u = 2.0 ** -24
SCALE_X, SCALE_P = 2.0 ** 15, 2.0 ** 14   # of X and G, and of P, before they are split


def _norm(x):
    return float(torch.linalg.vector_norm(x))


def _product_error(a, b, scale_a, scale_b, out):
    """Of a b in f32 from two f16 parts a factor: each holds 2^-22 of a value (or half of 2^-24 over its scale, where
    that is more), the product of the low parts, 2^-22 again, is left out: 3 2^-22 of each product, independently, so
    of the root of their squares.  An addition is off by up to 2 u of what its sum has reached, evenly: by
    2 u / sqrt(3) in the mean.  A sum of k terms of either sign reaches sqrt(j) of them after j: sqrt(k / 2) in all.  On
    the diagonal of a symmetric product all terms are positive and the sum reaches j / k of its whole: sqrt(k / 3)."""
    k = a.shape[1]
    squares = math.sqrt(float(((a * a).sum(0) * (b * b).sum(1)).sum()))
    tiny = 2.0 ** -25 * (math.sqrt(a.numel()) / scale_a * _spectral(b) + math.sqrt(b.numel()) / scale_b * _spectral(a))
    diagonal = _norm(out.diagonal()) if out.shape[0] == out.shape[1] else 0.0
    add = 2 * u / math.sqrt(3)
    return (3 * 2.0 ** -22 + add * math.sqrt(k / 2)) * squares + add * math.sqrt(k / 3) * diagonal + tiny


def _spectral(x):
    """An upper bound of the spectral norm: the square root of |x x^T|."""
    g = x @ x.T if x.shape[0] <= x.shape[1] else x.T @ x
    return math.sqrt(_norm(g))


def _step(Y):
    G = Y @ Y.T
    GG = G @ G
    P = B * G + C * GG
    PY = P @ Y
    return G, GG, P, PY, A * Y + PY


def newton_schulz(v, steps, off=0.0):
    """X after `steps` steps from v (f64), and the bound on its error.  off: of v itself, relative to |v|.

    A step's own roundings: G's go through P = b G + c G^2 (|b| + 2 |c| |G| times), P's are multiplied with X, each
    elementwise combination rounds three times.  What the steps that follow make of an error is taken from 64 bits: a
    random change of 1e-6 of |X| is carried through them beside X.  Errors of the steps look like random changes to the
    steps that follow, so that twice its growth is allowed (and at least 1 for what the change's own direction
    misses)."""
    Y = v / (v.norm() + 1e-7)
    tall = v.shape[0] > v.shape[1]
    Y = Y.T if tall else Y
    gen = torch.Generator(device=v.device).manual_seed(1)
    at, own = [Y], [3 * u + off]
    for _ in range(steps):
        G, GG, P, PY, Z = _step(Y)
        own_g = _product_error(Y, Y.T, SCALE_X, SCALE_X, G)
        own_p = (abs(B) + 2 * C * min(1.47, _norm(G))) * own_g + C * _product_error(G, G, SCALE_X, SCALE_X, GG) + \
            3 * u * (abs(B) * _norm(G) + C * _norm(GG))
        own.append(min(1.21, _spectral(Y)) * own_p + _product_error(P, Y, SCALE_P, SCALE_X, PY) +
                   3 * u * (A * _norm(Y) + _norm(PY)))
        Y = Z
        at.append(Y)
    e = 0.0
    for t in range(steps + 1):
        change = torch.randn(Y.shape, generator=gen, device=v.device, dtype=torch.float64)
        change *= 1e-6 * _norm(at[t]) / _norm(change)
        Z = at[t] + change
        for _ in range(steps - t):
            Z = _step(Z)[4]
        e += own[t] * max(1.0, 2.0 * _norm(Z - Y) / _norm(change))
    return (Y.T if tall else Y), e


def emulated(v, steps, parts=2, dtype=torch.float16, spoil=None):
    """X as the kernels form it, on the CPU in f32: products of `parts` parts a factor.  spoil(X): after each step."""
    x = v.double()
    x = (x / (x.norm() + 1e-7)).float()
    tall = v.shape[0] > v.shape[1]
    x = x.T.contiguous() if tall else x

    def split(t, scale):
        out, t = [], t * scale
        for _ in range(parts):
            h = t.to(dtype).float()
            out.append(h / scale)
            t = t - h
        return out

    def product(a, b, sa, sb):
        a, b = split(a, sa), split(b, sb)
        y = a[0] @ b[0]
        return y if parts == 1 else (a[0] @ b[1] + a[1] @ b[0]) + y

    for _ in range(steps):
        g = product(x, x.T, SCALE_X, SCALE_X)
        p = C * product(g, g, SCALE_X, SCALE_X) + B * g
        x = A * x + product(p, x, SCALE_P, SCALE_X)
        if spoil is not None:
            spoil(x)
    return x.T if tall else x
