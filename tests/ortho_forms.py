"""The orthogonalised update in 64 bits, with the roundings of qb_orthogonalize
or without them, and the bound that its results have to keep.

A result o is some r rounded to bf16, r off the formula's `want` by what the
update rounds inside.  Value by value, with d the distance of a value to the
nearest bf16 number, |o - want| <= |o - r| + |r - want| = d(r) + |r - want| <=
d(want) + 2 |r - want|; so what |o - want| has above d(want) is, as a norm, at
most twice |r - want|, however large the rounding to bf16 itself is.

|r - want|: values held in two fp16 parts and products without those of two low
parts (`held`), and sums in 32 bits (`in_32_bits`), are each simulated for the
matrix at hand.  The kernels make as many roundings of both kinds in another
order, some up and some down where the simulations go the other way: at most 4
times the two together, and 16 steps of 2^-22 where a matrix is so small that
the simulations may be right by chance.
"""
import torch

POLY = (3.4445, -4.7750, 2.0315)
X, S = 4096.0, 256.0                                   # what x, and S and P, are held times


def one(t, scale):
    return (t * scale).half().double() / scale


def two(t, scale):
    hi = one(t, scale)
    return hi + one(t - hi, scale)


def formula(x, steps=5, poly=POLY):
    a, b, c = poly
    x = x.double()
    n = torch.linalg.vector_norm(x)
    x = x / n if n > 0 else x
    tall = x.shape[0] > x.shape[1]
    x = x.T.contiguous() if tall else x
    for _ in range(steps):
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.T if tall else x


def in_32_bits(x, steps=5, poly=POLY):
    a, b, c = poly
    n = torch.linalg.vector_norm(x.double())
    x = (x.double() / n).float() if n > 0 else x.float()
    tall = x.shape[0] > x.shape[1]
    x = x.T.contiguous() if tall else x
    for _ in range(steps):
        s = x @ x.T.contiguous()
        x = a * x + (b * s + c * (s @ s)) @ x
    return (x.T if tall else x).double()


def held(x, steps=5, poly=POLY, without=()):
    """Every value in two parts.  `without`: what a wrong form leaves out, of
    "x", "S", "P" (low parts where they are written), "add x", "add S" (where
    they are added) and "S: AB" and the like (pass A part, B part of a product)."""
    a, b, c = poly
    x = x.double()
    n = torch.linalg.vector_norm(x)
    x = x / n if n > 0 else x
    tall = x.shape[0] > x.shape[1]
    x = x.T.contiguous() if tall else x

    def keep(t, scale, name):
        hi = one(t, scale)
        return hi, torch.zeros_like(hi) if name in without else one(t - hi, scale)

    def product(p, q, name):
        t = p[0] @ q[0]
        if name + ": hl" not in without:
            t = t + p[0] @ q[1]
        if name + ": lh" not in without:
            t = t + p[1] @ q[0]
        return t

    x = keep(x, X, "x")
    for _ in range(steps):
        s = keep(product(x, (x[0].T, x[1].T), "S"), S, "S")
        p = keep(b * (s[0] if "add S" in without else s[0] + s[1]) + c * product(s, s, "SS"), S, "P")
        x = keep(a * (x[0] if "add x" in without else x[0] + x[1]) + product(p, x, "Px"), X, "x")
    x = x[0] + x[1]
    return x.T if tall else x


def coarse(x, steps=5, poly=POLY):
    """qb_orthogonalize_coarse's roundings: x in one part for S and P x, and for matrices of 256 rows and more S and P in
    one part in the first three steps, the last two apart."""
    a, b, c = poly
    x = x.double()
    n = torch.linalg.vector_norm(x)
    x = x / n if n > 0 else x
    tall = x.shape[0] > x.shape[1]
    x = two(x.T.contiguous() if tall else x, X)
    for i in range(steps):
        rough = min(x.shape) >= 256 and i < 3 and i + 2 < steps
        r = one(x, X)
        s = two(r @ r.T, S)
        q = one(s, S) if rough else s
        p = (one if rough else two)(b * s + c * (q @ q), S)
        x = two(a * x + p @ r, X)
    return x.T if tall else x


def norm(t):
    return torch.linalg.vector_norm(t.double())


def above_rounding(o, want):
    """What |o - want| has above the distance of `want` to the nearest bf16 number, as a norm."""
    d = (want.to(torch.bfloat16).double() - want).abs()
    return norm(((o.double() - want).abs() - d).clamp(min=0))


def bound(x, want, **kw):
    """Of above_rounding, for a result in two parts throughout."""
    inside = norm(held(x, **kw) - want) + norm(in_32_bits(x, **kw) - want)
    return 2 * (16 * 2.0 ** -22 * norm(want) + 4 * inside)
