"""How far the attention of one new token may be from its definition in 64 bits, key by key.

With s_j the scores (natural units), M the largest, p_j = e^(s_j - lse) and o = sum p_j v_j:

* A product of 16-bit or 8-bit values is exact in fp32; hd of them are added with at most (hd + 4) 2^-24 of the sum of
  their magnitudes lost.  The scale is five roundings off at most (square root, quotient, the cache's scale, log2 e and
  its product), its product with the sum one more (2^-21 of |s_j|), the difference to the running maximum one of a
  number of at most |s_j| + |M| (2^-23 of it).  Together E_j; o moves by sum p_j E_j |v_j - o| to first order, the lse
  by sum p_j E_j.
* The exponential is 2^-22 off; so is each of the factors that a running maximum's growth brings, at most one for
  every 16 keys and a few for the joins: D of a weight.
* A weight w, 2^e <= w < 2^(e+1), enters the product with v as a pair of bf16 parts (the first leaves up to 2^(e-8), of
  which the second loses up to 2^(e-17)), a pair of f16 parts of 2^15 times it (2^(e-11), 2^(e-23); where the second is
  subnormal 2^-25, 2^-40 of the largest weight) or in fp32.
* A sum over the keys is added up in steps of 16 keys and two parts, each 2^-23 of what there is; then one division,
  one product, and one rounding to the output's type.
"""
import numpy as np
import torch

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}        # half a step of the type's subnormal numbers


def reference(q, k, v, scale):
    """q [hd], k, v [n, hd], 64 bits: scores, weights, output, lse."""
    s = scale * (k @ q)
    m = s.max()
    e = np.exp(s - m)
    return s, e / e.sum(), (e / e.sum()) @ v, m + np.log(e.sum())


def bound(q, k, v, scale, t, ct):
    """(output, its bound [hd], lse, its bound) for queries of type t on a cache of type ct; k and v as values."""
    s, p, o, lse = reference(q, k, v, scale)
    n, hd = k.shape
    E = (hd + 4) * 2.0 ** -24 * scale * (np.abs(k) @ np.abs(q)) + np.abs(s) * 2.0 ** -21 + (np.abs(s) + abs(s.max())) * 2.0 ** -23
    D = (n / 16 + 12) * 1.25 * 2.0 ** -22
    pair = {"f32": 0.0, "bf16": 2.0 ** -17}.get(ct, 2.0 ** -23)
    small = 2.0 ** -40 * p.max() if ct in ("f16", "e4m3") else 0.0
    steps = (n / 8 + 20) * 2.0 ** -23
    mass = p @ np.abs(v)
    tol = 1.01 * (p * E) @ np.abs(v - o) + (mass + np.abs(o)) * (D + pair) + small * np.abs(v).sum(0) + mass * steps
    tol += np.abs(o) * (steps + 2.0 ** -22)
    tol += HALF[t] * (np.abs(o) + tol) + LEAST[t]
    return o, tol, lse, 1.01 * p @ E + D + steps + 2.0 ** -23 * abs(lse)


def rounded(x, t):
    if t == "f32":
        return x
    return torch.from_numpy(np.asarray(x)).to({"bf16": torch.bfloat16, "f16": torch.float16}[t]).double().numpy()


def with_weights_as(q, k, v, scale, t, part, parts, up):
    """The output with weights 2^up e^(s - M) held as one or two parts of type `part`, all else exact."""
    s = scale * (k @ q)
    w = np.exp(s - s.max()) * 2.0 ** up
    held = rounded(w, part)
    if parts == 2:
        held = held + rounded(w - held, part)
    return rounded(held @ v / w.sum(), t)


def sink(g, n, hd, above, q, scale):
    """n keys of which the first has a score of `above` for each of the queries q [G, hd] and value zero; the other
    scores are of unit variance."""
    k, v = g.standard_normal((n, hd)), g.standard_normal((n, hd))
    k[0] = np.linalg.pinv(q) @ np.full(len(q), above / scale)
    v[0] = 0
    return k, v
