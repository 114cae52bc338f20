"""Bounds shared by the tests of the packed and cached attention calls."""
import numpy as np


def tolerances(q, k, scale, mag, o_ref):
    """(per-element bound on O, bound on LSE), from the arithmetic:

    * a score is an fp32 sum of d exact bf16 products: off by at most d 2^-23 |q||k| scale; the
      scaled, shifted exponent rounds by 2^-23 of its size (at most 2 scale |q||k| + 8);
    * an exponential is off by 7.5e-5 (FMA-pipe polynomial) or 2^-21 (MUFU) of its value, so a
      weight by eps in all; the row sum and its log add 2^-20;
    * P is rounded to bf16 (half a step: 2^-8 of the value), O once more.
    """
    d = q.shape[-1]
    size = scale * float(q.double().norm(dim=-1).max()) * float(k.double().norm(dim=-1).max() if k.numel() else 0)
    eps = np.expm1(d * 2.0 ** -23 * size + 2.0 ** -23 * (2 * size + 8)) + 7.5e-5 + 2.0 ** -20
    return (2.0 ** -8 + 2.1 * eps) * mag + 2.0 ** -8 * np.abs(o_ref) * (1 + 2.0 ** -7) + 1e-30, eps + 2.0 ** -20
