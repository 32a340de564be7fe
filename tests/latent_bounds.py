"""How far the latent attention's roundings may carry an output: per element the
worst case of every term at once, and as a root mean square."""
import numpy as np

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}                   # half a step of the type, relative
START = {"bf16": 28, "f16": 112}                             # a row's largest weight, at least


def absorbed(r, kind):
    """Error limits per element of the absorbed form (oracle.latent.Result ``r``).

    A query number is a sum of P e4m3 parts (bf16 2, fp16 3), each off by half a
    step of 4 bits, 2^-4 of what was left: 2^-4P of the number, or, where that is
    below e4m3's smallest step, half of it: 2^-10, against the row's largest number
    in (224, 448], 2^-17.8 of it.  q_latent's own numbers have fewer bits than the
    parts hold, so only the floor is left; the rotated numbers come by way of fp16
    as well (bf16: 2^-11; with three parts what fp16 leaves is added to what the first
    part leaves, 2^-4 of the number, rounded twice: 2^-14).  A logit moves by no more than
    those times the |k| they meet, a weight by twice that with its sum.

    Weights are split the same way, times their token's scale,
    at a scale where the largest of a part of the row is at least 28 (fp16: 112): the
    floor is 2^-10 / 28 of the row's largest product.  fp32 sums of 576 products and some
    thousand keys: 2^-16 of the terms is generous.  Then the output's rounding."""
    step = 2.0 ** -8 + 2.0 ** -11 if kind == "bf16" else 2.0 ** -12 + 2.0 ** -14
    logit = step * r.turned + 2.0 ** -17.8 * r.ones + 2.0 ** -18 * r.all
    weight = step + 2.0 ** -16
    bound = r.spread * (np.expm1(2 * logit)[..., None] + weight) + r.floor * 2.0 ** -10 / START[kind]
    return _rounded(bound, r, kind)


def expanded(r, kind):
    """The expanded form: rotated queries rounded once to the type, weights to sums of
    two numbers of it (2^-16, or less); the rest as above."""
    logit = U[kind] * r.turned + 2.0 ** -18 * r.all
    weight = 2.0 ** -16 + 2.0 ** -16
    return _rounded(r.spread * (np.expm1(2 * logit)[..., None] + weight), r, kind)


def _rounded(bound, r, kind):
    return bound * (1 + U[kind]) + np.abs(r.out) * U[kind] + (2.0 ** -24 if kind == "f16" else 0.0) + 1e-30


def absorbed_rms(r, kind):
    """Root mean square over all elements.  An error spread evenly over +- h has the
    mean square h^2 / 3; errors of a row's weights are independent, so their squares
    add.  The parts' errors are taken at their worst size (2^-8, 2^-12) for every
    weight, logits' at theirs: a part that is lost is 2^-4 of a weight, sixteen
    (two hundred) times as much."""
    step = 2.0 ** -8 + 2.0 ** -11 if kind == "bf16" else 2.0 ** -12 + 2.0 ** -14
    logit = step * r.turned + 2.0 ** -17.8 * r.ones
    square = r.square * (step ** 2 / 3 + (4 * logit[..., None] ** 2) / 3) + r.out ** 2 * U[kind] ** 2 / 3 \
        + (r.spread * 2.0 ** -16) ** 2 + (r.floor * 2.0 ** -10 / START[kind]) ** 2 / 3 / 64
    return float(np.sqrt(square.mean()))
