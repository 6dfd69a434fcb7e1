"""Bounds for the 16-bit attention outputs and the rotated rows (not a test module; no GPU).

Attention.  With u = half a step of the 16-bit type (fp16 2^-11, bf16 2^-8, relative):
* each softmax weight is rounded to the type before it multiplies v: at most u per weight, so at
  most u * sum_t p_t |v_t| = u * size (weights that fall below the type's normal range keep an
  absolute error that is smaller still: at most 2^-34 of the largest weight each);
* the result is rounded to the type: u * |out| (and half the least subnormal, 2^-25, in fp16);
* a score is a float32 sum of D products: at most D 2^-23 span off, span = scale * sum_d |q_d k_d|
  (2^-23: the tensor cores may cut where float32 rounds); its exponential is 2^-21 off in itself,
  and its argument's rounding is covered by taking D + 8.  A weight moves by that relative error,
  and so does their sum: twice it, times size.  Sums of up to 2^18 terms in float32 add 2^-20.
"""
from __future__ import annotations

import numpy as np

HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def score_error(D: int, span):
    return (D + 8) * 2.0 ** -23 * span + 2.0 ** -20


def attn_tolerance(ref_out, size, span, D: int, kind: str):
    u = HALF_STEP[kind]
    e = score_error(D, np.asarray(span))[..., None]
    return u * (1 + 4 * u) * (size + np.abs(ref_out)) + 2 * e * size + 2.0 ** -25


def assert_rows_close(got, ref_out, size, span, kind: str, ctx: str = "") -> None:
    got = np.asarray(got, dtype=np.float64)
    tol = attn_tolerance(ref_out, size, span, got.shape[-1], kind)
    bad = ~(np.abs(got - ref_out) <= tol)
    assert not bad.any(), (
        f"{ctx}: {int(bad.sum())} of {bad.size} outside; first at {np.argwhere(bad)[0]}, worst "
        f"{np.nanmax(np.abs(got - ref_out) / tol):.3g} of the tolerance")


def assert_lse_close(got, ref, span, D: int, ctx: str = "") -> None:
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    none = np.isneginf(ref)
    assert np.array_equal(np.isneginf(got), none), f"{ctx}: rows without keys"
    tol = score_error(D, np.asarray(span)) + 2.0 ** -22 * np.abs(np.where(none, 0, ref)) + 2.0 ** -20
    d = np.abs(np.where(none, 0, got) - np.where(none, 0, ref))
    assert (d <= tol).all(), f"{ctx}: lse off by {d.max():.3g}"


def norm_rope_tolerance(x, w, ref, eps: float, kind: str):
    """Half a step of the result, plus what float32 costs before it: the mean of D squares
    (D + 2 roundings), the square root's reciprocal (2 ulp), four products and sums, and the
    sine and cosine's 2^-21 of the pair's magnitude -- all relative to the row's largest value."""
    y = np.abs(np.asarray(x, dtype=np.float64))
    D = y.shape[-1]
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.abs(np.asarray(w, np.float64))
    big = y.max(-1, keepdims=True)
    return (HALF_STEP[kind] * np.abs(ref) + 2 * big * ((D + 2) * 2.0 ** -25 + 8 * 2.0 ** -24
                                                       + 2.0 ** -20) + 2.0 ** -25)
