"""The orthogonalising iteration in 64 bits, and how far the kernels may be off.

In the 2-norm over a matrix, relative to the result:
* ``half``: A and B are rounded to fp16 (2^-11 of each value at most, 2^-11 / sqrt(3) in
  the mean square), X to fp16 where it is multiplied.  Each step's error in B X is at most
  (|b| s^2 + 2 |c| s^4) times the rounding of the factors, s the largest singular value: with
  s <= 1.2 some 16 * 2^-11 / sqrt(3) where every value had the largest rounding and all
  directions the largest s; the values that the iteration has near its end (s between 0.7
  and 1.2, b s^2 + c s^4 about -2.5) give a quarter of it, 4 * 2^-11 / sqrt(3) = 2^-9.8, and
  errors of the steps before are damped (the slope of the polynomial there is below 1 in
  size).  HALF_OFF takes twice that, for two such steps.
* exact: fp16 pairs carry 22 bits, the dropped products 2^-22 of each, sums over up to
  thousands of products in fp32 some 2^-21; the polynomial's slope of up to |a| = 3.5 per
  step for small singular values multiplies only errors of X itself, which is kept in fp32:
  3.5^5 * 2^-24 = 2^-15 at worst, for a matrix whose singular values are all tiny beside one
  of them.  EXACT_OFF is for the random matrices of the tests, 2^-17.
"""

import torch

COEFF = (3.4445, -4.7750, 2.0315)
HALF_OFF = 2.0 ** -8.5
EXACT_OFF = 2.0 ** -17
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def reference(g, steps=5, coefficients=COEFF, eps=1e-7):
    a, b, c = coefficients
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (x.norm() + eps)
    for _ in range(steps):
        A = x @ x.T
        x = a * x + (b * A + c * A @ A) @ x
    return x.T if tall else x


def check(got, want, half, scale=1.0):
    """got: bf16 or fp32, want: 64 bits; ``scale``: 2-norm that the error belongs to, as a
    share of want's (an update inside a weight)."""
    assert got.shape == want.shape
    assert got.isfinite().all()
    off = (HALF_OFF if half else EXACT_OFF) * scale + ROUND[got.dtype]
    e = (got.double() - want).norm() / want.norm()
    assert e <= off, (float(e), off)
    # single values: four standard deviations of an error spread evenly would be below
    # six; a tile that is wrong or missing is far above
    rms = want.norm() / want.numel() ** 0.5
    worst = ((got.double() - want).abs() / torch.maximum(rms, want.abs())).max()
    assert worst <= 24 * off, (float(worst), off)
