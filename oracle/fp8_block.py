"""FP8 (E4M3) linear layer with one scale per block of 128: quantize, dequantize, GEMM.

TEST INFRASTRUCTURE ONLY (see the package docstring).

A tensor [rows, cols] is cut into blocks of 128 columns by 1 row (activations) or 128
rows (weights); blocks at the right and lower edges are shorter.  Per block:

* ``s = max(fl(amax / 448), 2**-126)`` in float32, or 1 for a block of zeros;
* the code of ``x`` is the E4M3FN code nearest the real quotient ``x / s``, ties to the
  even code, with the sign of ``x``.  The quotient is formed in float64: two float32
  values whose quotient is not a midpoint ``t`` of two codes differ from it by at least
  ``2**-30`` relatively (``x - t s`` is a multiple of an ulp of ``t s``, whose significand has
  at most 29 bits), far more than float64 rounds by, and a quotient that is one is
  exact in float64, so the search decides as exact arithmetic would.

GEMM: ``Y = A_hat @ B_hat^T`` with ``A`` [M, K] of 1 x 128 blocks and ``B`` [N, K] of
128 x 128 blocks, in float64.
"""

import numpy as np

from .formats import E4M3_MAX, E4M3_NONNEG, _nearest_code, e4m3_decode

BLOCK = 128


def _blocks(n):
    return -(-n // BLOCK)


def _spread(s, block_rows, rows, cols):
    """A block scale array repeated to [rows, cols] (float64)."""
    return np.repeat(np.repeat(np.asarray(s, np.float64), block_rows, 0), BLOCK, 1)[:rows, :cols]


def scales(x, block_rows):
    x = np.abs(np.asarray(x, dtype=np.float32))
    rows, cols = x.shape
    amax = np.array([[x[r:r + block_rows, c:c + BLOCK].max() for c in range(0, cols, BLOCK)]
                     for r in range(0, rows, block_rows)], dtype=np.float32).reshape(-1, _blocks(cols))
    s = np.maximum(amax / np.float32(E4M3_MAX), np.float32(2.0 ** -126)).astype(np.float32)
    return np.where(amax == 0, np.float32(1.0), s)


def quantize(x, block_rows=1):
    """(q uint8 of x's shape, s float32 [ceil(rows / block_rows), ceil(cols / 128)])."""
    x = np.asarray(x, dtype=np.float32)
    if not np.all(np.isfinite(x)):
        raise ValueError("fp8 block quantize: non-finite input")
    s = scales(x, block_rows)
    y = np.minimum(np.abs(x).astype(np.float64) / _spread(s, block_rows, *x.shape), E4M3_MAX)
    code = _nearest_code(y, E4M3_NONNEG).astype(np.uint8)
    return (np.signbit(x).astype(np.uint8) << 7) | code, s


def dequantize(q, s, block_rows=1):
    """Exact float64 values."""
    return e4m3_decode(q) * _spread(s, block_rows, *np.shape(q))


def gemm(a_q, a_s, b_q, b_s):
    """Y [M, N] (float64)."""
    return dequantize(a_q, a_s, 1) @ dequantize(b_q, b_s, BLOCK).T


def gemm_bound(a_q, a_s, b_q, b_s, fp8_unit=False):
    """Elementwise bound on the error of a float32 evaluation of the same sums.

    Each output sums K exact products; the additions inside a block (at most 128) and over
    the blocks, the product of the two scales and its product with the block's sum each
    round once, by at most 2**-23 of the running absolute sum (2**-24 to nearest; doubled, since
    a matrix unit may cut instead).

    ``fp8_unit``: the products go through the FP8 matrix unit, which adds those of eight
    consecutive k at a common scale: every product but the largest is cut towards zero to a
    multiple of ``2**-13 * 2**(ea + eb)``, ``ea`` and ``eb`` the exponents of the largest product's
    factors, so that unit is at most ``2**-13`` of the largest product, which is at most the
    largest ``|a|`` times the largest ``|b|`` of the eight.  Seven cuts per group."""
    a, b = np.abs(dequantize(a_q, a_s, 1)), np.abs(dequantize(b_q, b_s, BLOCK))
    terms = min(BLOCK, np.shape(a_q)[1]) + np.shape(a_s)[1] + 3
    bound = terms * 2.0 ** -23 * (a @ b.T)
    if fp8_unit:  # K is a multiple of 16: whole groups
        ga, gb = (v.reshape(v.shape[0], -1, 8).max(2) for v in (a, b))
        bound += 7 * 2.0 ** -13 * (ga @ gb.T)
    return bound
