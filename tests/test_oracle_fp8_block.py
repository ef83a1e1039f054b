"""Pins of the block-scaled FP8 oracle and of the few-token routed-expert oracle (no GPU):
exact rational arithmetic, representable inputs that must survive, edge blocks, one-hot
operands that expose a transposed or shifted scale, and agreement with the routed oracle's
own stages."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import fp8_block as P
from oracle import moe as OM
from oracle import moe_decode as OD
from oracle.formats import e4m3_decode


def _nearest(y):
    """E4M3 code of a non-negative rational by brute force, ties to the even code."""
    best = min(range(127), key=lambda c: (abs(y - Fraction(float(e4m3_decode(c)))), c % 2))
    return best


@pytest.mark.parametrize("amax", [1.0, 0.75, 3.0, 448.0, 1e-3])
def test_codes_against_exact_rationals(amax):
    """Values on and next to the midpoints of the rounded scale's grid, where a float32
    quotient may land on a midpoint that the real one misses."""
    rng = np.random.default_rng(3)
    s = np.float32(max(np.float32(amax) / np.float32(448.0), np.float32(2.0 ** -126)))
    mids = (e4m3_decode(np.arange(126)) + e4m3_decode(np.arange(1, 127))) / 2
    x = np.float32(mids * float(s))
    x = np.concatenate([[np.float32(amax)], x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(1e9)),
                        np.float32(amax) * np.float32(3.0) * np.exp2(-rng.integers(2, 20, 40))]).astype(np.float32)
    x = x[np.abs(x) <= amax]
    for lo in range(0, len(x), 127):
        row = np.zeros((1, 128), np.float32)
        row[0, 0] = amax
        part = x[lo:lo + 127]
        row[0, 1:1 + len(part)] = part
        q, sc = P.quantize(row)
        assert sc[0, 0] == s
        for xi, qi in zip(row[0], q[0]):
            assert qi == _nearest(min(Fraction(float(xi)) / Fraction(float(s)), Fraction(448)))


def test_blocks_edges_and_zeros():
    x = np.zeros((130, 272), np.float32)
    x[0, 0] = -448.0
    x[127, 127] = 2.0
    x[129, 271] = 896.0
    for br, shape in ((1, (130, 3)), (128, (2, 3))):
        q, s = P.quantize(x, br)
        assert s.shape == shape
        want = x.astype(np.float64)
        if br == 1:  # the row's own scale, 2 / 448, is no float32: 448 times its rounding comes back
            want[127, 127] = 448.0 * float(np.float32(2.0) / np.float32(448.0))
        np.testing.assert_array_equal(P.dequantize(q, s, br), want)
    q, s = P.quantize(x, 128)
    assert s[0, 0] == 1.0 and s[1, 2] == 2.0 and s[0, 1] == 1.0
    _, s = P.quantize(np.full((1, 16), 2.0 ** -140, np.float32))
    assert s[0, 0] == np.float32(2.0 ** -126)


def test_gemm_picks_the_block_scales():
    M, N, K = 3, 257, 272
    aq, bq = np.zeros((M, K), np.uint8), np.zeros((N, K), np.uint8)
    a_s = np.arange(1, M * 3 + 1, dtype=np.float32).reshape(M, 3)
    b_s = (10.0 ** np.arange(9)).astype(np.float32).reshape(3, 3)
    one = 0x38
    for m in range(M):
        for k in (0, 127, 128, 255, 256, 271):
            aq[:], bq[:] = 0, 0
            aq[m, k] = one
            bq[:, k] = one
            y = P.gemm(aq, a_s, bq, b_s)
            np.testing.assert_array_equal(y[m], np.repeat(a_s[m, k // 128] * b_s[:, k // 128], 128)[:N])
            assert not np.any(np.delete(y, m, 0))
            assert np.all(P.gemm_bound(aq, a_s, bq, b_s) >= 0)


def test_decode_layer_matches_the_routed_stages():
    """With activations that NVFP4 would carry exactly nothing distinguishes the layers up to h."""
    rng = np.random.default_rng(5)
    T, E, k, H, I = 5, 6, 3, 48, 32
    x = rng.standard_normal((T, H)).astype(np.float32)
    lg = rng.standard_normal((T, E)).astype(np.float32)
    gu = OM.quantize_experts(rng.standard_normal((E, 2 * I, H)).astype(np.float32))
    dn = OM.quantize_experts(rng.standard_normal((E, H, I)).astype(np.float32))
    out, bound = OD.forward(x, lg, k, gu, dn)
    want = np.zeros((T, H))
    ids, w = OM.route(lg, k)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            wg, wd = OD._dequant(gu, e), OD._dequant(dn, e)
            want[t] += w[t, j] * (wd @ OM.silu_gate((wg @ x[t].astype(np.float64))[None])[0])
    np.testing.assert_allclose(out, want, rtol=1e-12, atol=1e-12)
    assert np.all(bound > 0) and np.all(bound < 1e-2 * np.abs(out).max())
