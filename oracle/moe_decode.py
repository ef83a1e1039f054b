"""The routed-expert layer with NVFP4 weights and activations that are not quantized.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Routing as in ``moe`` (top-k, equal logits by lower id, softmax over the selected); per
token and selected expert ``h = SiLU(Wg x) * (Wu x)``, ``out = sum_j w_j Wd h_j``, everything
in float64 over exactly dequantized weights.

``forward`` also returns a bound on the error of a float32 evaluation, carried through the
layer element by element: a sum of n products rounds at most n times by 2**-23 of the sum
of absolute values (as in ``fp8_block``); |SiLU'| <= 1.1; the gate's exponential, reciprocal and
products cost a few units of 2**-23 of |h|; routing weights are within 16 * 2**-24 of theirs.
Carrying x and h as f16 values under a power of two costs, per value, 2**-11 (one f16, half
a step) or 2**-22 (the rounding of what one f16 leaves, in a second), and half the smallest f16
step, 2**-25, under a row maximum of at least 2**14: 2**-39 of the row's largest value.
Below 2**-126 a float32 may lose all of itself: that much for an h (the product of a gate and
an up value, each in range) and for a product of the down projection and its weighted sum.
"""

import numpy as np

from .moe import route
from .nvfp4 import dequantize

U = 2.0 ** -23
TINY = 2.0 ** -126


def _dequant(w, e):
    q, s, g = w
    return dequantize(np.asarray(q)[e], np.asarray(s)[e], np.asarray(g)[e])


def forward(x, logits, k, w_gate_up, w_down, x_bits=22, h_bits=22):
    """(out, bound), float64 [T, H].  ``x_bits``: None for an x that f16 holds exactly."""
    x = np.asarray(x, dtype=np.float64)
    T, H = x.shape
    ids, w = route(logits, k)
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        wgu, wd = _dequant(w_gate_up, e), _dequant(w_down, e)
        inter = wd.shape[1]
        z = x[t] @ wgu.T
        dx = 2.0 ** -39 * np.abs(x[t]).max(1, keepdims=True) + (0 if x_bits is None else 2.0 ** -x_bits) * np.abs(x[t])
        ez = ((H + 4) * U * np.abs(x[t]) + dx) @ np.abs(wgu).T
        (zg, zu), (eg, eu) = np.split(z, 2, 1), np.split(ez, 2, 1)
        act = zg / (1.0 + np.exp(-zg))
        h = act * zu
        eh = 1.1 * eg * np.abs(zu) + np.abs(act) * eu + 1.1 * eg * eu
        # e^-z: |z| 2^-23 of the exponent's own rounding, at most |z| * silu's slope again
        eh = eh + (np.abs(h) + 1.1 * np.abs(zg * zu)) * 8 * U
        eh = eh + np.abs(h) * 2.0 ** -h_bits + 2.0 ** -39 * np.abs(h).max(1, keepdims=True) + TINY
        wj = w[t, j][:, None]
        np.add.at(out, t, wj * (h @ wd.T))
        np.add.at(bound, t, wj * (eh @ np.abs(wd).T + (inter + k + 24) * U * (np.abs(h) @ np.abs(wd).T))
                  + (inter + k) * TINY)
    return out, bound
