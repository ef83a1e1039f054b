"""The routed-expert layer with NVFP4 weights and activations that are not quantized.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Routing as in ``moe`` (top-k, equal logits by lower id, softmax over the selected); per
token and selected expert ``h = SiLU(Wg x) * (Wu x)``, ``out = sum_j w_j Wd h_j``, everything
in float64 over exactly dequantized weights.

``forward`` also returns a bound on the error of a float32 evaluation, carried through the
layer element by element: a sum of n products rounds at most n times by 2**-23 of the sum
of absolute values (as in ``fp8_block``); |SiLU'| <= 1.1; the gate's exponential, reciprocal and
products cost a few units of 2**-23 of |h|, and carrying h to ``h_bits`` bits costs
2**-h_bits of it; routing weights are within 16 * 2**-24 of theirs.
"""

import numpy as np

from .moe import route
from .nvfp4 import dequantize

U = 2.0 ** -23


def _dequant(w, e):
    q, s, g = w
    return dequantize(np.asarray(q)[e], np.asarray(s)[e], np.asarray(g)[e])


def forward(x, logits, k, w_gate_up, w_down, h_bits=24):
    """(out, bound), float64 [T, H]."""
    x = np.asarray(x, dtype=np.float64)
    T, H = x.shape
    ids, w = route(logits, k)
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        wgu, wd = _dequant(w_gate_up, e), _dequant(w_down, e)
        inter = wd.shape[1]
        z = x[t] @ wgu.T
        ez = (H + 4) * U * (np.abs(x[t]) @ np.abs(wgu).T)
        (zg, zu), (eg, eu) = np.split(z, 2, 1), np.split(ez, 2, 1)
        act = zg / (1.0 + np.exp(-zg))
        h = act * zu
        eh = 1.1 * eg * np.abs(zu) + np.abs(act) * eu + 1.1 * eg * eu
        # e^-z: |z| 2^-23 of the exponent's own rounding, at most |z| * silu's slope again
        eh = eh + (np.abs(h) + 1.1 * np.abs(zg * zu)) * 8 * U + np.abs(h) * 2.0 ** -h_bits
        wj = w[t, j][:, None]
        np.add.at(out, t, wj * (h @ wd.T))
        np.add.at(bound, t, wj * (eh @ np.abs(wd).T + (inter + k + 24) * U * (np.abs(h) @ np.abs(wd).T)))
    return out, bound
