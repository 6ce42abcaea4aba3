"""Plain CPU oracle for the mixture-of-experts token movement: sorting by
expert, dispatch and combination of rows, and their gradients.

TEST INFRASTRUCTURE ONLY.  Only the test suite and
``__graft_entry__.smoke()`` may import or run this module.  The library under
``quantized_linear_gemm_b200/`` never calls it, links it or shares code with it.

It produces the row order and the offsets that ``moe_oracle``'s grouped
product reads (no page defines the movement itself; ai-radar.it, section
"Oltre Hopper: Blackwell, AMD, TPU e il perimetro del fork", names the expert
products).
"""

from __future__ import annotations

import numpy as np


def moe_sort(ids, E: int):
    """(offsets [E + 1], order [n], slots like ids), int32: a stable sort of
    the flattened ids; ids outside [0, E) take no row."""
    ids = np.asarray(ids)
    flat = ids.reshape(-1).astype(np.int64)
    n = flat.size
    rows = [i for e in range(E) for i in np.nonzero(flat == e)[0]]
    order = np.full(n, -1, dtype=np.int32)
    slots = np.full(n, -1, dtype=np.int32)
    for p, i in enumerate(rows):
        order[p] = i
        slots[i] = p
    counts = [int(np.sum(flat == e)) for e in range(E)]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return offsets, order, slots.reshape(ids.shape)


def permute(x, slots, base):
    """A copy of base [P, ...] with x[t] at every slot of token t that lies in [0, P)."""
    out = np.array(base)
    for t in range(slots.shape[0]):
        for s in slots[t]:
            if 0 <= s < out.shape[0]:
                out[s] = x[t]
    return out


def unpermute(y, slots, weights=None):
    """(sum_j w[t, j] y[slots[t, j]], sum of magnitudes), fp64 [T, H]."""
    y = np.asarray(y, dtype=np.float64)
    T, k = slots.shape
    out = np.zeros((T, y.shape[1]))
    mag = np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            s = int(slots[t, j])
            if 0 <= s < y.shape[0]:
                term = y[s] * (1.0 if weights is None else float(weights[t, j]))
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


def unpermute_backward(dout, y, slots, weights, base_dy):
    """(dy, dweights, sum of |dout| |y| per weight), fp64; rows of dy without a slot come from base_dy."""
    dout = np.asarray(dout, dtype=np.float64)
    y = np.asarray(y, dtype=np.float64)
    dy = np.array(base_dy, dtype=np.float64)
    T, k = slots.shape
    dw = np.zeros((T, k))
    mag = np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            s = int(slots[t, j])
            if 0 <= s < y.shape[0]:
                dy[s] = dout[t] * float(weights[t, j])
                dw[t, j] = float(dout[t] @ y[s])
                mag[t, j] = float(np.abs(dout[t]) @ np.abs(y[s]))
    return dy, dw, mag
