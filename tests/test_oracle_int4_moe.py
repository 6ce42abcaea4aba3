"""Pins of the 4-bit weight oracle and of the token-movement oracle on values
worked out by hand.  CPU only."""

import numpy as np
import pytest

from oracle import int4_oracle as I
from oracle import moe_tokens_oracle as T


def test_pack_puts_the_even_k_in_the_low_half():
    q = np.array([[1, 2, 15, 0, 7, 8, 3, 4]], dtype=np.uint8)
    b = I.pack(q)
    assert b.tolist() == [[0x21, 0x0F, 0x87, 0x43]]
    assert np.array_equal(I.unpack(b), q)


def test_symmetric_group_by_hand():
    w = np.zeros((1, 32), dtype=np.float32)
    w[0, :8] = [7.0, -7.0, 0.5, 1.5, 2.5, -0.5, 3.49, -8.0]     # amax 8: s = bf16(8 / 7) = 1.140625
    q, s, z = I.quant_weight_int4(w, 32, False)
    assert z is None and s[0, 0] == np.float32(1.140625)
    codes = I.unpack(q)[0]
    want = [np.clip(np.rint(np.float32(v) / np.float32(1.140625)), -8, 7) + 8 for v in w[0]]
    assert codes.tolist() == want
    assert codes[7] == 1 and codes[0] == 14 and codes[8] == 8


def test_group_with_zero_points_by_hand():
    w = np.zeros((1, 32), dtype=np.float32)
    w[0, 0], w[0, 1], w[0, 2] = 3.0, -12.0, 0.5                  # hi - lo = 15: s = 1, z = 12
    q, s, z = I.quant_weight_int4(w, 32, True)
    codes = I.unpack(q)[0]
    assert s[0, 0] == 1.0 and z[0, 0] == 12
    assert codes[:4].tolist() == [15, 0, 12, 12]                 # 0.5 rounds to even: 0
    d = I.dequant(q, s, z)
    assert d[0, :3].tolist() == [3.0, -12.0, 0.0]


def test_all_zero_group_gets_the_smallest_scale():
    for zp in (False, True):
        q, s, z = I.quant_weight_int4(np.zeros((2, 64), dtype=np.float32), 32, zp)
        assert np.all(s == np.float32(2.0 ** -126)) and np.all(I.dequant(q, s, z) == 0)


def test_product_by_hand():
    q = np.full((1, 32), 8, dtype=np.uint8)
    q[0, 3], q[0, 30] = 10, 5                                   # 2 and -3 without zero points
    x = np.zeros((1, 32))
    x[0, 3], x[0, 30] = 4.0, 1.0
    c, mag = I.int4_mm_ref(x, I.pack(q), [[0.5]], None, bias=[10.0])
    assert c[0, 0] == 10.0 + 0.5 * (8 - 3) and mag[0, 0] == 10.0 + 0.5 * 11


def test_sort_by_hand():
    off, order, slots = T.moe_sort(np.array([[2, 0], [-1, 2], [0, 7]]), 3)
    assert off.tolist() == [0, 2, 2, 4]
    assert order.tolist() == [1, 4, 0, 3, -1, -1]
    assert slots.tolist() == [[2, 0], [-1, 3], [1, -1]]


def test_movement_by_hand():
    slots = np.array([[1, -1], [0, 2]])
    x = np.array([[1.0, 2.0], [3.0, 4.0]])
    assert T.permute(x, slots, np.full((3, 2), 9.0)).tolist() == [[3, 4], [1, 2], [3, 4]]
    y = np.array([[1.0, 0.0], [2.0, 1.0], [5.0, 5.0]])
    w = np.array([[0.5, 9.0], [2.0, 1.0]])
    out, _ = T.unpermute(y, slots, w)
    assert out.tolist() == [[1.0, 0.5], [7.0, 5.0]]
    assert T.unpermute(y, slots)[0].tolist() == [[2, 1], [6, 5]]
    dy, dw, _ = T.unpermute_backward(x, y, slots, w, np.zeros((3, 2)))
    assert dy.tolist() == [[6, 8], [0.5, 1], [3, 4]] and dw.tolist() == [[4, 0], [3, 35]]


@pytest.mark.parametrize("seed", [0, 1])
def test_gradients_agree_with_differences(seed):
    """out is linear in y and in the weights, so differences give the gradients up to fp64 rounding."""
    g = np.random.default_rng(seed)
    tokens, k, E, H = 5, 3, 4, 6
    ids = g.integers(-1, E, (tokens, k))
    off, order, slots = T.moe_sort(ids, E)
    P = tokens * k
    y, w, dout = g.normal(size=(P, H)), g.normal(size=(tokens, k)), g.normal(size=(tokens, H))
    dy, dw, _ = T.unpermute_backward(dout, y, slots, w, np.zeros((P, H)))
    def loss(y, w):
        return float((T.unpermute(y, slots, w)[0] * dout).sum())
    for i in range(P):
        d = np.zeros_like(y)
        d[i, 2] = 1.0
        assert abs(loss(y + d, w) - loss(y - d, w) - 2 * dy[i, 2]) < 1e-9
    for t in range(tokens):
        d = np.zeros_like(w)
        d[t, 1] = 1.0
        assert abs(loss(y, w + d) - loss(y, w - d) - 2 * dw[t, 1]) < 1e-9
    x, dxs = g.normal(size=(tokens, H)), g.normal(size=(P, H))
    kept = np.zeros(P, dtype=bool)
    kept[: off[-1]] = True
    dx = T.unpermute(dxs, slots)[0]
    base = np.zeros((P, H))
    for t in range(tokens):
        d = np.zeros_like(x)
        d[t, 3] = 1.0
        diff = ((T.permute(x + d, slots, base) - T.permute(x - d, slots, base)) * dxs).sum()
        assert abs(diff - 2 * dx[t, 3]) < 1e-9
