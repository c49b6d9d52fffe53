"""Pins of the paged operators' oracle: closed forms worked out by hand."""
import math

import numpy as np

from oracle import paged as P


def test_plan_by_hand():
    # page size 4; request 0 holds 3 tokens and adds 2 (one in its page, one on a fresh page), request 1 is new
    table = [[7, 9, 9], [9, 9, 9]]
    t, lens, cu, pos, slots, cursor, met = P.paged_plan([3, 0], [2, 5], table, [2, 5, 0, 1], 1, 4, 9)
    assert t.tolist() == [[7, 5, 9], [0, 1, 9]] and lens.tolist() == [5, 5] and cu.tolist() == [0, 2, 7]
    assert pos.tolist() == [3, 4, 0, 1, 2, 3, 4, 0, 0]
    assert slots.tolist() == [31, 20, 0, 1, 2, 3, 4, -1, -1]
    assert cursor == 4 and not met


def test_plan_without_pages():
    t, lens, cu, pos, slots, cursor, met = P.paged_plan([0, 0], [3, 3], [[8, 8], [8, 8]], [5], 0, 2, 6)
    assert t.tolist() == [[5, -1], [-1, -1]] and slots.tolist() == [10, 11, -1, -1, -1, -1]
    assert cursor == 1 and met and cu.tolist() == [0, 3, 6] and lens.tolist() == [3, 3]


def test_rotation_by_hand():
    x = np.zeros((2, 1, 16))
    x[:, 0, 1], x[:, 0, 9] = 3.0, 4.0
    inv = np.zeros(8)
    inv[1] = math.pi / 2
    y = P.rope_rotate(x, [[1, 2]], inv, [8])
    np.testing.assert_allclose(y[0, 0, [1, 9]], [-4.0, 3.0], atol=1e-15)
    np.testing.assert_allclose(y[1, 0, [1, 9]], [-3.0, -4.0], atol=1e-15)
    z = np.zeros((1, 1, 24))
    z[0, 0, 10], z[0, 0, 11] = 1.0, 0.0
    y = P.rope_rotate(z, [[0], [5]], np.full(8, math.pi), [1, 7], offset=8, interleaved=True)   # pair 1 follows axis 1
    np.testing.assert_allclose(y[0, 0, [10, 11]], [-1.0, 0.0], atol=1e-14)


def test_decode_by_hand():
    k = np.array([[0.0, 1.0], [0.0, 1.0], [5.0, 0.0]])
    v = np.array([[1.0], [3.0], [100.0]])
    out, lse, w = P.decode_attention(np.array([-1000.0, 0.0]), k, v, 1.0)
    assert out[0] == 2.0 and abs(lse - math.log(2.0)) < 1e-15 and w.tolist() == [0.5, 0.5, 0.0]
    out, lse, _ = P.decode_attention(np.ones(2), k[:0], v[:0], 1.0)
    assert out[0] == 0.0 and lse == -np.inf
