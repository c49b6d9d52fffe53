"""The oracle of the 4-bit cache against the definition of its formats (no GPU)."""
import numpy as np
import pytest

from oracle import paged4 as Q
from oracle.formats import e4m3_decode


def test_e2m1_values():
    assert Q.e2m1_decode(range(8)).tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert Q.e2m1_decode(range(8, 16)).tolist() == [0, -0.5, -1, -1.5, -2, -3, -4, -6]


def test_e2m1_rounds_to_nearest_even():
    assert (Q.e2m1_encode_rne_satfinite(Q.e2m1_decode(range(1, 16))) == [*range(1, 8), 0, *range(9, 16)]).sum() == 14  # -0 keeps its sign
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for x, code in ties.items():
        assert Q.e2m1_encode_rne_satfinite([x, -x]).tolist() == [code, code | 8]
        assert Q.e2m1_encode_rne_satfinite([np.nextafter(x, 9)]).tolist() == [code + (code % 2 == 0 and x in (0.25, 1.25, 2.5, 5.0))]
    assert Q.e2m1_encode_rne_satfinite([7.0, 1e30, np.inf, -np.inf]).tolist() == [7, 7, 7, 15]


def test_pack_and_unpack():
    codes = np.arange(32).reshape(2, 16) % 16
    assert Q.pack(codes).tolist()[0] == [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]
    assert (Q.unpack(Q.pack(codes)) == codes).all()


def test_blocks_keep_their_largest_value():
    rng = np.random.default_rng(0)
    y = rng.standard_normal((200, 64)).astype(np.float32) * np.exp2(rng.integers(-3, 8, (200, 1)))
    codes, scales = Q.quantise(y, 1.0)
    z, s = y.reshape(200, 4, 16).astype(np.float64), e4m3_decode(scales)
    top = np.abs(z).max(-1)
    assert np.all(np.abs(s - top / 6) <= np.maximum(2.0 ** -4 * top / 6, 2.0 ** -10) * 1.000001)
    held = Q.held(codes, scales).reshape(z.shape)
    x = np.abs(z) / s[..., None]
    half = np.where(x < 2, 0.25, np.where(x < 4, 0.5, 1.0))
    assert np.all(np.abs(held - z) <= half * s[..., None] * 1.000001)


@pytest.mark.parametrize("block,codes,scale", [
    ([0.0] * 16, [0] * 8, 0x00), ([6.0] + [0.0] * 15, [0x07] + [0] * 7, 0x38), ([np.inf] + [448.0] * 15, [0x27] + [0x22] * 7, 0x7E),
    ([1e-6] * 16, [0] * 8, 0x00)])
def test_edges_of_a_block(block, codes, scale):
    c, s = Q.quantise(np.array(block, dtype=np.float32), 1.0)
    assert s.tolist() == [scale] and c.tolist() == codes


def test_nan_makes_the_scale_nan():
    block = np.ones(32, dtype=np.float32)
    block[5] = np.nan
    c, s = Q.quantise(block, 1.0)
    assert s[0] == 0x7F and s[1] != 0x7F
    held = Q.held(c, s)
    assert np.isnan(held[:16]).all() and np.isfinite(held[16:]).all()
