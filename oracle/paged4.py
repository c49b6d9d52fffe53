"""Oracle of the 4-bit paged cache: the e2m1 format, blocks of 16 channels with an e4m3 scale.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Written from the format's definition: OCP FP4 e2m1 has one sign bit, two
exponent bits with bias 1 and one mantissa bit, so its magnitudes are 0, 0.5, 1, 1.5, 2, 3, 4 and 6 in the order of their codes,
and there is neither an infinity nor a NaN.
"""
from __future__ import annotations

import numpy as np

from .formats import e4m3_decode, e4m3_encode_rne_satfinite

GROUP = 16


def _e2m1_fields(codes) -> np.ndarray:
    c = np.asarray(codes, dtype=np.int64)
    e, m = (c >> 1) & 3, (c & 1).astype(np.float64)
    mag = np.where(e == 0, m * 0.5, (1.0 + m / 2.0) * np.exp2(e - 1.0))
    return np.where(c & 8, -mag, mag)


_E2M1 = _e2m1_fields(np.arange(16))


def e2m1_decode(codes) -> np.ndarray:
    """Codes 0 .. 15 as float64 values."""
    return _E2M1[np.asarray(codes, dtype=np.int64) & 15]


def e2m1_encode_rne_satfinite(x) -> np.ndarray:
    """The nearest code of each value, ties to the even code, beyond 6 the code of 6; by comparison of distances."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 6.0)[..., None]
    d = np.abs(a - _E2M1[:8])
    near = d == d.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    return (pick | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def unpack(codes) -> np.ndarray:
    """Bytes [..., D / 2] as codes [..., D]: channel 2i in the low half of byte i."""
    codes = np.asarray(codes, dtype=np.uint8)
    return np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def pack(codes) -> np.ndarray:
    codes = np.asarray(codes, dtype=np.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def held(codes, scales) -> np.ndarray:
    """Values over their descale that bytes of codes [..., D / 2] and e4m3 scales [..., D / 16] stand for."""
    return e2m1_decode(unpack(codes)) * np.repeat(e4m3_decode(scales), GROUP, axis=-1)


def quantise(y, inv_descale) -> tuple[np.ndarray, np.ndarray]:
    """(bytes [..., D / 2], scales [..., D / 16]) of fp32 values, each operation in fp32 as the definition says."""
    f = np.float32
    with np.errstate(all="ignore"):
        z = (np.asarray(y, dtype=f) * f(inv_descale)).reshape(*np.shape(y)[:-1], np.shape(y)[-1] // GROUP, GROUP)
        top = np.abs(z).max(axis=-1)                        # NaN if one is
        scales = e4m3_encode_rne_satfinite(top * (f(1.0) / f(6.0)))
        s = e4m3_decode(scales).astype(f)
        r = np.where(s > 0, f(1.0) / s, f(0.0)).astype(f)
        codes = e2m1_encode_rne_satfinite(np.nan_to_num((z * r[..., None]).astype(f), nan=0.0, posinf=6.0, neginf=-6.0))
    return pack(codes.reshape(np.shape(y))), scales
