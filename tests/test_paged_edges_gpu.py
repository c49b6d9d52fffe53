"""GPU tests of the paged serving operators where their numbers, checks or choices could go wrong beside the ordinary cases:
the bits that the weights keep, values that are not finite, steps over capacity, batches of every size."""
import math

import numpy as np
import pytest
import torch

from _paged_util import SHAPES, bits, decode_tolerance, dtype_of, f64, fill_tokens, make_cache, random_table, random_values
from fp8_causal_prefill_gb300 import paged_decode_attn, zyfa_check_errors
from oracle import paged as P

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class _Batch:
    """A decode batch over a paged cache: q, the caches, the table and each request's keys and values."""

    def __init__(self, kind, shape, lens, H, H_kv, page=16, width=None, seed=0):
        rng = np.random.default_rng(seed)
        d_qk, d_v = SHAPES[shape]
        table, pages = random_table(lens, page, rng, width)
        self.kind, self.lens, self.page, self.table = kind, list(lens), page, table
        self.kc, self.vc = make_cache(pages, page, H_kv, shape, kind)
        self.q = random_values((len(lens), H, d_qk), kind, rng)
        self.k = [random_values((n, H_kv, d_qk), kind, rng) for n in lens]
        self.v = [random_values((n, H_kv, d_v), kind, rng) for n in lens]
        for b in range(len(lens)):
            self.fill(b)
        self.scale = 1.0 / math.sqrt(d_qk)
        self.descale = torch.tensor([1 / 64.0], device="cuda") if kind == "fp8" else None

    def fill(self, b):
        """Writes request b's keys and values into its pages."""
        t = np.arange(self.lens[b])
        slots = torch.from_numpy(self.table[b, t // self.page].astype(np.int64) * self.page + t % self.page).cuda()
        fill_tokens(self.kc, slots, self.k[b])
        fill_tokens(self.vc, slots, self.v[b])

    def attend(self, **kw):
        d = self.descale
        out, lse = paged_decode_attn(self.q, self.kc, self.vc, torch.from_numpy(self.table).cuda(), i32(self.lens), q_descale=d, k_descale=d,
                                     v_descale=d, return_lse=True, **kw)
        assert zyfa_check_errors() == 0
        return f64(out), f64(lse)

    def rows(self):
        """(b, h, query, keys, values) of every row, in float64 and real units (values without their descale)."""
        f = 1 / 64.0 if self.kind == "fp8" else 1.0
        H, H_kv = self.q.shape[1], self.kc.shape[2]
        q = f64(self.q) * f
        for b in range(len(self.lens)):
            k, v = f64(self.k[b]) * f, f64(self.v[b])
            for h in range(H):
                yield b, h, q[b, h], k[:, h * H_kv // H], v[:, h * H_kv // H]


# ------------------------------------------------------------------------------------------------
# the bits that the weights keep

@pytest.mark.parametrize("shape", ["64", "128", "mla"])
@pytest.mark.parametrize("page", [7, 16])
def test_decode_bf16_weights_keep_16_bits(shape, page):
    """Weights multiply a bf16 V as a sum of two bf16 numbers, the second the rest of the first: a rounding is off by 2^-8 of what
    it rounds, so the two are off by 2^-16.  Rows whose values nearly cancel show a weight of 8 bits; the tolerance is that of the other tests
    with 2^-16 in place of 2^-8."""
    x = _Batch("bf16", shape, [2, 5, 64, 300, 5000], 8, 2, page=page, seed=page)
    out, lse = x.attend()
    worst = 0.0
    for b, h, q, k, v in x.rows():
        ref, ref_lse, w = P.decode_attention(q, k, v, x.scale)
        tol, lse_tol = decode_tolerance(q, k, v, x.scale, 1.0, ref, w, "bf16")
        tol = tol - 2 * (2.0 ** -8 - 2.0 ** -16) * (w @ np.abs(v)) * 1.01
        worst = max(worst, float((np.abs(out[b, h] - ref) / tol).max()))
        assert abs(lse[b, h] - ref_lse) <= lse_tol + 2.0 ** -22 * abs(ref_lse)
    assert worst <= 1.0, worst
