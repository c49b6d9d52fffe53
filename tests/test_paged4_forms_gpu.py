"""GPU tests of forms that a 4-bit cache's sizes decide."""
import numpy as np
import pytest
import torch

import test_paged4_gpu as base
from _paged4_util import fill4, make_cache4, random_codes, raw
from _paged_util import SHAPES, bits, random_values
from fp8_causal_prefill_gb300 import paged_decode_attn, paged_read, zyfa_check_errors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("page", [32, 1000, 4096])
@pytest.mark.parametrize("shape,H,H_kv", [("64", 4, 4), ("64", 12, 1), ("128", 16, 8), ("mla", 2, 2)])
def test_a_cache_of_one_page(shape, H, H_kv, page, layout):
    """The same tokens in a cache of one page, and in the first of two pages."""
    rng = np.random.default_rng(page)
    two = make_cache4(2, page, H_kv, shape, layout)
    for i, d in enumerate(SHAPES[shape]):
        fill4(two[i], two[2 + i], np.arange(page), *random_codes((page, H_kv, d), rng, 2.0))
    one = make_cache4(1, page, H_kv, shape, layout)
    for x, y in zip(one, two):
        raw(x).copy_(raw(y)[:1])
    lens = torch.tensor([page, 1, 0, page // 2 + 3], dtype=torch.int32, device="cuda")
    table = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    q = random_values((4, H, SHAPES[shape][0]), "bf16", rng)
    got = [paged_decode_attn(q, *c[:2], table, lens, return_lse=True, k_scales=c[2], v_scales=c[3]) for c in (one, two, [x[:1] for x in two])]
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    assert not torch.isnan(got[0][0]).any() and (got[0][0][2] == 0).all()
    cu = torch.tensor([0, page], dtype=torch.int32, device="cuda")
    for x, y in zip(*(paged_read(*c[:2], table[:1], cu, page, k_scales=c[2], v_scales=c[3]) for c in (one, two))):
        assert torch.equal(bits(x), bits(y))
    assert zyfa_check_errors() == 0


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", ["64", "128", "mla"])
def test_stores_of_any_number_of_waves(shape, interleaved):
    """Rotations that split a block of 16 channels, whose kernels hold fewer blocks an SM, and one that does not."""
    for N in (303, 305, 1217, 9729):
        base._store_case(shape, N, 2, 1, interleaved=interleaved, rot=16, offset=8, seed=N)
        base._store_case(shape, N, 1, 1, interleaved=interleaved, rot=32, offset=16, seed=N)
