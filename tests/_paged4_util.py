"""Shared by the GPU tests of the 4-bit paged cache."""
from __future__ import annotations

import numpy as np
import torch

from _paged_util import E4M3, SHAPES
from oracle import paged4 as Q

NAN_SCALE = 0x7F


def _poison(shape, value):
    return torch.full(shape, value, dtype=torch.uint8, device="cuda")


def make_cache4(pages, page, H_kv, shape, layout="nhd", typed=False):
    """(k_cache, v_cache, k_scales, v_scales) of codes 6 with NaN scales: whatever is read that should not be, or left unwritten,
    shows.  Layouts: tokens before heads, heads before tokens, all four within a token's row, K and V halves of one tensor."""
    d_qk, d_v = SHAPES[shape]
    sizes = (d_qk // 2, d_v // 2, d_qk // 16, d_v // 16)
    if layout == "row":                                       # [codes of all heads | their scales] of a token
        total = -(-H_kv * sum(sizes) // 16) * 16
        both = _poison((pages, page, total), NAN_SCALE)
        cut = np.cumsum([0] + [H_kv * s for s in sizes])
        out = [both[..., a:b].unflatten(-1, (H_kv, s)) for a, b, s in zip(cut, cut[1:], sizes)]
    elif layout == "hnd":
        out = [_poison((pages, H_kv, page, s), NAN_SCALE).permute(0, 2, 1, 3) for s in sizes]
    elif layout == "joint":                                   # K and V of a head side by side
        codes = _poison((pages, page, H_kv, sizes[0] + sizes[1]), NAN_SCALE)
        scales = _poison((pages, page, H_kv, sizes[2] + sizes[3]), NAN_SCALE)
        out = [codes[..., :sizes[0]], codes[..., sizes[0]:], scales[..., :sizes[2]], scales[..., sizes[2]:]]
    else:
        out = [_poison((pages, page, H_kv, s), NAN_SCALE) for s in sizes]
    if typed:
        out = [t.view(torch.float4_e2m1fn_x2) if i < 2 else t.view(E4M3) for i, t in enumerate(out)]
    return out


def raw(t):
    return t.view(torch.uint8)


def random_codes(shape, rng, about=128.0):
    """(bytes [..., D / 2], scale bytes [..., D / 16]) of values [..., D] about N(0, about): quantised normal values."""
    x = rng.standard_normal(shape) * about
    return Q.quantise(x, 1.0)


def fill4(cache, scales, slots, codes, scale_codes):
    page = cache.shape[1]
    slots = torch.as_tensor(slots, device="cuda")
    raw(cache)[slots // page, slots % page] = torch.from_numpy(codes).cuda()
    raw(scales)[slots // page, slots % page] = torch.from_numpy(scale_codes).cuda()


def held_of(cache, scales):
    return Q.held(raw(cache).cpu().numpy(), raw(scales).cpu().numpy())
