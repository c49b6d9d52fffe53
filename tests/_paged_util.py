"""Shared by the GPU tests of the paged operators: caches of every layout, tolerances from the arithmetic."""
from __future__ import annotations

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn
SHAPES = {"64": (64, 64), "128": (128, 128), "mla": (192, 128)}
POISON = {"fp8": 0x7F, "bf16": 0x7FC0}          # NaN in either type


def dtype_of(kind):
    return E4M3 if kind == "fp8" else torch.bfloat16


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def poisoned(shape, kind):
    """A tensor of NaN codes: whatever is read that should not be, or left unwritten, shows."""
    if kind == "fp8":
        return torch.full(shape, POISON[kind], dtype=torch.uint8, device="cuda").view(E4M3)
    return torch.full(shape, POISON[kind], dtype=torch.int16, device="cuda").view(torch.bfloat16)


def make_cache(pages, page, H_kv, shape, kind, layout="nhd"):
    """(k_cache, v_cache) views [pages, page, H_kv, D] of poisoned storage in one of three layouts."""
    d_qk, d_v = SHAPES[shape]
    if layout == "nhd":
        return poisoned((pages, page, H_kv, d_qk), kind), poisoned((pages, page, H_kv, d_v), kind)
    if layout == "hnd":
        return (poisoned((pages, H_kv, page, d_qk), kind).permute(0, 2, 1, 3),
                poisoned((pages, H_kv, page, d_v), kind).permute(0, 2, 1, 3))
    both = poisoned((pages, page, H_kv, d_qk + d_v), kind)      # K and V of a head side by side
    return both[..., :d_qk], both[..., d_qk:]


def bits(t):
    """The tensor's bit patterns: NaN compares equal to itself."""
    return t.view(torch.uint8) if t.dtype == E4M3 else t.view(torch.int16)


def random_values(shape, kind, rng, scale=1.0):
    """Random values as a CUDA tensor of the type; e4m3 codes are 64 times the values."""
    x = torch.from_numpy(rng.standard_normal(shape) * scale)
    if kind == "fp8":
        return (x * 64.0).clamp(-448, 448).float().to(E4M3).cuda()
    return x.to(torch.bfloat16).cuda()


def fill_tokens(cache, slots, rows):
    """cache[slot] = row for [n, H_kv, D] rows."""
    page = cache.shape[1]
    bits(cache)[slots // page, slots % page] = bits(rows)


def random_table(lens, page, rng, width=None, spare=3):
    """(table [B, width] with -7 where no token lies, number of pages): every page used once, in random order."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    width = max(need, default=0) if width is None else width
    table = np.full((len(lens), width), -7, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at: at + n]
        at += n
    return table, pages


def decode_tolerance(q, k, v, scale, dv, ref, w, kind):
    """Largest error the decode's arithmetic allows for one row, per channel (q, k in real units).

    Scores: an fp32 sum of D products, each partial sum at most S = sum |q_d k_d|, is off by D 2^-24 S; scaling
    and subtracting the maximum round the score, of magnitude X at most, three times (2^-24 X each) and the
    scale factor itself carries 3 roundings.  exp2 adds 2^-22.  Together each weight is off by e relative.
    Weights round to bf16 (2^-8) or fp16 (2^-11; below 2^-29 of the largest weight by 2^-40 absolute).  n
    weights and products are summed in fp32 (n 2^-24), and out rounds to bf16 (2^-8).
    """
    n, d = k.shape
    S = (np.abs(k) @ np.abs(q)).max() * scale
    e = d * 2.0 ** -24 * S + 6 * 2.0 ** -24 * S + 2.0 ** -22
    r = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    spread = w @ np.abs(v) * dv
    flush = n * 2.0 ** -40 * np.abs(v).max(axis=0) * dv if kind == "fp8" else 0.0
    return 2.0 ** -8 * np.abs(ref) * 1.01 + (2 * e + 2 * r + 2 * n * 2.0 ** -24) * spread * 1.01 + flush, e + n * 2.0 ** -24 + 2.0 ** -22
