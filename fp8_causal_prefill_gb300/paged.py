"""Tensor-level calls of the paged serving operators.

A serving step runs ``paged_plan`` (pages, slots and positions of its tokens from request lengths),
``rope_paged_store`` (rotates queries and keys, writes keys and values into their slots) and
``paged_decode_attn`` (one query token per request attends over its pages); prompts go through
``flash_attn_func`` on the dense copies that ``rope_paged_store`` can write in the same pass.

A paged cache is a pair of CUDA tensors [num_pages, page_size, H_kv, D]: ``torch.float8_e4m3fn`` (or
``torch.uint8`` holding e4m3 codes) or ``torch.bfloat16``.  Only D has to be contiguous, so permuted views
of [num_pages, H_kv, page_size, D] tensors and halves of a combined tensor work too.  Every call runs
on the current CUDA stream of its tensors' device, allocates through PyTorch's allocator only, and does
not synchronise; what a kernel meets (no page left, a bad page) is reported by ``zyfa_check_errors``.

The argument checks and the calls into libzyfa.so are native (``csrc/paged_binding.cpp``): these calls
are made for every token, and small ones take the GPU a few microseconds.  Wrong types and layouts raise
TypeError, wrong sizes and devices ValueError, a status of the library ZyfaError.
"""
from __future__ import annotations

import os
from typing import NamedTuple

import torch

from .api import ZyfaError, load_library

_native = None


class PagedPlan(NamedTuple):
    """What a serving step needs beside its block table: see ``paged_plan``."""
    seq_lens: torch.Tensor    # [B] int32, lengths with the new tokens
    cu_tokens: torch.Tensor   # [B + 1] int32, first token row of each request
    positions: torch.Tensor   # [max_tokens] int32
    slots: torch.Tensor       # [max_tokens] int64, -1 for rows behind the last token
    cursor: torch.Tensor      # [1] int32, pages of the pool taken so far


def _load():
    """The native binding; raises if it has not been built, or for another torch (there is no fallback path)."""
    global _native
    from . import build
    load_library()
    made_for = build.binding_built_for()
    if made_for not in (None, build._binding_target()):
        raise ZyfaError(4, f"the tensor binding was built for {made_for}; build it anew with `python -m fp8_causal_prefill_gb300.build`")
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_paged.so")
    if not os.path.exists(path):
        raise ZyfaError(4, f"{path} is missing; build it with `python -m fp8_causal_prefill_gb300.build`")
    from . import _paged
    _native = _paged
    return _paged


def paged_plan(cached_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
               cursor: torch.Tensor, page_size: int, max_tokens: int, out: PagedPlan | None = None) -> PagedPlan:
    """Pages, slots and positions of a step in which request b, holding ``cached_lens[b]`` tokens, adds
    ``new_lens[b]`` (int32 CUDA tensors [B]).

    Pages that the new tokens start are taken from ``free_pages`` (int32) at ``cursor`` (int32, one value)
    and written into ``block_table`` (int32 [B, max_pages]; other entries stay as they are).  Token rows are
    numbered request after request; rows from the last token up to ``max_tokens`` get position 0 and slot -1.
    ``out`` gives the result's tensors (for captured graphs), none in the place of another or of an input, but
    ``out.cursor`` may be ``cursor`` itself.  Without it they are made in one allocation.
    """
    return (_native or _load()).plan(cached_lens, new_lens, block_table, free_pages, cursor, page_size, max_tokens, out, PagedPlan)


class Rope:
    """Rotary positions for ``rope_paged_store``.

    ``inv_freq``: float32 CUDA tensor [rot_dim / 2], radians per unit of position for each channel pair;
    ``axis_pairs``: how many consecutive pairs follow each position axis (default: all follow one axis);
    ``offset``: first rotated channel; ``interleaved``: pairs (2i, 2i + 1) instead of (i, i + rot_dim / 2).
    """

    __slots__ = ("_spec",)

    def __init__(self, inv_freq: torch.Tensor, axis_pairs=None, offset: int = 0, interleaved: bool = False):
        self._spec = (_native or _load()).rope(inv_freq, axis_pairs, offset, interleaved)

    inv_freq = property(lambda self: self._spec[0])
    axis_pairs = property(lambda self: self._spec[1])


def rope_paged_store(q: torch.Tensor | None, k: torch.Tensor | None, v: torch.Tensor | None, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, slots: torch.Tensor, positions: torch.Tensor | None = None,
                     rope: Rope | None = None, *, q_descale=None, k_descale=None, v_descale=None,
                     q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                     v_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Rotate a step's bf16 queries [N, H, D_qk] and keys [N, H_kv, D_qk] by their positions, write keys and values
    [N, H_kv, D_v] into cache slots ``slots`` (int64 [N], distinct; below 0: a padding row, for which nothing is written),
    and return the queries in the cache's type.

    ``q``, ``k`` and ``v`` may be slices of one projection (dense heads, any token stride that is a multiple
    of 8).  ``positions`` is int32 [N], or [axes, N] for a ``rope`` with several axes; without ``rope`` nothing is
    rotated.  For an e4m3 cache the descales (float32, one value or H_kv values) divide what is stored.
    For a bf16 cache they are not used, as in the prefill.  ``k_out`` and ``v_out`` [N, H_kv, D] receive dense copies, as
    ``flash_attn_func`` reads them.  ``q`` may be None (keys and values only), or ``k`` and ``v`` (queries only).  What is
    written must not overlap what is read, nor rows of the cache one another.
    """
    return (_native or _load()).store(q, k, v, k_cache, v_cache, slots, positions, None if rope is None else rope._spec,
                                      q_descale, k_descale, v_descale, q_out, k_out, v_out)


def paged_decode_workspace_bytes(B: int, H: int, H_kv: int, D_v: int, max_len: int) -> int:
    """Bytes of the ``workspace`` that ``paged_decode_attn`` needs for these sizes, with ``max_len`` the tokens a row
    of the block table can name (its columns times the page size)."""
    return load_library().zyfa_attn_decode_paged_workspace_bytes(B, H, H_kv, D_v, max_len)


def paged_decode_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                      seq_lens: torch.Tensor, softmax_scale: float | None = None, *, q_descale=None, k_descale=None,
                      v_descale=None, out: torch.Tensor | None = None, return_lse: bool = False,
                      workspace: torch.Tensor | None = None):
    """Attention of one query token per request, ``q`` [B, H, D_qk] in the cache's type, over the first
    ``seq_lens[b]`` tokens (int32 [B]) of the pages that ``block_table`` (int32 [B, max_pages]) names.

    Returns bfloat16 [B, H, D_v] (0 for a request without tokens), and with ``return_lse`` also the float32
    log-sum-exp [B, H] (-inf without tokens).  e4m3 descales hold one value, H_kv values, as ``rope_paged_store`` takes
    them, or B * H_kv values ([request][KV head]); for a bf16 cache they are not used.
    ``workspace`` (uint8 CUDA, ``paged_decode_workspace_bytes``) is allocated per call if not given; calls that
    may overlap on the GPU need one each.  A NaN among a row's scores makes the row NaN.
    """
    return (_native or _load()).decode(q, k_cache, v_cache, block_table, seq_lens, softmax_scale, q_descale, k_descale,
                                       v_descale, out, return_lse, workspace)
