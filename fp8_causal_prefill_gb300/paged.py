"""Tensor-level calls of the paged serving operators (argument checks and marshalling only).

A serving step runs ``paged_plan`` (pages, slots and positions of its tokens from request lengths),
``rope_paged_store`` (rotates queries and keys, writes keys and values into their slots) and
``paged_decode_attn`` (one query token per request attends over its pages); prompts go through
``flash_attn_func`` on the dense copies that ``rope_paged_store`` can write in the same pass.

A paged cache is a pair of CUDA tensors [num_pages, page_size, H_kv, D]: ``torch.float8_e4m3fn`` (or
``torch.uint8`` holding e4m3 codes) or ``torch.bfloat16``.  Only D has to be contiguous, so permuted views
of [num_pages, H_kv, page_size, D] tensors and halves of a combined tensor work too.  Every call runs
on the current CUDA stream of its tensors' device, allocates through PyTorch's allocator only, and does
not synchronise; what a kernel meets (no page left, a bad page) is reported by ``zyfa_check_errors``.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from .api import ZYFA_DTYPE_BF16, ZYFA_DTYPE_E4M3, PagedCache, RopeOptions, ZyfaError, load_library

_CODES = {torch.float8_e4m3fn: ZYFA_DTYPE_E4M3, torch.uint8: ZYFA_DTYPE_E4M3, torch.bfloat16: ZYFA_DTYPE_BF16}


# address of a device's current stream (torch.cuda.current_stream builds a Stream object for it: 1 us of a 10 us call)
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


class PagedPlan(NamedTuple):
    """What a serving step needs beside its block table: see ``paged_plan``."""
    seq_lens: torch.Tensor    # [B] int32, lengths with the new tokens
    cu_tokens: torch.Tensor   # [B + 1] int32, first token row of each request
    positions: torch.Tensor   # [max_tokens] int32
    slots: torch.Tensor       # [max_tokens] int64, -1 for rows behind the last token
    cursor: torch.Tensor      # [1] int32, pages of the pool taken so far


def _call(dev: int, fn, *args) -> None:
    if dev == torch.cuda.current_device():
        st = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _stream(dev))
    if st != 0:
        raise ZyfaError(st, fn.__name__)


def _check(t, name: str, dtype, dev: int, shape: tuple) -> int:
    """Address of a contiguous tensor of this type, device and shape."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} CUDA tensor")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be on the same CUDA device as the other tensors")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _table(t, B: int, dev: int) -> tuple:
    """Address, row stride and width of a block table whose rows may be part of a wider tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != 2:
        raise TypeError("block_table must be an int32 CUDA tensor [B, max_pages]")
    rows, width = t.shape
    if rows != B or t.get_device() != dev:
        raise ValueError(f"block_table must have {B} rows, on the same device as the other tensors")
    s0, s1 = t.stride()
    if width > 1 and s1 != 1:
        raise ValueError("block_table rows must be contiguous")
    if rows > 1 and s0 < width:
        raise ValueError("block_table rows must not overlap")
    return t.data_ptr(), (s0 if rows > 1 else width), width


def _descale(t, name: str, per_head: int, dev: int) -> tuple:
    if t is None:
        return None, None
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 CUDA tensor or None")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the same CUDA device as the other tensors")
    n = t.numel()
    if n == 1:
        return t.data_ptr(), 0
    if n != per_head:
        raise ValueError(f"{name} must hold 1 or {per_head} values, got {n}")
    return t.data_ptr(), 1


def _descales(q, k, v, per_head: int, dev: int) -> tuple:
    """Three addresses and their common form: 0 per tensor, 1 per head."""
    if q is None and k is None and v is None:
        return None, None, None, 0
    (a, fa), (b, fb), (c, fc) = (_descale(t, n, per_head, dev) for t, n in ((q, "q_descale"), (k, "k_descale"),
                                                                             (v, "v_descale")))
    forms = {f for f in (fa, fb, fc) if f is not None}
    if len(forms) > 1:
        raise ValueError("descales must all be per tensor or all per head")
    return a, b, c, forms.pop()


def _cache(k, v) -> tuple:
    """(zyfa_paged_cache_t, device, H_kv, D_qk, D_v) of a cache's two tensors."""
    code = _CODES.get(k.dtype) if isinstance(k, torch.Tensor) else None
    if code is None or not isinstance(v, torch.Tensor) or v.dtype != k.dtype or k.dim() != 4 or v.dim() != 4:
        raise TypeError("k_cache and v_cache must be e4m3 or bfloat16 CUDA tensors [num_pages, page_size, H_kv, D] of one type")
    pages, page, H_kv, D_qk = k.shape
    D_v = v.shape[3]
    dev = k.get_device()
    if v.shape[:3] != k.shape[:3] or v.get_device() != dev or dev < 0:
        raise ValueError("k_cache and v_cache must agree in pages, page size, heads and CUDA device")
    ks, vs = k.stride(), v.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("the last dimension of k_cache and v_cache must be contiguous")
    if pages < 2 or page < 2 or H_kv < 2:  # a dimension of one element may carry any stride
        ks = [s if n > 1 else D_qk for s, n in zip(ks, k.shape)]
        vs = [s if n > 1 else D_v for s, n in zip(vs, v.shape)]
    c = PagedCache(k.data_ptr(), v.data_ptr(), code, page, pages, H_kv, D_qk, D_v, ks[0], ks[1], ks[2], vs[0], vs[1], vs[2])
    return c, dev, H_kv, D_qk, D_v


def paged_plan(cached_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
               cursor: torch.Tensor, page_size: int, max_tokens: int, out: PagedPlan | None = None) -> PagedPlan:
    """Pages, slots and positions of a step in which request b, holding ``cached_lens[b]`` tokens, adds
    ``new_lens[b]`` (int32 CUDA tensors [B]).

    Pages that the new tokens start are taken from ``free_pages`` (int32) at ``cursor`` (int32, one value)
    and written into ``block_table`` (int32 [B, max_pages]; other entries stay as they are).  Token rows are
    numbered request after request; rows from the last token up to ``max_tokens`` get position 0 and slot -1.
    ``out`` gives the result's tensors (for captured graphs); ``out.cursor`` may be ``cursor`` itself.
    """
    if not isinstance(cached_lens, torch.Tensor):
        raise TypeError("cached_lens must be a contiguous torch.int32 CUDA tensor")
    dev, B, i32 = cached_lens.get_device(), cached_lens.shape[0] if cached_lens.dim() == 1 else -1, torch.int32
    page_size, max_tokens = int(page_size), int(max_tokens)
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    c = _check(cached_lens, "cached_lens", i32, dev, (B,))
    n = _check(new_lens, "new_lens", i32, dev, (B,))
    table, stride, width = _table(block_table, B, dev)
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise TypeError("free_pages must be a contiguous torch.int32 CUDA tensor [num_free]")
    free = _check(free_pages, "free_pages", i32, dev, free_pages.shape)
    at = _check(cursor, "cursor", i32, dev, (1,))
    if out is None:
        d = cached_lens.device
        out = PagedPlan(torch.empty(B, dtype=i32, device=d), torch.empty(B + 1, dtype=i32, device=d),
                        torch.empty(max_tokens, dtype=i32, device=d), torch.empty(max_tokens, dtype=torch.int64, device=d),
                        torch.empty(1, dtype=i32, device=d))
        o = [t.data_ptr() for t in out]
    else:
        o = [_check(t, "out." + name, torch.int64 if name == "slots" else i32, dev, (size,))
             for t, name, size in zip(out, PagedPlan._fields, (B, B + 1, max_tokens, max_tokens, 1))]
    _call(dev, load_library().zyfa_paged_plan, c, n, B, page_size, table, stride, width, free, free_pages.shape[0], at,
          o[4], o[0], o[1], o[2], o[3], max_tokens)
    return out


class Rope:
    """Rotary positions for ``rope_paged_store``.

    ``inv_freq``: float32 CUDA tensor [rot_dim / 2], radians per unit of position for each channel pair;
    ``axis_pairs``: how many consecutive pairs follow each position axis (default: all follow one axis);
    ``offset``: first rotated channel; ``interleaved``: pairs (2i, 2i + 1) instead of (i, i + rot_dim / 2).
    """

    def __init__(self, inv_freq: torch.Tensor, axis_pairs=None, offset: int = 0, interleaved: bool = False):
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
            raise TypeError("inv_freq must be a contiguous float32 CUDA tensor [rot_dim / 2]")
        pairs = inv_freq.shape[0]
        address = _check(inv_freq, "inv_freq", torch.float32, inv_freq.get_device(), (pairs,))
        axis_pairs = (pairs,) if axis_pairs is None else tuple(int(n) for n in axis_pairs)
        if not 1 <= len(axis_pairs) <= 4 or sum(axis_pairs) != pairs or min(axis_pairs) < 0:
            raise ValueError(f"axis_pairs must be 1 to 4 counts that sum to {pairs}")
        self.inv_freq, self.num_axes = inv_freq, len(axis_pairs)
        self._options = RopeOptions(address, 2 * pairs, int(offset), 1 if interleaved else 0, len(axis_pairs),
                                    (ctypes.c_int * 4)(*axis_pairs))


def _rows(t, name: str, N: int, heads: int, D: int, dev: int) -> tuple:
    """Address and token stride of a bf16 [N, heads, D] tensor with dense heads."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be a bfloat16 CUDA tensor [N, heads, D]")
    if t.shape != (N, heads, D) or t.get_device() != dev:
        raise ValueError(f"{name} must have shape {(N, heads, D)} on the cache's device, got {tuple(t.shape)}")
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != D):
        raise ValueError(f"the heads of one token of {name} must be contiguous")
    return t.data_ptr(), (s[0] if N > 1 else heads * D)


def _dense(t, name: str, code: int, shape: tuple, dev: int) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or _CODES.get(t.dtype) != code or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA tensor of the cache's type")
    if t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name} must have shape {shape} on the cache's device, got {tuple(t.shape)}")
    return t.data_ptr()


def rope_paged_store(q: torch.Tensor | None, k: torch.Tensor | None, v: torch.Tensor | None, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, slots: torch.Tensor, positions: torch.Tensor | None = None,
                     rope: Rope | None = None, *, q_descale=None, k_descale=None, v_descale=None,
                     q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                     v_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Rotate a step's bf16 queries [N, H, D_qk] and keys [N, H_kv, D_qk] by their positions, write keys and values
    [N, H_kv, D_v] into cache slots ``slots`` (int64 [N]; below 0: a padding row, for which nothing is written),
    and return the queries in the cache's type.

    ``q``, ``k`` and ``v`` may be slices of one projection (dense heads, any token stride that is a multiple
    of 8).  ``positions`` is int32 [N], or [axes, N] for a ``rope`` with several axes; without ``rope`` nothing is
    rotated.  For an e4m3 cache the descales (float32, one value or H_kv values) divide what is stored.
    ``k_out`` and ``v_out`` [N, H_kv, D] receive dense copies, as ``flash_attn_func`` reads them.  ``q`` may be None (keys and
    values only), or ``k`` and ``v`` (queries only).
    """
    c, dev, H_kv, D_qk, D_v = _cache(k_cache, v_cache)
    code = c.dtype
    some = q if q is not None else k
    if some is None or (k is None) != (v is None) or not isinstance(some, torch.Tensor) or some.dim() != 3:
        raise TypeError("q, or k and v, must be given as [N, heads, D]")
    N, H = some.shape[0], some.shape[1] if q is not None else H_kv
    qp = kp = vp = qo = None
    qs = ks = vs = 0
    if q is not None:
        qp, qs = _rows(q, "q", N, H, D_qk, dev)
        if q_out is None:
            q_out = torch.empty((N, H, D_qk), dtype=k_cache.dtype, device=q.device)
            qo = q_out.data_ptr()
        else:
            qo = _dense(q_out, "q_out", code, (N, H, D_qk), dev)
            if qo == qp and N:
                raise ValueError("q_out must not be q")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k is not None:
        kp, ks = _rows(k, "k", N, H_kv, D_qk, dev)
        vp, vs = _rows(v, "v", N, H_kv, D_v, dev)
    elif k_out is not None or v_out is not None:
        raise ValueError("k_out or v_out without k and v")
    ko = _dense(k_out, "k_out", code, (N, H_kv, D_qk), dev)
    vo = _dense(v_out, "v_out", code, (N, H_kv, D_v), dev)
    if N and ((ko is not None and ko == kp) or (vo is not None and vo == vp)):
        raise ValueError("k_out and v_out must not be k and v")
    sp = _check(slots, "slots", torch.int64, dev, (N,))
    pp, stride, opts = None, 0, None
    if rope is not None:
        if rope.inv_freq.get_device() != dev:
            raise ValueError("rope.inv_freq must be on the cache's device")
        if not isinstance(positions, torch.Tensor) or positions.dtype != torch.int32:
            raise TypeError("positions must be an int32 CUDA tensor [N] or [axes, N]")
        if positions.dim() == 1 and rope.num_axes == 1:
            shape_ok, stride = positions.shape[0] == N, N
        else:
            shape_ok, stride = positions.shape == (rope.num_axes, N), positions.stride(0) if rope.num_axes > 1 else N
        if not shape_ok or positions.get_device() != dev or (N > 1 and positions.stride(-1) != 1):
            raise ValueError(f"positions must be [{rope.num_axes}, {N}] with contiguous rows, on the cache's device")
        pp, opts = positions.data_ptr(), ctypes.byref(rope._options)
    if code == ZYFA_DTYPE_E4M3:
        dq, dk, dv, per_head = _descales(q_descale, k_descale, v_descale, H_kv, dev)
    else:
        dq = dk = dv = None
        per_head = 0
    _call(dev, load_library().zyfa_rope_paged_store, qp, kp, vp, qs, ks, vs, qo, ko, vo, pp, stride, sp, N, H,
          ctypes.byref(c), opts, dq, dk, dv, per_head)
    return q_out


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
    log-sum-exp [B, H] (-inf without tokens).  e4m3 descales hold one value or B * H_kv values ([request][KV head]).
    ``workspace`` (uint8 CUDA, ``paged_decode_workspace_bytes``) is allocated per call if not given; calls that
    may overlap on the GPU need one each.
    """
    c, dev, H_kv, D_qk, D_v = _cache(k_cache, v_cache)
    if not isinstance(q, torch.Tensor) or _CODES.get(q.dtype) != c.dtype or q.dim() != 3:
        raise TypeError("q must be a CUDA tensor [B, H, D_qk] of the cache's type")
    B, H, D = q.shape
    s = q.stride()
    if D != D_qk or q.get_device() != dev:
        raise ValueError(f"q must have {D_qk} channels, on the cache's device")
    if H < 1 or H % H_kv:
        raise ValueError(f"the number of query heads must be a multiple of {H_kv}")
    if s[2] != 1 or (H > 1 and s[1] != D):
        raise ValueError("the heads of one request of q must be contiguous")
    table, stride, width = _table(block_table, B, dev)
    lens = _check(seq_lens, "seq_lens", torch.int32, dev, (B,))
    if out is None:
        out = torch.empty((B, H, D_v), dtype=torch.bfloat16, device=q.device)
        op = out.data_ptr()
    else:
        op = _check(out, "out", torch.bfloat16, dev, (B, H, D_v))
    lse = torch.empty((B, H), dtype=torch.float32, device=q.device) if return_lse else None
    if c.dtype == ZYFA_DTYPE_E4M3:
        dq, dk, dv, per_head = _descales(q_descale, k_descale, v_descale, B * H_kv, dev)
    else:
        dq = dk = dv = None
        per_head = 0
    lib = load_library()
    if workspace is None:
        workspace = torch.empty(lib.zyfa_attn_decode_paged_workspace_bytes(B, H, H_kv, D_v, width * c.page_size), dtype=torch.uint8,
                                device=q.device)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != dev:
        raise TypeError("workspace must be a contiguous uint8 tensor on the cache's device")
    _call(dev, lib.zyfa_attn_decode_paged, q.data_ptr(), s[0] if B > 1 else H * D, ctypes.byref(c), table, stride, width,
          lens, op, None if lse is None else lse.data_ptr(), B, H, 0.0 if softmax_scale is None else float(softmax_scale),
          dq, dk, dv, per_head, workspace.data_ptr(), workspace.numel())
    return (out, lse) if return_lse else out
