"""Refusals and choices of the paged serving operators that need no GPU: memory that two would write, loads that
the dependent launch does not order."""
import ctypes
import itertools
import os
import random

import pytest
import torch

from fp8_causal_prefill_gb300 import build
from test_paged_host import A, _cache, _decode, _plan, _store, lib  # noqa: F401


def _rows(strides, extents):
    return [sum(i * s for i, s in zip(at, strides)) for at in itertools.product(*(range(n) for n in extents))]


def _overlap(strides, extents, D):
    rows = sorted(_rows(strides, extents))
    return any(b - a < D for a, b in zip(rows, rows[1:]))


# 4 pages of 16 tokens of 2 heads of 128 channels: (page, token, head) strides
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("strides,apart", [
    ((4096, 256, 128), True), ((4096, 128, 2048), True), ((8192, 512, 256), True), ((256, 1024, 128), True), ((128, 1024, 512), True),
    ((4160, 256, 128), True), ((256, 4096, 128), True), ((2048, 128, 8192), True), ((1 << 46, 256, 128), True),
    ((4096, 128, 128), False), ((128, 256, 128), False), ((256, 2048, 1024), True), ((256, 512, 128), False), ((4096, 128, 256), False), ((4080, 256, 128), False),
    ((4096, 256, 144), False), ((512, 128, 1024), False), ((4096, 1 << 46, 1 << 46), False)])
def test_store_refuses_strides_that_overlap_together(lib, strides, apart, which):  # noqa: F811
    assert _overlap(strides, (4, 16, 2), 128) == (not apart)
    kw = {f"{which}_{n}_stride": s for n, s in zip(("page", "token", "head"), strides)}
    assert _store(lib, _cache(**kw), N=0) == (0 if apart else 1)


def test_store_accepts_views_of_dense_tensors_and_nothing_that_overlaps(lib):  # noqa: F811
    rng = random.Random(1)
    accepted = 0
    for _ in range(4000):
        extents = [rng.choice([1, 2, 3, 5]) for _ in range(3)]                  # pages, tokens, heads
        D, D_v = rng.choice([(64, 64), (128, 128), (192, 128)])
        order, strides, span = rng.sample(range(3), 3), [0, 0, 0], D
        for i in order:                                                         # a view of a dense tensor, innermost dimension first
            strides[i] = span + 64 * rng.choice([0, 0, 0, 1, 7])
            span = strides[i] * extents[i]
        dense = rng.random() < 0.5
        if not dense:
            strides[rng.randrange(3)] = 64 * rng.randrange(20)
        kw = {f"{w}_{n}_stride": s for w in "kv" for n, s in zip(("page", "token", "head"), strides)}
        st = _store(lib, _cache(num_pages=extents[0], page_size=extents[1], H_kv=extents[2], D_qk=D, D_v=D_v, **kw), N=0, H=extents[2])
        assert st in (0, 1) and not (dense and st) and not (st == 0 and _overlap(strides, extents, D))
        accepted += st == 0
    assert 2000 < accepted < 3900


def _in_one_place(lib, extents, strides, D, D_v, offset):  # noqa: F811
    """The store's answer for V `offset` elements behind K, in the same strides, and whether rows of the two overlap."""
    kw = {f"{w}_{n}_stride": s for w in "kv" for n, s in zip(("page", "token", "head"), strides)}
    base = 1 << 30
    c = _cache(k=base, v=base + offset, num_pages=extents[0], page_size=extents[1], H_kv=extents[2], D_qk=D, D_v=D_v, **kw)
    rows = _rows(strides, extents)
    return c, any(x - D_v < y < x + D for x in rows for y in (z + offset for z in rows))


def test_store_refuses_keys_and_values_in_one_place(lib):  # noqa: F811
    # (calls that are accepted are made only where there is no GPU to take their addresses, which are not memory)
    rng = random.Random(2)
    refused = 0
    while refused < 300:
        extents = [rng.choice([1, 2, 3, 4]) for _ in range(3)]
        D, D_v = rng.choice([(64, 64), (128, 128), (192, 128)])
        strides, span = [0, 0, 0], D
        for i in rng.sample(range(3), 3):
            strides[i] = span + 64 * rng.choice([0, 1, 2, 7])
            span = strides[i] * extents[i]
        offset = 16 * rng.randrange(-span // 16 - 20, span // 16 + 20)
        c, meet = _in_one_place(lib, extents, strides, D, D_v, offset)
        if meet:
            assert _store(lib, c, H=extents[2], q=0, k=A, v=A, slots=A) == 1
            refused += 1
        elif not torch.cuda.is_available():
            assert _store(lib, c, H=extents[2], q=0, k=A, v=A, slots=A) == 4    # past every check
    c, _ = _in_one_place(lib, (4, 16, 2), (4096, 256, 128), 128, 128, 0)
    assert _store(lib, c) == 1


@pytest.mark.parametrize("name", ["paged.cuh", "decode.cuh", "zyfa_paged_plan.cu", "zyfa_rope_store.cu"])
def test_kernels_that_start_early_read_by_ordinary_loads(name):
    # what they read is written by the kernel before, while they may already run: never read-only data
    text = open(os.path.join(build.CSRC, name)).read()
    assert "launch_dependent" in text
    for word in ("__ldg", "ld.global.nc", "ld.nc", "__restrict__", "tex."):
        assert word not in text, word


# Tokens that a request may have where it is one block's work: kLongest tiles of at most 128 tokens (4 warps of 32 keys)
SMALL_TABLE = 8 * 128


def _launches(lib, kind, shape, H, H_kv, page, tokens, B):  # noqa: F811
    D, D_v = shape
    c = _cache(dtype=kind, page_size=page, num_pages=1000, H_kv=H_kv, D_qk=D, D_v=D_v, k_page_stride=page * H_kv * D, k_token_stride=H_kv * D,
               k_head_stride=D, v_page_stride=page * H_kv * D_v, v_token_stride=H_kv * D_v, v_head_stride=D_v)
    return lib.zyfa_attn_decode_paged_launches(ctypes.byref(c), -(-tokens // page), B, H, 152)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("shape,H,H_kv", [((64, 64), 16, 16), ((64, 64), 2, 2), ((128, 128), 32, 8), ((128, 128), 32, 32), ((128, 128), 40, 40),
                                          ((128, 128), 64, 4), ((128, 128), 32, 1), ((192, 128), 16, 16), ((192, 128), 128, 128)])
def test_requests_of_wide_tables_are_split_whatever_their_number(lib, kind, shape, H, H_kv):  # noqa: F811
    """Lengths are not known where the work is divided.  A table of many tokens may hold one long request among short ones at every
    number of requests, also where whole requests would fill the GPU evenly were all as long."""
    for page in (16, 64):
        for tokens in (2 * SMALL_TABLE, 4096, 8192, 32768, 131072):
            assert {_launches(lib, kind, shape, H, H_kv, page, tokens, B) for B in range(1, 513)} == {2}
    # a few tokens are one block's work
    assert _launches(lib, kind, shape, H, H_kv, 16, 16, 1) == 1 and _launches(lib, kind, shape, H, H_kv, 16, 32, 100) == 1


def test_launch_counts_of_refused_calls_and_odd_pages(lib):  # noqa: F811
    assert _launches(lib, 0, (128, 128), 32, 8, 16, 64, 32) == 1 and _launches(lib, 0, (128, 128), 32, 8, 7, 64, 32) == 2
    assert _launches(lib, 0, (128, 128), 32, 8, 16, 64, 0) == 0 and _launches(lib, 0, (128, 96), 32, 8, 16, 64, 1) == 0
    assert _launches(lib, 0, (128, 128), 31, 8, 16, 64, 1) == 0 and lib.zyfa_attn_decode_paged_launches(None, 4, 1, 8, 152) == 0
    assert lib.zyfa_attn_decode_paged_launches(ctypes.byref(_cache()), 4, 1, 4, -1) == 0


def test_decode_forms_of_descales(lib):  # noqa: F811
    # one value, one a request and head (1), one a head for all requests (3); for no requests, since addresses are not memory
    assert [_decode(lib, _cache(), B=0, per=per) for per in (0, 1, 3)] == [0, 0, 0]
    assert [_decode(lib, _cache(), B=0, per=per) for per in (2, 4, -1)] == [1, 1, 1]


def test_stalled_self_test_validates_its_arguments_like_the_call(lib):  # noqa: F811
    def call(B=3, H=4, ws=A, q=A, page=16):
        return lib.zyfa_selftest_stalled_decode(q or None, 512, ctypes.byref(_cache(page_size=page)), A, 8, 8, A, A, B, H, ws or None, 1 << 40, None)

    assert [call(B=0), call(B=-1), call(H=3), call(ws=0), call(q=0), call(q=A + 8), call(page=0), call(B=65537)] == [0, 1, 1, 1, 1, 3, 1, 2]


# Buffers far apart, none of which is memory: calls that are accepted are made only where there is no GPU
FAR = {name: (i + 1) << 32 for i, name in enumerate(("q", "k", "v", "qo", "ko", "vo", "kc", "vc", "c", "n", "t", "free", "ci", "co", "sl", "cu", "pos", "slots"))}


def _accepted(call):
    return torch.cuda.is_available() or call() == 4


# 10 tokens of 4 and 2 heads of 128 channels, bf16; an e4m3 cache: q_out has 5120 bytes, k_out and v_out 2560
STORE = dict(qs=1024, ks=1024, vs=1024, H=4, **{x: FAR[x] for x in ("q", "k", "v", "qo", "ko", "vo", "slots")})


@pytest.mark.parametrize("kw,apart", [
    ({}, True), (dict(k=FAR["q"] + 1024, v=FAR["q"] + 1536), True),             # slices of one projection
    (dict(ko=FAR["qo"] + 5120), True), (dict(ko=FAR["qo"] - 2560), True), (dict(vo=FAR["ko"] + 2560), True),
    (dict(qo=FAR["q"] + 9 * 2048 + 1024), True), (dict(qo=FAR["q"] - 5120), True), (dict(ko=FAR["q"], q=0), True),
    (dict(ko=FAR["qo"]), False), (dict(ko=FAR["qo"] + 5104), False), (dict(ko=FAR["qo"] - 2544), False), (dict(vo=FAR["ko"]), False),
    (dict(vo=FAR["qo"] + 16), False), (dict(qo=FAR["q"]), False), (dict(qo=FAR["q"] + 9 * 2048 + 1008), False), (dict(qo=FAR["q"] - 5104), False),
    (dict(ko=FAR["k"] + 2048), False), (dict(vo=FAR["q"] + 1040), False), (dict(qo=FAR["v"] + 9 * 2048), False)])
def test_store_refuses_outputs_that_overlap(lib, kw, apart):  # noqa: F811
    call = lambda: _store(lib, _cache(k=FAR["kc"], v=FAR["vc"]), **{**STORE, **kw})  # noqa: E731
    assert _accepted(call) if apart else call() == 1


PLAN = dict(B=4, mp=8, ts=10, nf=10, mt=32, **{x: FAR[x] for x in ("c", "n", "t", "free", "ci", "co", "sl", "cu", "pos", "slots")})


@pytest.mark.parametrize("kw,apart", [
    ({}, True), (dict(co=FAR["ci"]), True), (dict(cu=FAR["sl"] + 16), True), (dict(sl=FAR["cu"] + 20), True), (dict(n=FAR["c"] + 16), True),
    (dict(c=FAR["t"] + 32, B=1), True), (dict(co=FAR["t"] + 32), True), (dict(pos=FAR["slots"] + 256), True), (dict(sl=FAR["c"], B=0), True),
    (dict(sl=FAR["c"] + 12), False), (dict(sl=FAR["n"] - 12), False), (dict(cu=FAR["c"] - 16), False), (dict(cu=FAR["sl"] + 12), False),
    (dict(pos=FAR["slots"] + 252), False), (dict(slots=FAR["pos"] + 120), False), (dict(co=FAR["sl"] + 12), False), (dict(co=FAR["free"] + 36), False),
    (dict(co=FAR["t"] + 28), False), (dict(co=FAR["t"] + 3 * 40), False), (dict(pos=FAR["free"] + 36), False), (dict(slots=FAR["ci"] - 248), False),
    (dict(sl=FAR["t"] + 32), False)])
def test_plan_refuses_results_that_overlap(lib, kw, apart):  # noqa: F811
    call = lambda: _plan(lib, **{**PLAN, **kw})  # noqa: E731
    assert _accepted(call) if apart else call() == 1
