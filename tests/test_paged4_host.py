"""Refusals of the operators of the 4-bit paged cache, without a GPU: the C entry points reject bad arguments before anything is
enqueued, the tensor-level calls before the library is reached."""
import ctypes
import os
import random

import pytest
import torch

from fp8_causal_prefill_gb300 import api, build, paged_decode_attn, paged_read, rope_paged_store
from test_paged_edges_host import _overlap, _rows
from test_paged_host import A, BAD_CACHES, _rope, lib  # noqa: F401

# Buffers far apart, none of which is memory: calls that are accepted are made only where there is no GPU
NAMES = ("q", "k", "v", "qo", "ko", "vo", "kc", "vc", "ks", "vs", "table", "cu", "starts", "slots", "pos", "d")
FAR = {name: (i + 1) << 32 for i, name in enumerate(NAMES)}


def n_(x):
    return x or None


def _accepted(call):
    return torch.cuda.is_available() or call() == 4


def _cache(**kw):
    c = dict(k=FAR["kc"], v=FAR["vc"], dtype=2, page_size=16, num_pages=4, H_kv=2, D_qk=128, D_v=128, k_page_stride=2048, k_token_stride=128,
             k_head_stride=64, v_page_stride=2048, v_token_stride=128, v_head_stride=64)
    c.update(kw)
    return api.PagedCache(*(c[name] for name, _ in api.PagedCache._fields_))


def _scales(**kw):
    c = dict(k=FAR["ks"], v=FAR["vs"], k_page_stride=256, k_token_stride=16, k_head_stride=8, v_page_stride=256, v_token_stride=16,
             v_head_stride=8)
    c.update(kw)
    return api.PagedScales(*(c[name] for name, _ in api.PagedScales._fields_))


def _ref(x):
    return ctypes.byref(x) if x else None


def _store(lib, cache, scales, rope=None, **kw):  # noqa: F811
    a = dict(q=FAR["q"], k=FAR["k"], v=FAR["v"], qs=512, ks=256, vs=256, qo=FAR["qo"], ko=0, vo=0, pos=FAR["pos"], ps=10, slots=FAR["slots"], N=10,
             H=4, dk=0, dv=0, per=0)
    a.update(kw)
    return lib.zyfa_rope_paged_store_e2m1(n_(a["q"]), n_(a["k"]), n_(a["v"]), a["qs"], a["ks"], a["vs"], n_(a["qo"]), n_(a["ko"]), n_(a["vo"]),
                                          n_(a["pos"]), a["ps"], n_(a["slots"]), a["N"], a["H"], _ref(cache), _ref(scales), _ref(rope), n_(a["dk"]),
                                          n_(a["dv"]), a["per"], None)


def _decode(lib, cache, scales, **kw):  # noqa: F811
    a = dict(q=A, qs=512, table=A, ts=8, mp=8, lens=A, out=A, lse=0, B=3, H=4, scale=0.0, dk=0, dv=0, per=0, ws=A, wb=1 << 40)
    a.update(kw)
    return lib.zyfa_attn_decode_paged_e2m1(n_(a["q"]), a["qs"], _ref(cache), _ref(scales), n_(a["table"]), a["ts"], a["mp"], n_(a["lens"]),
                                           n_(a["out"]), n_(a["lse"]), a["B"], a["H"], a["scale"], n_(a["dk"]), n_(a["dv"]), a["per"],
                                           n_(a["ws"]), a["wb"], None)


def _stalled(lib, cache, scales, **kw):  # noqa: F811
    a = dict(q=A, qs=512, table=A, ts=8, mp=8, lens=A, out=A, B=3, H=4, ws=A, wb=1 << 40)
    a.update(kw)
    return lib.zyfa_selftest_stalled_decode_e2m1(n_(a["q"]), a["qs"], _ref(cache), _ref(scales), n_(a["table"]), a["ts"], a["mp"], n_(a["lens"]),
                                                 n_(a["out"]), a["B"], a["H"], n_(a["ws"]), a["wb"], None)


def _read(lib, cache, scales, **kw):  # noqa: F811
    a = dict(table=FAR["table"], ts=8, mp=8, cu=FAR["cu"], starts=FAR["starts"], B=3, ko=FAR["ko"], vo=FAR["vo"], N=10, out=1, dk=0, dv=0, per=0,
             ok=0, ov=0, operh=0)
    a.update(kw)
    return lib.zyfa_paged_read(_ref(cache), _ref(scales), n_(a["table"]), a["ts"], a["mp"], n_(a["cu"]), n_(a["starts"]), a["B"], n_(a["ko"]),
                               n_(a["vo"]), a["N"], a["out"], n_(a["dk"]), n_(a["dv"]), a["per"], n_(a["ok"]), n_(a["ov"]), a["operh"], None)


CALLS = (_store, _decode, _stalled, _read)


@pytest.mark.parametrize("kw,expect", [b for b in BAD_CACHES if "k_token_stride" not in b[0]] + [(dict(k_token_stride=136), 3), (dict(dtype=-1), 1)])
def test_bad_caches_are_refused(lib, kw, expect):  # noqa: F811
    for call in CALLS:
        assert call(lib, _cache(**kw), _scales()) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(k=0), 1), (dict(v=0), 1), (dict(k=A + 2), 3), (dict(v=A + 1), 3), (dict(k_page_stride=-4), 1), (dict(v_head_stride=-8), 1),
    (dict(k_token_stride=18), 3), (dict(v_head_stride=2), 3), (dict(k_head_stride=1 << 47), 2), (dict(v_page_stride=1 << 47), 2)])
def test_bad_scales_are_refused(lib, kw, expect):  # noqa: F811
    for call in CALLS:
        assert call(lib, _cache(), _scales(**kw)) == expect


def test_each_call_takes_the_caches_it_is_for(lib):  # noqa: F811
    for call in CALLS:
        assert call(lib, None, _scales()) == 1 and call(lib, _cache(), None) == 1
    for dtype in (0, 1):
        wide = _cache(dtype=dtype, k_page_stride=4096, v_page_stride=4096, k_token_stride=256, v_token_stride=256, k_head_stride=128, v_head_stride=128)
        assert [call(lib, wide, _scales()) for call in CALLS] == [1, 1, 1, 1]
        assert _accepted(lambda: _read(lib, wide, None))
        # and the calls for wider caches take none of 4 bits
        four = ctypes.byref(_cache())
        assert lib.zyfa_attn_decode_paged(A, 512, four, A, 8, 8, A, A, None, 3, 4, 0.0, None, None, None, 0, A, 1 << 40, None) == 1
        assert lib.zyfa_rope_paged_store(A, A, A, 512, 256, 256, A, None, None, A, 10, A, 10, 4, four, None, None, None, None, 0, None) == 1
        assert lib.zyfa_selftest_stalled_decode(A, 512, four, A, 8, 8, A, A, 3, 4, A, 1 << 40, None) == 1
        assert lib.zyfa_attn_decode_paged_launches(four, 4, 1, 4, 152) == 0


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), 1), (dict(H=0), 1), (dict(H=3), 1), (dict(per=2), 1), (dict(per=3), 1), (dict(q=0, k=0, v=0), 1), (dict(k=0), 1), (dict(v=0), 1),
    (dict(qo=0), 1), (dict(slots=0), 1), (dict(qs=-8), 1), (dict(N=1 << 31), 2), (dict(H=1 << 17), 2), (dict(ks=1 << 41), 2),
    (dict(q=A + 8), 3), (dict(k=A + 2), 3), (dict(v=A + 4), 3), (dict(qo=A + 8), 3), (dict(ko=A + 8), 3), (dict(vo=A + 1), 3),
    (dict(qs=516), 3), (dict(ks=257), 3), (dict(vs=258), 3), (dict(slots=A + 4), 3), (dict(dk=A + 2), 3), (dict(dv=A + 3), 3),
    (dict(N=0), 0), (dict(N=0, q=A, slots=0, qo=0), 0)])
def test_store_refusals(lib, kw, expect):  # noqa: F811
    assert _store(lib, _cache(), _scales(), **kw) == expect


@pytest.mark.parametrize("kw,more,expect", [
    (dict(rot=24, pairs=(12, 0, 0, 0)), {}, 1), (dict(offset=8), {}, 1), (dict(rot=64, offset=4, pairs=(32, 0, 0, 0)), {}, 1),
    (dict(axes=2, pairs=(32, 31, 0, 0)), {}, 1), (dict(inv=None), {}, 1), (dict(), dict(pos=0), 1),
    (dict(axes=2, pairs=(32, 32, 0, 0)), dict(ps=9), 1), (dict(inv=A + 2), {}, 3), (dict(), dict(pos=A + 2), 3)])
def test_rope_refusals(lib, kw, more, expect):  # noqa: F811
    assert _store(lib, _cache(), _scales(), _rope(**kw), **more) == expect


def _strides(which, strides):
    return {f"{which}_{n}_stride": s for n, s in zip(("page", "token", "head"), strides)}


# 4 pages of 16 tokens of 2 heads: (page, token, head) strides of rows of 64 bytes of codes; an eighth of them for 8 bytes of scales
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("strides,apart", [
    ((2048, 128, 64), True), ((2048, 64, 1024), True), ((4096, 256, 128), True), ((128, 512, 64), True), ((1 << 46, 128, 64), True),
    ((2048, 64, 64), False), ((64, 128, 64), False), ((2048, 64, 128), False), ((2016, 128, 64), False), ((2048, 128, 32), False),
    ((0, 128, 64), False), ((2048, 0, 64), False), ((2048, 128, 0), False)])
def test_store_refuses_rows_that_overlap(lib, strides, apart, which):  # noqa: F811
    assert _overlap(strides, (4, 16, 2), 64) == (not apart)
    assert _store(lib, _cache(**_strides(which, strides)), _scales(), N=0) == (0 if apart else 1)
    assert _store(lib, _cache(), _scales(**_strides(which, [s // 8 for s in strides])), N=0) == (0 if apart else 1)
    # reading through such strides is well defined
    assert _accepted(lambda: _read(lib, _cache(**_strides(which, strides)), _scales(), ko=1 << 60, vo=1 << 61))
    assert _decode(lib, _cache(**_strides(which, strides)), _scales(**_strides(which, [s // 8 for s in strides])), B=0) == 0


def test_store_refuses_two_of_the_four_tensors_in_one_place(lib):  # noqa: F811
    """K, V and the scales of both within rows of the same strides, at random offsets."""
    rng = random.Random(3)
    refused = 0
    while refused < 300:
        extents = [rng.choice([1, 2, 3]) for _ in range(3)]
        D, D_v = rng.choice([(64, 64), (128, 128), (192, 128)])
        sizes = {"kc": D // 2, "vc": D_v // 2, "ks": D // 16, "vs": D_v // 16}
        strides, span = [0, 0, 0], 16 * -(-sum(sizes.values()) // 16)
        for i in rng.sample(range(3), 3):
            strides[i] = span + 16 * rng.choice([0, 0, 1, 7])
            span = strides[i] * extents[i]
        one, two = rng.sample(sorted(sizes), 2)
        step = 4 if "s" in one + two else 16
        at = dict(FAR)
        at[two] = at[one] + step * rng.randrange(-span // step - 5, span // step + 5)
        if at["kc"] % 16 or at["vc"] % 16:
            continue
        rows = _rows(strides, extents)
        meet = any(x - sizes[two] < y < x + sizes[one] for x in rows for y in (z + at[two] - at[one] for z in rows))
        c = _cache(k=at["kc"], v=at["vc"], num_pages=extents[0], page_size=extents[1], H_kv=extents[2], D_qk=D, D_v=D_v, **_strides("k", strides),
                   **_strides("v", strides))
        s = _scales(k=at["ks"], v=at["vs"], **_strides("k", strides), **_strides("v", strides))
        call = lambda: _store(lib, c, s, H=extents[2], ks=D * extents[2], vs=D_v * extents[2], q=0)  # noqa: E731,B023
        if meet:
            assert call() == 1
            refused += 1
        else:
            assert _accepted(call)


# 10 tokens of 4 and 2 heads of 128 channels, bf16: q_out has 10240 bytes, k_out and v_out 5120
STORE = dict(qs=1024, ks=1024, vs=1024, H=4, ko=FAR["ko"], vo=FAR["vo"])


@pytest.mark.parametrize("kw,apart", [
    ({}, True), (dict(k=FAR["q"] + 1024, v=FAR["q"] + 1536), True), (dict(ko=FAR["qo"] + 10240), True), (dict(ko=FAR["qo"] - 5120), True),
    (dict(vo=FAR["ko"] + 5120), True), (dict(ko=FAR["q"], q=0), True), (dict(ko=FAR["qo"], q=0), True), (dict(ko=FAR["qo"]), False),
    (dict(ko=FAR["qo"] + 10224), False), (dict(ko=FAR["qo"] - 5104), False), (dict(vo=FAR["ko"]), False), (dict(qo=FAR["q"]), False),
    (dict(qo=FAR["q"] - 10224), False), (dict(ko=FAR["k"] + 2048), False), (dict(vo=FAR["q"] + 1040), False)])
def test_store_refuses_outputs_that_overlap(lib, kw, apart):  # noqa: F811
    call = lambda: _store(lib, _cache(), _scales(), **{**STORE, **kw})  # noqa: E731
    assert _accepted(call) if apart else call() == 1


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), 1), (dict(H=0), 1), (dict(H=3), 1), (dict(mp=-1), 1), (dict(ts=7), 1), (dict(per=2), 1), (dict(per=4), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(qs=-16), 1),
    (dict(q=0), 1), (dict(out=0), 1), (dict(lens=0), 1), (dict(table=0), 1), (dict(ws=0), 1), (dict(wb=0), 1),
    (dict(mp=1 << 27, ts=1 << 27), 2), (dict(B=65537), 2), (dict(H=65538), 2), (dict(B=60000, H=4096), 2), (dict(B=65536, mp=1 << 15, ts=1 << 15), 2),
    (dict(q=A + 8), 3), (dict(qs=516), 3), (dict(out=A + 2), 3), (dict(lens=A + 2), 3), (dict(table=A + 1), 3),
    (dict(lse=A + 2), 3), (dict(dk=A + 1), 3), (dict(dv=A + 3), 3), (dict(ws=A + 4), 3), (dict(B=0), 0), (dict(B=0, per=3), 0),
    (dict(B=0, q=0, out=0, lens=0, table=0, ws=0), 0)])
def test_decode_refusals(lib, kw, expect):  # noqa: F811
    assert _decode(lib, _cache(), _scales(), **kw) == expect
    if not {"scale", "per", "lse", "dk", "dv"} & set(kw):
        assert _stalled(lib, _cache(), _scales(), **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), 1), (dict(N=-1), 1), (dict(mp=-1), 1), (dict(ts=7), 1), (dict(per=2), 1), (dict(per=-1), 1), (dict(operh=2), 1), (dict(operh=3), 1),
    (dict(out=2), 1), (dict(out=-1), 1), (dict(ko=0, vo=0), 1), (dict(cu=0), 1), (dict(table=0), 1), (dict(mp=1 << 27, ts=1 << 27), 2),
    (dict(B=65537), 2), (dict(N=1 << 31), 2), (dict(ko=A + 8), 3), (dict(vo=A + 4), 3), (dict(table=A + 2), 3), (dict(cu=A + 1), 3),
    (dict(starts=A + 2), 3), (dict(dk=A + 2), 3), (dict(dv=A + 1), 3), (dict(ok=A + 3), 3), (dict(ov=A + 2), 3), (dict(N=0), 0), (dict(B=0), 0),
    (dict(N=0, cu=0, table=0, ko=0, vo=0), 0)])
def test_read_refusals(lib, kw, expect):  # noqa: F811
    assert _read(lib, _cache(), _scales(), **kw) == expect
    assert _read(lib, _cache(H_kv=65537), _scales()) == 2


# 10 rows of 2 heads of 128 channels as bf16 are 5120 bytes, as e4m3 2560; the cache's codes 8192, its scales 1024
@pytest.mark.parametrize("kw,apart", [
    ({}, True), (dict(starts=0), True), (dict(ko=0), True), (dict(vo=0), True), (dict(mp=0, ts=0, table=0), True), (dict(per=1, dk=FAR["d"]), True),
    (dict(vo=FAR["ko"] + 5120), True), (dict(vo=FAR["ko"] - 5120), True), (dict(ko=FAR["kc"] - 5120, vo=FAR["vc"] + 8192), True),
    (dict(ko=FAR["ks"] - 5120, vo=FAR["vs"] + 1024), True), (dict(ko=FAR["cu"] + 16, vo=FAR["table"] - 5120), True), (dict(out=0, vo=FAR["ko"] + 2560), True),
    (dict(vo=FAR["ko"]), False), (dict(vo=FAR["ko"] + 5104), False), (dict(out=0, vo=FAR["ko"] + 2544), False), (dict(ko=FAR["kc"]), False),
    (dict(ko=FAR["kc"] - 5104), False), (dict(vo=FAR["kc"] + 8176), False), (dict(vo=FAR["vc"] + 16), False), (dict(ko=FAR["ks"] + 1008), False),
    (dict(vo=FAR["vs"] - 5104), False), (dict(ko=FAR["table"] + 64), False), (dict(vo=FAR["cu"]), False), (dict(ko=FAR["starts"]), False),
    (dict(ko=FAR["d"] + 16, dk=FAR["d"], per=1), False), (dict(ko=FAR["d"] + 16, dk=FAR["d"], per=3), True), (dict(vo=FAR["d"], dv=FAR["d"]), False),
    (dict(out=0, vo=FAR["d"], ov=FAR["d"]), False)])
def test_read_refuses_outputs_that_overlap(lib, kw, apart):  # noqa: F811
    call = lambda: _read(lib, _cache(), _scales(), **kw)  # noqa: E731
    assert _accepted(call) if apart else call() == 1


@pytest.mark.parametrize("name", ["decode_e2m1.cuh", "rope.cuh", "zyfa_decode_e2m1.cu", "zyfa_rope_store_e2m1.cu", "zyfa_paged_read.cu"])
def test_kernels_that_start_early_read_by_ordinary_loads(name):
    text = open(os.path.join(build.CSRC, name)).read()
    for word in ("__ldg", "ld.global.nc", "ld.nc", "__restrict__", "tex."):
        assert word not in text, word


def test_tensor_calls_refuse_host_tensors_and_wrong_types():
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    codes, scales = torch.zeros(4, 16, 2, 64, dtype=u8), torch.zeros(4, 16, 2, 8, dtype=u8)
    lens, table, slots = torch.zeros(3, dtype=i32), torch.zeros(3, 4, dtype=i32), torch.zeros(3, dtype=torch.int64)
    q = torch.zeros(3, 4, 128, dtype=bf)
    calls = [lambda c, s: paged_decode_attn(q, c, c, table, lens, k_scales=s, v_scales=s),
             lambda c, s: rope_paged_store(q, None, None, c, c, slots, k_scales=s, v_scales=s),
             lambda c, s: paged_read(c, c, table, torch.zeros(4, dtype=i32), 8, k_scales=s, v_scales=s)]
    for call in calls:
        with pytest.raises(ValueError):
            call(codes, scales)                                                 # not on a GPU
        with pytest.raises(TypeError):
            call(codes.to(bf), scales)
        with pytest.raises(TypeError):
            call(codes, scales.float())
        with pytest.raises(TypeError):
            call(codes[0], scales)
    for one in (dict(k_scales=scales), dict(v_scales=scales)):
        with pytest.raises(TypeError):
            paged_decode_attn(q, codes, codes, table, lens, **one)
        with pytest.raises(TypeError):
            rope_paged_store(q, None, None, codes, codes, slots, **one)
        with pytest.raises(TypeError):
            paged_read(codes, codes, table, lens, 8, **one)
    with pytest.raises(TypeError):
        paged_read(codes, codes, table, lens, 8, dtype=torch.float16, k_scales=scales, v_scales=scales)
