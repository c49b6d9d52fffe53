"""Refusals of the paged serving operators, without a GPU: the C entry points reject bad arguments before
anything is enqueued, the tensor-level calls before the library is reached."""
import ctypes

import pytest
import torch

from fp8_causal_prefill_gb300 import Rope, api, build, paged_decode_attn, paged_plan, rope_paged_store

A = 1 << 20  # a 16-byte aligned fake address; validation rejects the calls before any dereference


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load_library()


def _cache(**kw):
    c = dict(k=A, v=A, dtype=0, page_size=16, num_pages=4, H_kv=2, D_qk=128, D_v=128)
    c.update({k: v for k, v in kw.items() if k in c})
    c.update(k_page_stride=4096, k_token_stride=256, k_head_stride=128, v_page_stride=4096, v_token_stride=256,
             v_head_stride=128)
    c.update(kw)
    return api.PagedCache(*(c[name] for name, _ in api.PagedCache._fields_))


BAD_CACHES = [(dict(dtype=5), 1), (dict(page_size=0), 1), (dict(page_size=65537), 1), (dict(num_pages=0), 1), (dict(H_kv=0), 1),
              (dict(D_qk=96), 2), (dict(D_v=64), 2), (dict(k=0), 1), (dict(v=0), 1), (dict(k=A + 8), 3), (dict(v=A + 1), 3),
              (dict(k_page_stride=-16), 1), (dict(k_token_stride=264), 3), (dict(v_head_stride=8), 3),
              (dict(num_pages=1 << 31), 2), (dict(v_page_stride=1 << 47), 2)]


def _decode(lib, cache, **kw):
    a = dict(q=A, qs=512, table=A, ts=8, mp=8, lens=A, out=A, lse=0, B=3, H=4, scale=0.0, dq=0, dk=0, dv=0, per=0, ws=A,
             wb=1 << 40)
    a.update(kw)
    n = lambda x: x or None  # noqa: E731
    return lib.zyfa_attn_decode_paged(n(a["q"]), a["qs"], ctypes.byref(cache) if cache else None, n(a["table"]), a["ts"], a["mp"],
                                      n(a["lens"]), n(a["out"]), n(a["lse"]), a["B"], a["H"], a["scale"], n(a["dq"]), n(a["dk"]),
                                      n(a["dv"]), a["per"], n(a["ws"]), a["wb"], None)


@pytest.mark.parametrize("kw,expect", BAD_CACHES)
def test_bad_caches_are_refused(lib, kw, expect):
    assert _decode(lib, _cache(**kw)) == expect
    assert _store(lib, _cache(**kw)) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), 1), (dict(H=0), 1), (dict(H=3), 1), (dict(mp=-1), 1), (dict(ts=7), 1), (dict(per=2), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(qs=-16), 1),
    (dict(q=0), 1), (dict(out=0), 1), (dict(lens=0), 1), (dict(table=0), 1), (dict(ws=0), 1), (dict(wb=0), 1),
    (dict(mp=1 << 27, ts=1 << 27), 2), (dict(B=65537), 2), (dict(H=65538), 2), (dict(B=60000, H=4096), 2),
    (dict(q=A + 8), 3), (dict(qs=520), 3), (dict(out=A + 2), 3), (dict(lens=A + 2), 3), (dict(table=A + 1), 3),
    (dict(lse=A + 2), 3), (dict(dq=A + 2), 3), (dict(dk=A + 1), 3), (dict(dv=A + 3), 3), (dict(ws=A + 4), 3),
    (dict(B=0), 0), (dict(B=0, q=0, out=0, lens=0, table=0, ws=0), 0),
])
def test_decode_refusals(lib, kw, expect):
    assert _decode(lib, _cache(), **kw) == expect


def test_decode_refuses_more_tiles_than_its_schedule_numbers(lib):
    # 65536 requests of 2^15 tiles: 2^31, and just below that with what lies between the requests
    assert _decode(lib, _cache(), B=65536, mp=1 << 15, ts=1 << 15) == 2
    assert _decode(lib, _cache(), B=65536, mp=(1 << 15) - 1, ts=1 << 15) == 2


def test_decode_needs_a_cache(lib):
    assert _decode(lib, None) == 1
    assert _store(lib, None) == 1


def test_decode_workspace_sizes(lib):
    f = lib.zyfa_attn_decode_paged_workspace_bytes
    assert f(0, 4, 2, 128, 64) == 0 and f(1, 3, 2, 128, 64) == 0 and f(1, 0, 1, 128, 64) == 0 and f(1, 2, 0, 128, 64) == 0
    assert f(1, 2, 2, 96, 64) == 0 and f(1, 2, 2, 128, -1) == 0
    assert 0 < f(1, 2, 2, 128, 0) <= f(1, 2, 2, 128, 256) < f(1, 2, 2, 128, 1 << 20) < f(4, 64, 2, 128, 1 << 20) < 1 << 26


def _store(lib, cache, rope=None, **kw):
    a = dict(q=A, k=A, v=A, qs=512, ks=256, vs=256, qo=A, ko=0, vo=0, pos=A, ps=10, slots=A, N=10, H=4, dq=0, dk=0, dv=0, per=0)
    a.update(kw)
    n = lambda x: x or None  # noqa: E731
    return lib.zyfa_rope_paged_store(n(a["q"]), n(a["k"]), n(a["v"]), a["qs"], a["ks"], a["vs"], n(a["qo"]), n(a["ko"]), n(a["vo"]),
                                     n(a["pos"]), a["ps"], n(a["slots"]), a["N"], a["H"], ctypes.byref(cache) if cache else None,
                                     ctypes.byref(rope) if rope else None, n(a["dq"]), n(a["dk"]), n(a["dv"]), a["per"], None)


def _rope(inv=A, rot=128, offset=0, interleaved=0, axes=1, pairs=(64, 0, 0, 0)):
    return api.RopeOptions(inv, rot, offset, interleaved, axes, (ctypes.c_int * 4)(*pairs))


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), 1), (dict(H=0), 1), (dict(H=3), 1), (dict(per=2), 1), (dict(q=0, k=0, v=0), 1), (dict(k=0), 1), (dict(v=0), 1),
    (dict(qo=0), 1), (dict(slots=0), 1), (dict(qs=-8), 1), (dict(N=1 << 31), 2), (dict(H=1 << 17), 2), (dict(ks=1 << 41), 2),
    (dict(q=A + 8), 3), (dict(k=A + 2), 3), (dict(v=A + 4), 3), (dict(qo=A + 8), 3), (dict(ko=A + 8), 3), (dict(vo=A + 1), 3),
    (dict(qs=516), 3), (dict(ks=257), 3), (dict(vs=258), 3), (dict(slots=A + 4), 3), (dict(dq=A + 1), 3), (dict(dk=A + 2), 3),
    (dict(dv=A + 3), 3), (dict(N=0), 0), (dict(N=0, q=A, slots=0, qo=0), 0),
])
def test_store_refusals(lib, kw, expect):
    assert _store(lib, _cache(), **kw) == expect


@pytest.mark.parametrize("kw,more,expect", [
    (dict(rot=-16), {}, 1), (dict(rot=24, pairs=(12, 0, 0, 0)), {}, 1), (dict(rot=144, pairs=(72, 0, 0, 0)), {}, 1),
    (dict(offset=8), {}, 1), (dict(offset=-8), {}, 1), (dict(rot=64, offset=4, pairs=(32, 0, 0, 0)), {}, 1),
    (dict(interleaved=2), {}, 1), (dict(axes=0), {}, 1), (dict(axes=5), {}, 1), (dict(pairs=(63, 0, 0, 0)), {}, 1),
    (dict(axes=2, pairs=(65, -1, 0, 0)), {}, 1), (dict(axes=2, pairs=(32, 31, 0, 0)), {}, 1), (dict(inv=None), {}, 1),
    (dict(), dict(pos=0), 1), (dict(axes=2, pairs=(32, 32, 0, 0)), dict(ps=9), 1), (dict(inv=A + 2), {}, 3), (dict(), dict(pos=A + 2), 3),
])
def test_rope_refusals(lib, kw, more, expect):
    assert _store(lib, _cache(), _rope(**kw), **more) == expect


def test_store_refuses_overlapping_cache_rows(lib):
    # reading through such strides is well defined, writing is not
    for kw in (dict(k_head_stride=0), dict(v_head_stride=64), dict(k_token_stride=0), dict(v_token_stride=64),
               dict(k_page_stride=0), dict(v_page_stride=16)):
        assert _store(lib, _cache(**kw)) == 1


def _plan(lib, **kw):
    a = dict(c=A, n=A, B=4, page=16, t=A, ts=8, mp=8, free=A, nf=10, ci=A, co=A, sl=A, cu=A, pos=A, slots=A, mt=32)
    a.update(kw)
    n = lambda x: x or None  # noqa: E731
    return lib.zyfa_paged_plan(n(a["c"]), n(a["n"]), a["B"], a["page"], n(a["t"]), a["ts"], a["mp"], n(a["free"]), a["nf"], n(a["ci"]),
                               n(a["co"]), n(a["sl"]), n(a["cu"]), n(a["pos"]), n(a["slots"]), a["mt"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), 1), (dict(mt=-1), 1), (dict(nf=-1), 1), (dict(mp=-1), 1), (dict(ts=7), 1), (dict(page=0), 1), (dict(page=65537), 1),
    (dict(c=0), 1), (dict(n=0), 1), (dict(t=0), 1), (dict(free=0), 1), (dict(ci=0), 1), (dict(co=0), 1), (dict(sl=0), 1),
    (dict(cu=0), 1), (dict(pos=0), 1), (dict(slots=0), 1), (dict(mp=1 << 27, ts=1 << 27), 2), (dict(B=65537), 2),
    (dict(c=A + 1), 3), (dict(n=A + 2), 3), (dict(t=A + 2), 3), (dict(free=A + 2), 3), (dict(ci=A + 2), 3), (dict(co=A + 2), 3),
    (dict(sl=A + 2), 3), (dict(cu=A + 2), 3), (dict(pos=A + 2), 3), (dict(slots=A + 4), 3),
])
def test_plan_refusals(lib, kw, expect):
    assert _plan(lib, **kw) == expect


def test_plan_refuses_results_in_place_of_the_lengths(lib):
    # several blocks read the lengths, each at its own time
    far = dict(c=A, n=A + 64, t=A + 128, free=A + 512, ci=A + 1024, co=A + 1024, sl=A + 2048, cu=A + 2560, pos=A + 4096, slots=A + 8192)
    for kw in (dict(sl=far["c"]), dict(sl=far["n"]), dict(cu=far["c"]), dict(cu=far["n"])):
        assert _plan(lib, **{**far, **kw}) == 1


def test_tensor_calls_refuse_host_tensors_and_wrong_types():
    bf, i32 = torch.bfloat16, torch.int32
    cache = torch.zeros(4, 16, 2, 128, dtype=bf)
    lens, table = torch.zeros(3, dtype=i32), torch.zeros(3, 4, dtype=i32)
    q = torch.zeros(3, 4, 128, dtype=bf)
    with pytest.raises(ValueError):
        paged_decode_attn(q, cache, cache, table, lens)                       # not on a GPU
    with pytest.raises(TypeError):
        paged_decode_attn(q, cache.half(), cache.half(), table, lens)
    with pytest.raises(TypeError):
        paged_decode_attn(q, cache, cache.float(), table, lens)
    with pytest.raises(ValueError):
        rope_paged_store(q, None, None, cache, cache, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        paged_plan(lens, lens, table, lens, lens[:1], 16, 8)
    with pytest.raises(TypeError):
        paged_plan(lens.long(), lens, table, lens, lens[:1], 16, 8)
    with pytest.raises(ValueError):
        paged_plan(lens, lens, table, lens, lens[:1], 16, -1)
    with pytest.raises(ValueError):
        Rope(torch.zeros(8))
    with pytest.raises(TypeError):
        Rope(torch.zeros(8, dtype=torch.float64))
