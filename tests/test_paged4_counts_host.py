"""Host tests of what a 4-bit decode call enqueues: the number of its launches, and whether tokens are loaded in boxes of a page."""
import ctypes

import pytest

from fp8_causal_prefill_gb300 import api
from test_paged4_host import FAR, _cache, _scales
from test_paged_host import lib  # noqa: F401

SHAPES = {"64": (64, 64), "128": (128, 128), "mla": (192, 128)}


def _dense(shape, H_kv, page, pages=1000, layout="nhd", **kw):
    """A dense cache and its scales: [page][token][head], or [page][head][token]."""
    strides = lambda n: (page * H_kv * n, H_kv * n, n) if layout == "nhd" else (page * H_kv * n, n, page * n)  # noqa: E731
    (d, dv), names = SHAPES[shape], ("page_stride", "token_stride", "head_stride")
    of = lambda k, v: {f"{t}_{name}": x for t, n in (("k", k), ("v", v)) for name, x in zip(names, strides(n))}  # noqa: E731
    cache = _cache(page_size=page, num_pages=pages, H_kv=H_kv, D_qk=d, D_v=dv, **{**of(d // 2, dv // 2), **kw.get("cache", {})})
    return cache, _scales(**{**of(d // 16, dv // 16), **kw.get("scales", {})})


def _count(lib, caches, B, H, max_pages, sms=152):  # noqa: F811
    """(launches, boxes: None if it was not told)."""
    boxes = ctypes.c_int(-1)
    n = lib.zyfa_attn_decode_paged_e2m1_launches(*(None if x is None else ctypes.byref(x) for x in caches), max_pages, B, H, sms, ctypes.byref(boxes))
    return n, None if boxes.value < 0 else boxes.value


# Tokens that a request may have where it is one block's work: 8 tiles of at most 128 tokens (4 warps of 32 keys)
SMALL_TABLE = 8 * 128


@pytest.mark.parametrize("shape,H,H_kv", [("64", 16, 16), ("64", 2, 2), ("64", 12, 1), ("128", 32, 8), ("128", 40, 40), ("128", 64, 4), ("128", 32, 1),
                                          ("mla", 16, 16), ("mla", 128, 128)])
def test_requests_of_wide_tables_are_split_whatever_their_number(lib, shape, H, H_kv):  # noqa: F811
    # (lengths are not known where the work is divided)
    for page in (16, 64, 7):
        for tokens in (2 * SMALL_TABLE, 8192, 131072):
            assert {_count(lib, _dense(shape, H_kv, page), B, H, -(-tokens // page))[0] for B in range(1, 513, 7)} == {2}
        # a few tokens are one block's work
        for B in (1, 3, 100):
            assert _count(lib, _dense(shape, H_kv, page), B, H, -(-32 // page))[0] == 1


@pytest.mark.parametrize("shape", ["64", "128", "mla"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_pages_of_multiples_of_8_tokens_come_in_boxes(lib, shape, layout):  # noqa: F811
    for page in (8, 16, 24, 48, 64, 256):
        for H_kv in (1, 2, 3, 4, 8, 12, 16):
            for group in (1, 4, 8, 16):
                assert _count(lib, _dense(shape, H_kv, page, layout=layout), 5, group * H_kv, 1000) == (2, 1), (page, H_kv, group)
    for page in (1, 4, 7, 20):
        assert _count(lib, _dense(shape, 4, page, layout=layout), 5, 16, 5000) == (2, 0)


@pytest.mark.parametrize("shape,of_many", [("64", (8, 12, 24)), ("128", (6, 8, 10, 14)), ("mla", (8, 12, 20))])
def test_numbers_of_heads_that_come_in_boxes(lib, shape, of_many):  # noqa: F811
    boxes = lambda H_kv, group, layout="nhd": _count(lib, _dense(shape, H_kv, 16, layout=layout), 5, group * H_kv, 500)[1] == 1  # noqa: E731
    assert all(boxes(H_kv, group) for H_kv in (1, 2, 3, 4, *of_many) for group in (1, 16))
    assert all(boxes(H_kv, 32) for H_kv in (1, 2)) and boxes(1, 33) and boxes(1, 64)
    assert shape != "128" or all(boxes(H_kv, 24) for H_kv in (4, *of_many))
    assert all(boxes(H_kv, group, "hnd") for H_kv in (1, 3, 5, 7, 10, 13) for group in (1, 9, 17, 40))


def test_strides_that_boxes_cannot_have(lib):  # noqa: F811
    piece = lambda **kw: _count(lib, _dense("128", 4, 16, **kw), 5, 16, 64) == (2, 0)  # noqa: E731
    assert not piece()
    for name in ("k_page_stride", "v_page_stride", "k_token_stride", "v_token_stride", "k_head_stride", "v_head_stride"):
        assert piece(cache={name: 0}), name
    assert piece(scales=dict(k_token_stride=36)) and piece(scales=dict(v_page_stride=516)) and piece(scales=dict(k=FAR["ks"] + 8))


@pytest.mark.parametrize("shape", ["64", "128", "mla"])
def test_one_page_has_no_page_stride(lib, shape):  # noqa: F811
    # (what a tensor of one page gives as the stride may be anything that the calls accept)
    for H_kv in (1, 2, 4, 8):
        for stride in (0, 4, 8, 12, 36):
            caches = _dense(shape, H_kv, 4096, pages=1, cache=dict(k_page_stride=0, v_page_stride=32), scales=dict(k_page_stride=stride, v_page_stride=stride))
            assert _count(lib, caches, 5, 4 * H_kv, 1) == (2, 1), (H_kv, stride)


def test_counts_of_refused_calls(lib):  # noqa: F811
    c, s = _dense("128", 4, 16)
    assert _count(lib, (c, s), 5, 16, 64) == (2, 1)
    assert lib.zyfa_attn_decode_paged_e2m1_launches(ctypes.byref(c), ctypes.byref(s), 64, 5, 16, 152, None) == 2
    for caches, B, H, sms in (((c, s), 0, 16, 152), ((c, s), -1, 16, 152), ((c, s), 5, 15, 152), ((c, s), 5, 16, -1), ((None, s), 5, 16, 152),
                              ((c, None), 5, 16, 152), ((_cache(dtype=0), s), 5, 2, 152), ((_cache(page_size=0), s), 5, 2, 152),
                              ((c, _scales(k=FAR["ks"] + 2)), 5, 16, 152), ((_cache(D_v=96), s), 5, 2, 152)):
        assert _count(lib, caches, B, H, 64, sms) == (0, None)
    assert _count(lib, (c, s), 5, 16, 1 << 27) == (0, None)                     # more than 2^30 tokens
