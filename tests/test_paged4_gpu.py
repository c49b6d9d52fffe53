"""GPU tests of the 4-bit paged cache against its float64 oracle: rotation and store, reading back, single-token attention, and a
run of them together."""
import math

import numpy as np
import pytest
import torch

from _paged4_util import fill4, held_of, make_cache4, random_codes, raw
from _paged_util import E4M3, SHAPES, bits, decode_tolerance, f64, make_cache, poisoned, random_table, random_values
from fp8_causal_prefill_gb300 import (Rope, flash_attn_func, paged_decode_attn, paged_decode_workspace_bytes, paged_plan, paged_read,
                                      rope_paged_store, zyfa_check_errors)
from oracle import paged as P
from oracle import paged4 as Q
from oracle.formats import e4m3_decode, e4m3_encode_rne_satfinite

pytestmark = pytest.mark.gpu

BAD_PAGE = 7


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f32(x):
    return torch.tensor(x, dtype=torch.float32, device="cuda")


# ------------------------------------------------------------------------------------------------
# rotation and store

def _near_held(codes, scales, z, slack):
    """Codes and scales against float64 values z over the descale, which the kernel's z is within `slack` of.

    The scale is max|z| / 6 to within half a step of e4m3 (2^-4 of it, 2^-10 where it is below 2^-6), the product by 1/6 and its constant
    rounding once each; a code is within half the distance to its neighbours, 0.25 below 2, 0.5 below 4, else 1, or 6 (1 + 2^-4) - 6 where
    the scale was rounded down; the quotient's three roundings move it by less than 2^-21 of itself.
    """
    z = z.reshape(*z.shape[:-1], z.shape[-1] // 16, 16)
    slack = np.asarray(slack)[..., None, None] * 1.1                           # [tokens, heads] -> of each block and channel
    s, top = e4m3_decode(scales), np.abs(z).max(-1)
    held = Q.held(codes, scales).reshape(z.shape)
    off = slack[..., 0] / 6 + 2.0 ** -22 * top
    want = np.minimum(top / 6, 448.0)
    assert np.all(np.abs(s - want) <= np.maximum(2.0 ** -4 * want, 2.0 ** -10) + off), float(np.abs(s - want).max())
    s = s[..., None]
    x = np.abs(z) / np.where(s > 0, s, 1)
    step = np.where(x < 2.01, 0.25, np.where(x < 4.01, 0.5, 1.0))
    tol = np.where(s > 0, step * s, np.abs(z)) + slack + 2.0 ** -20 * np.abs(z)
    err = np.abs(held - z)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())


def _store_case(shape, N, H, H_kv, page=16, rot=None, offset=0, interleaved=False, pairs=None, layout="nhd", strided=False, pad=0,
                dense=False, per_head=False, descales=True, base=0, rope=True, parts="qkv", seed=0, typed=False):
    rng = np.random.default_rng(seed)
    d_qk, d_v = SHAPES[shape]
    rot = d_qk if rot is None else rot
    rows = N + pad
    q, k, v = (torch.from_numpy(rng.standard_normal((rows, h, d))).to(torch.bfloat16) for h, d in ((H, d_qk), (H_kv, d_qk), (H_kv, d_v)))
    q64, k64, v64 = f64(q), f64(k), f64(v)
    if strided:                                                               # slices of one projection
        joint = torch.cat([t.flatten(1) for t in (q, k, v)], 1).cuda()
        q, k, v = (t.unflatten(1, (h, d)) for t, h, d in zip(torch.split(joint, [H * d_qk, H_kv * d_qk, H_kv * d_v], 1),
                                                           (H, H_kv, H_kv), (d_qk, d_qk, d_v)))
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    pages = -(-rows // page) + 2
    kc, vc, ks, vs = make_cache4(pages, page, H_kv, shape, layout, typed)
    before = [raw(t).clone() for t in (kc, vc, ks, vs)]
    slots = rng.permutation(pages * page)[:rows].astype(np.int64)
    padding = rng.permutation(rows)[:pad]                                     # padding rows anywhere
    slots[padding] = -1
    real = np.setdiff1d(np.arange(rows), padding)
    pairs = [rot // 2] if pairs is None else pairs
    positions = (base + rng.integers(0, 5000, (len(pairs), rows))).astype(np.int32)
    inv = (10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)
    ds = [f32((rng.random(H_kv if per_head else 1) + 1.0) / 400) if descales else None for _ in range(2)]
    spin = Rope(torch.from_numpy(inv).cuda(), axis_pairs=pairs, offset=offset, interleaved=interleaved) if rope else None
    q_out = poisoned((rows, H, d_qk), "bf16") if "q" in parts else None
    k_out, v_out = (poisoned((rows, H_kv, d), "bf16") if dense else None for d in (d_qk, d_v))
    pos = torch.from_numpy(positions).cuda()
    got = rope_paged_store(q if "q" in parts else None, k if "k" in parts else None, v if "k" in parts else None, kc, vc,
                           torch.from_numpy(slots).cuda(), (pos[0] if len(pairs) == 1 else pos) if rope else None, spin, k_descale=ds[0],
                           v_descale=ds[1], q_out=q_out, k_out=k_out, v_out=v_out, k_scales=ks, v_scales=vs)
    assert got is q_out and zyfa_check_errors() == 0
    turn = (lambda x: P.rope_rotate(x, positions, inv, pairs, offset, interleaved)) if rope else (lambda x: x)
    slack = lambda x: 2.0 ** -19 * np.abs(x).max(-1, keepdims=True)  # noqa: E731  rotation in fp32, as for the wider caches

    def dense_ok(out, x64):
        y = turn(x64)[real] if x64 is not v64 else x64[real]
        assert np.all(np.abs(f64(out)[real] - y) <= 2.0 ** -8 * np.abs(y) + 1.1 * slack(x64)[real])
        assert np.isnan(f64(out)[padding]).all()

    if "q" in parts:
        dense_ok(q_out, q64)
    after = [raw(t).cpu().numpy() for t in (kc, vc, ks, vs)]
    if "k" not in parts:
        assert all(np.array_equal(x, y.cpu().numpy()) for x, y in zip(after, before))
        return
    s = slots[real]
    y = turn(k64)
    d = [np.ones(H_kv) if x is None else np.broadcast_to(f64(x), (H_kv,)) for x in ds]
    at = lambda t: t[s // page, s % page]  # noqa: E731
    scale = d[0][None, :, None]
    # the reciprocal and the product round once each
    _near_held(at(after[0]), at(after[2]), y[real] / scale, (slack(k64)[real] / scale + 2.0 ** -22 * np.abs(y[real] / scale).max(-1, keepdims=True))[..., 0])
    for h in range(H_kv):                                                      # values: bit for bit
        codes, scales = Q.quantise(v64[real][:, h], np.float32(1.0) / np.float32(d[1][h]))
        assert np.array_equal(at(after[1])[:, h], codes) and np.array_equal(at(after[3])[:, h], scales)
        if not rope:
            codes, scales = Q.quantise(k64[real][:, h], np.float32(1.0) / np.float32(d[0][h]))
            assert np.array_equal(at(after[0])[:, h], codes) and np.array_equal(at(after[2])[:, h], scales)
    other = np.setdiff1d(np.arange(pages * page), s)                           # every other slot is as it was
    for x, w in zip(after, before):
        assert np.array_equal(x[other // page, other % page], w.cpu().numpy()[other // page, other % page])
    if dense:
        dense_ok(k_out, k64)
        dense_ok(v_out, v64)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", ["64", "128", "mla"])
def test_store_shapes(shape, interleaved):
    d = SHAPES[shape][0]
    _store_case(shape, 37, 6, 2, interleaved=interleaved, dense=True, pad=4, seed=1)
    _store_case(shape, 5, 3, 3, interleaved=interleaved, rot=32, offset=d - 32, seed=2, typed=True)
    _store_case(shape, 9, 4, 1, interleaved=interleaved, rot=48, offset=8, seed=3, strided=True)      # blocks that turn by half
    _store_case(shape, 9, 4, 2, interleaved=interleaved, rot=16, offset=24, seed=4, strided=True)
    _store_case(shape, 1, 1, 1, interleaved=interleaved, rot=16, offset=16, seed=5, page=1)
    _store_case(shape, 9, 2, 1, rope=False, seed=6)


@pytest.mark.parametrize("shape", ["64", "128", "mla"])
def test_store_many_tokens(shape):
    _store_case(shape, 3001, 5, 1, pad=7, seed=13, pairs=[8, 16], rot=48, offset=8)
    _store_case(shape, 9001, 2, 2, pad=100, seed=14, interleaved=True, dense=True, strided=True)
    _store_case(shape, 20011, 1, 1, pad=3, seed=15, rot=64)


@pytest.mark.parametrize("pairs", [[16, 24, 24], [0, 64], [1, 2, 3, 58], [64, 0, 0]])
def test_store_axes(pairs):
    _store_case("128", 23, 8, 2, pairs=pairs, pad=2, strided=True, seed=5)
    _store_case("128", 23, 8, 2, pairs=pairs, interleaved=True, seed=6)


@pytest.mark.parametrize("layout", ["nhd", "hnd", "joint", "row"])
@pytest.mark.parametrize("page", [1, 7, 48])
def test_store_layouts(layout, page):
    _store_case("64", 50, 8, 4, page=page, layout=layout, dense=True, seed=7)
    _store_case("mla", 50, 4, 4, page=page, layout=layout, rot=64, offset=128, per_head=True, seed=8, typed=True)


@pytest.mark.parametrize("base", [1_000_000, 2_147_000_000, -2_147_483_648])
def test_store_far_positions(base):
    _store_case("128", 31, 4, 2, base=base, seed=9)


def test_store_parts():
    _store_case("128", 11, 4, 2, parts="q", seed=10)
    _store_case("128", 11, 4, 2, parts="kv", seed=11, dense=True)
    _store_case("128", 11, 4, 2, descales=False, seed=13)
    _store_case("128", 11, 20, 20, per_head=True, seed=14)
    _store_case("64", 3, 71, 71, seed=15)
    _store_case("128", 700, 8, 2, seed=16, pad=60, dense=True)
    _store_case("64", 0, 4, 2, seed=17, pad=3)
    _store_case("mla", 2500, 3, 1, rot=64, offset=128, seed=18, pad=3)


def test_store_blocks_at_the_edges_of_the_format():
    # zeros, the smallest and largest scales, infinities and NaN, each in blocks of their own and beside finite ones
    d = 64
    rows = np.zeros((9, 1, d), dtype=np.float32)
    rows[1] = 2.0 ** -133                                                       # the smallest bf16 value
    rows[2, 0, :16], rows[2, 0, 16:32] = 6 * 2.0 ** -10, 6.1 * 2.0 ** -10       # a scale on the tie below 2^-9, and above it
    rows[3] = 2688.0                                                            # the largest value held
    rows[4] = 3e38
    rows[5, 0, 3], rows[5, 0, 20] = np.inf, -np.inf
    rows[6, 0, 17] = np.nan
    rows[7, 0, :16] = [-6, 6, -4, 4, -3, 3, -2, 2, -1.5, 1.5, -1, 1, -0.5, 0.5, -0.25, 0.25]
    rows[8, 0, ::7] = -1.0
    x = torch.from_numpy(rows).to(torch.bfloat16).cuda()
    kc, vc, ks, vs = make_cache4(2, 8, 1, "64")
    rope_paged_store(None, x, x, kc, vc, torch.arange(9, device="cuda"), k_scales=ks, v_scales=vs)
    codes, scales = Q.quantise(f64(x), 1.0)
    for c, s in ((kc, ks), (vc, vs)):
        c, s = (raw(t).flatten(0, 1)[:9].cpu().numpy() for t in (c, s))
        nan = np.isnan(e4m3_decode(scales))
        assert np.array_equal(s & 0x7F, scales & 0x7F) and nan.sum() == 1
        assert np.array_equal(np.where(nan[..., None], 0, c.reshape(*s.shape, 8)), np.where(nan[..., None], 0, codes.reshape(*s.shape, 8)))
    assert zyfa_check_errors() == 0


def test_store_keeps_slots_outside_untouched():
    kc, vc, ks, vs = make_cache4(2, 4, 1, "64")
    x = torch.full((3, 1, 64), 6.0, dtype=torch.bfloat16, device="cuda")
    q = rope_paged_store(x, -x, x, kc, vc, torch.tensor([3, 8, 1 << 40], device="cuda"), k_scales=ks, v_scales=vs)
    assert zyfa_check_errors() == BAD_PAGE and zyfa_check_errors() == 0
    assert torch.equal(q, x)
    k, v = held_of(kc, ks).reshape(8, 64), held_of(vc, vs).reshape(8, 64)
    assert (k[3] == -6).all() and (v[3] == 6).all() and np.isnan(np.delete(k, 3, 0)).all() and np.isnan(np.delete(v, 3, 0)).all()


# ------------------------------------------------------------------------------------------------
# reading back

def _read_case(kind, out, shape, H_kv, runs, page=16, layout="nhd", pad=0, per_head=0, descales=True, starts=True, seed=0, width=None):
    """runs: (first token, number of tokens) of each request."""
    rng = np.random.default_rng(seed)
    d_qk, d_v = SHAPES[shape]
    B = len(runs)
    table, pages = random_table([f + n for f, n in runs], page, rng, width)
    if kind == "e2m1":
        caches = make_cache4(pages, page, H_kv, shape, layout)
    else:
        caches = (*make_cache(pages, page, H_kv, shape, kind, layout), None, None)
    cu = np.cumsum([0] + [n for _, n in runs])
    N = int(cu[-1])
    rows = []
    for cache, scales, d in ((caches[0], caches[2], d_qk), (caches[1], caches[3], d_v)):
        slots = np.concatenate([table[b, t // page].astype(np.int64) * page + t % page for b, (f, n) in enumerate(runs) for t in [np.arange(f, f + n)]]
                               + [np.zeros(0, dtype=np.int64)])
        if kind == "e2m1":
            codes, sc = random_codes((N, H_kv, d), rng)
            fill4(cache, scales, slots, codes, sc)
            rows.append(Q.held(codes, sc))
        else:
            x = random_values((N, H_kv, d), kind, rng, 1.0)
            bits(cache)[slots // page, slots % page] = bits(x)
            rows.append(f64(x))
    many = {0: 1, 1: B * H_kv, 3: H_kv}[per_head]
    about = 1 / 128 if kind == "e2m1" else 1 / 64
    ds = [f32((rng.random(many) + 0.5) * about) if descales and kind != "bf16" else None for _ in range(2)]
    os_ = [f32((rng.random(H_kv if per_head else 1) + 1.0) / 64) if descales and out == "fp8" else None for _ in range(2)]
    outs = [poisoned((N + pad, H_kv, d), out) for d in (d_qk, d_v)]
    got = paged_read(caches[0], caches[1], torch.from_numpy(table).cuda(), i32(cu), starts=i32([f for f, _ in runs]) if starts else None,
                     k_scales=caches[2], v_scales=caches[3], k_descale=ds[0], v_descale=ds[1], k_out_descale=os_[0], v_out_descale=os_[1],
                     k_out=outs[0], v_out=outs[1])
    assert got[0] is outs[0] and got[1] is outs[1] and zyfa_check_errors() == 0
    request = np.repeat(np.arange(B), [n for _, n in runs])
    f = np.float32
    for t, x, d, o in zip(outs, rows, ds, os_):
        factor = np.ones((N, H_kv), dtype=f)
        if d is not None:
            dn = f64(d).astype(f)
            factor = factor * (dn.reshape(B, H_kv)[request] if per_head == 1 else dn.reshape(1, -1))
        if o is not None:
            factor = factor * (f(1.0) / f64(o).astype(f)).reshape(1, -1)
        y = (x.astype(f) * factor[..., None].astype(f)).astype(f)              # the definition's fp32 operations, bit for bit
        if out == "fp8":
            want = torch.from_numpy(e4m3_encode_rne_satfinite(y.astype(np.float64)))
        else:
            want = torch.from_numpy(y).to(torch.bfloat16).view(torch.int16)
        assert torch.equal(bits(t)[:N].cpu(), want)
        assert np.isnan(f64(t)[N:]).all()                                      # rows behind the last request are as they were


RAGGED = [(0, 5), (3, 0), (0, 33), (17, 1), (40, 90), (0, 0), (100, 16)]


@pytest.mark.parametrize("shape", ["64", "128", "mla"])
@pytest.mark.parametrize("out", ["bf16", "fp8"])
@pytest.mark.parametrize("kind", ["e2m1", "fp8", "bf16"])
def test_read_shapes(kind, out, shape):
    _read_case(kind, out, shape, 3, RAGGED, pad=6, seed=1)
    _read_case(kind, out, shape, 1, [(0, 1)], page=1, seed=2, starts=False)
    _read_case(kind, out, shape, 8, [(0, 700)], page=16, seed=3, starts=False, per_head=3)
    _read_case(kind, out, shape, 2, RAGGED, page=7, per_head=1, seed=4, pad=1, width=40)
    _read_case(kind, out, shape, 5, [(9, 64)], page=64, descales=False, seed=5)


@pytest.mark.parametrize("kind", ["e2m1", "fp8", "bf16"])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "joint"])
def test_read_layouts(kind, layout):
    _read_case(kind, "bf16", "128", 4, RAGGED, page=16, layout=layout, seed=6)
    _read_case(kind, "fp8", "mla", 3, RAGGED, page=5, layout=layout, seed=7)
    if kind == "e2m1":
        _read_case(kind, "bf16", "64", 3, RAGGED, page=8, layout="row", seed=8)


@pytest.mark.parametrize("B", [255, 256, 257, 1000, 3000])
def test_read_many_requests(B):
    # beyond a block's threads run starts are sampled; many requests have no tokens
    rng = np.random.default_rng(B)
    runs = [(int(a), int(n)) for a, n in zip(rng.integers(0, 30, B), rng.integers(0, 6, B) * (rng.random(B) < 0.5))]
    _read_case("e2m1", "bf16", "64", 1, runs, page=8, seed=B, pad=3)
    _read_case("e2m1", "fp8", "mla", 2, runs, page=8, seed=B + 1)


def test_read_one_long_run():
    _read_case("e2m1", "bf16", "128", 2, [(3, 20011)], page=48, seed=1)
    _read_case("e2m1", "fp8", "64", 1, [(0, 40000)], page=64, seed=2)
    _read_case("fp8", "bf16", "mla", 16, [(0, 1500), (700, 800)], page=32, seed=3)


def test_read_makes_its_rows():
    rng = np.random.default_rng(0)
    kc, vc = random_values((3, 4, 2, 64), "bf16", rng), random_values((3, 4, 2, 64), "bf16", rng)
    table, cu = i32([[2, 0], [1, -1]]), i32([0, 6, 9])
    k, v = paged_read(kc, vc, table, cu, 9)
    want = torch.cat([kc[2], kc[0][:2], kc[1][:3]])
    assert torch.equal(k, want) and k.dtype == torch.bfloat16 and v.shape == (9, 2, 64) and zyfa_check_errors() == 0
    k8, _ = paged_read(kc, vc, table, cu, 9, dtype=E4M3)
    assert torch.equal(bits(k8), bits(want.float().clamp(-448, 448).to(E4M3)))
    assert paged_read(kc, vc, table, cu, 0)[0].shape == (0, 2, 64)
    assert paged_read(kc, vc, table[:0], cu[:1], 5)[0].shape == (5, 2, 64)
    few, _ = paged_read(kc, vc, table, cu, 4)                                   # rows for some of the tokens
    assert torch.equal(few, want[:4])


def test_read_reports_tokens_without_a_page():
    rng = np.random.default_rng(0)
    kc, vc = random_values((3, 4, 2, 64), "bf16", rng), random_values((3, 4, 2, 64), "bf16", rng)
    for table, starts, zero in ((i32([[2, 3]]), None, slice(4, 8)), (i32([[2, -1]]), None, slice(4, 8)), (i32([[2, 1]]), i32([4]), slice(4, 8)),
                                (i32([[2, 1]]), i32([-3]), slice(0, 3)), (i32([[2, 1]]), i32([2_000_000_000]), slice(0, 8)),
                                (torch.empty((1, 0), dtype=torch.int32, device="cuda"), None, slice(0, 8))):
        k, v = paged_read(kc, vc, table, i32([0, 8]), 8, starts=starts)
        assert zyfa_check_errors() == BAD_PAGE and zyfa_check_errors() == 0
        at = np.zeros(8, dtype=bool)
        at[zero] = True
        assert (f64(k)[at] == 0).all() and (f64(v)[at] == 0).all() and (f64(k)[~at] != 0).any(-1).all()


def test_read_run_starts_that_do_not_begin_with_row_0():
    rng = np.random.default_rng(0)
    kc, vc = random_values((3, 4, 2, 64), "bf16", rng), random_values((3, 4, 2, 64), "bf16", rng)
    k, v = poisoned((9, 2, 64), "bf16"), poisoned((9, 2, 64), "bf16")
    paged_read(kc, vc, i32([[2, 0], [1, 1]]), i32([2, 5, 5]), k_out=k, v_out=v)
    assert torch.equal(k[2:5], kc[2][:3]) and np.isnan(f64(k)[:2]).all() and np.isnan(f64(v)[5:]).all() and zyfa_check_errors() == 0


def test_read_nan_scales_and_codes():
    kc, vc, ks, vs = make_cache4(1, 4, 1, "64")
    fill4(kc, ks, [0], np.full((1, 1, 32), 0x72, dtype=np.uint8), np.array([[[0x38, 0x7F, 0x38, 0xB8]]], dtype=np.uint8))
    fill4(vc, vs, [0], np.full((1, 1, 32), 0x00, dtype=np.uint8), np.array([[[0x38, 0x7F, 0x7E, 0x00]]], dtype=np.uint8))
    k, v = paged_read(kc, vc, i32([[0]]), i32([0, 1]), 1, k_scales=ks, v_scales=vs)
    k8, _ = paged_read(kc, vc, i32([[0]]), i32([0, 1]), 1, k_scales=ks, v_scales=vs, dtype=E4M3)
    x = np.tile([1.0, 6.0], 32)
    x[16:32] = np.nan
    x[48:] *= -1                                                                # a scale's sign counts
    np.testing.assert_array_equal(f64(k)[0, 0], x)
    np.testing.assert_array_equal(f64(k8)[0, 0], x)
    np.testing.assert_array_equal(f64(v)[0, 0], np.where(np.isnan(x), x, 0))


# ------------------------------------------------------------------------------------------------
# single-token attention

def _attend(q, caches, table, lens, scale=None, lse=True, ds=(None, None), **kw):
    return paged_decode_attn(q, caches[0], caches[1], table, lens, scale, k_scales=caches[2], v_scales=caches[3], k_descale=ds[0], v_descale=ds[1],
                             return_lse=lse, **kw)


def _decode_case(shape, lens, H, H_kv, page=16, layout="nhd", per_head=False, scale=None, seed=0, loud=1.0, width=None, strided_q=False, lse=True,
                 typed=False):
    rng = np.random.default_rng(seed)
    d_qk, d_v = SHAPES[shape]
    B = len(lens)
    table, pages = random_table(lens, page, rng, width)
    caches = make_cache4(pages, page, H_kv, shape, layout, typed)
    q = random_values((B, H, d_qk), "bf16", rng, loud)
    ks, vs = [], []
    for b, n in enumerate(lens):
        t = np.arange(n)
        slots = table[b, t // page].astype(np.int64) * page + t % page
        for to, (cache, scales), d, about in ((ks, (caches[0], caches[2]), d_qk, 128.0 * loud), (vs, (caches[1], caches[3]), d_v, 128.0)):
            codes, sc = random_codes((n, H_kv, d), rng, about)
            fill4(cache, scales, slots, codes, sc)
            to.append(Q.held(codes, sc))
    ds = [f32((rng.random(B * H_kv if per_head else 1) + 0.5) / 128) for _ in range(2)]
    if strided_q:
        wide = poisoned((B, H + 3, d_qk), "bf16")
        wide[:, :H] = q
        q = wide[:, :H]
    got = _attend(q, caches, torch.from_numpy(table).cuda(), i32(lens), scale, lse, ds)
    assert zyfa_check_errors() == 0
    out, got_lse = got if lse else (got, None)
    out, sc = f64(out), 1.0 / math.sqrt(d_qk) if scale is None else scale
    f = [np.broadcast_to(f64(d).reshape(-1, H_kv) if per_head else f64(d), (B, H_kv)) for d in ds]
    for b in range(B):
        q64 = f64(q[b])
        for h in range(H):
            hk = h // (H // H_kv)
            if lens[b] <= 0:
                assert (out[b, h] == 0).all() and (not lse or float(got_lse[b, h]) == -math.inf)
                continue
            kr, v64 = ks[b][:, hk] * f[0][b, hk], vs[b][:, hk]
            ref, ref_lse, w = P.decode_attention(q64[h], kr, v64 * f[1][b, hk], sc)
            # as for an e4m3 cache (fp16 weights); a query's rounding below 2^-28 of its largest is 2^-39 of that
            tol, lse_tol = decode_tolerance(q64[h], kr, v64, sc, f[1][b, hk], ref, w, "fp8")
            more = d_qk * 2.0 ** -39 * np.abs(q64[h]).max() * np.abs(kr).max() * sc
            assert np.all(np.abs(out[b, h] - ref) <= tol + 2 * more * (w @ np.abs(v64) * f[1][b, hk])), (b, h, float((np.abs(out[b, h] - ref) / tol).max()))
            if lse:
                assert abs(float(got_lse[b, h]) - ref_lse) <= lse_tol + more + 2.0 ** -23 * abs(ref_lse), (b, h, float(got_lse[b, h]), ref_lse)


@pytest.mark.parametrize("shape", ["64", "128", "mla"])
def test_decode_lengths(shape):
    lens = [0, 1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 127, 128, 129, 191, 192, 255, 256, 257, 300, 0, 511, 513]
    _decode_case(shape, lens, 4, 2, seed=1)
    _decode_case(shape, lens, 3, 3, page=7, seed=2, width=80)
    _decode_case(shape, lens, 8, 8, page=64, seed=3, typed=True)


@pytest.mark.parametrize("H,H_kv", [(1, 1), (2, 1), (3, 1), (5, 1), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 1), (128, 1), (14, 2), (21, 7)])
def test_decode_groups(H, H_kv):
    _decode_case("128", [77, 1, 300], H, H_kv, seed=H, per_head=True)
    _decode_case("64", [1000], H, H_kv, seed=H + 1)
    _decode_case("mla", [70, 140], H, H_kv, seed=H + 2)


@pytest.mark.parametrize("H,H_kv", [(10, 10), (20, 10), (11, 11), (12, 6), (32, 32), (24, 8), (32, 2), (96, 4), (6, 3), (4, 4)])
def test_decode_many_kv_heads(H, H_kv):
    # heads that do and do not fill the blocks that take them side by side
    _decode_case("64", [37, 300], H, H_kv, seed=H, per_head=True, page=32)
    _decode_case("128", [290, 3], H, H_kv, seed=H + 1, page=8)
    _decode_case("mla", [64, 129], H, H_kv, seed=H + 2, page=64)


@pytest.mark.parametrize("B,page", [(128, 16), (129, 16), (200, 7), (700, 16), (1100, 24)])
def test_decode_many_requests(B, page):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 90, B)
    lens[rng.permutation(B)[: B // 4]] = 0
    lens[3], lens[B - 1] = 800, 5
    _decode_case("64", lens.tolist(), 2, 1, seed=B, page=page)


@pytest.mark.parametrize("shape", ["64", "128", "mla"])
@pytest.mark.parametrize("B,H,H_kv", [(1, 8, 2), (7, 6, 3), (40, 20, 2), (300, 5, 5)])
def test_decode_small_tables(shape, B, H, H_kv):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 65, B)
    lens[:: 5] = 0
    lens[B // 2] = 64
    _decode_case(shape, lens.tolist(), H, H_kv, seed=B, page=16, width=4, per_head=True)
    _decode_case(shape, [0] * B, H, H_kv, seed=B, page=8, width=2)
    _decode_case(shape, [130] * min(B, 100), H, H_kv, seed=B + 1, page=32)


@pytest.mark.parametrize("layout", ["nhd", "hnd", "joint", "row"])
@pytest.mark.parametrize("page", [1, 7, 8, 16, 48, 256])
def test_decode_layouts(layout, page):
    _decode_case("128", [100, 513, 1], 8, 4, page=page, layout=layout, seed=5)
    _decode_case("64", [100, 213, 1], 12, 6, page=page, layout=layout, seed=6)
    _decode_case("64", [140, 33], 6, 3, page=page, layout=layout, seed=7)
    _decode_case("mla", [100, 213, 1], 4, 4, page=page, layout=layout, seed=8, strided_q=True)


def test_decode_long_contexts():
    _decode_case("128", [20000], 8, 2, page=64, seed=1)
    _decode_case("64", [9001, 3, 12000], 4, 4, page=16, seed=2)
    _decode_case("mla", [7777, 5000], 4, 4, page=32, seed=3)
    _decode_case("128", [6000, 1, 2500, 900], 64, 4, page=32, seed=4, per_head=True)


def test_decode_scales_and_loud_scores():
    _decode_case("128", [300, 1], 8, 2, scale=0.5, seed=1)
    _decode_case("64", [500], 4, 1, scale=2.0, loud=4.0, seed=2)               # one key takes nearly all the weight
    _decode_case("mla", [500], 4, 2, scale=1e-6, seed=3, lse=False)


@pytest.mark.parametrize("exponent", [-130, -100, -60, -20, 20, 60, 100])
def test_decode_queries_of_any_magnitude(exponent):
    # a power of two in the queries and its inverse in the scale change nothing but the last bits that fp32 has below its range
    rng = np.random.default_rng(3)
    caches = make_cache4(8, 16, 2, "128")
    for c, s in ((caches[0], caches[2]), (caches[1], caches[3])):
        codes, sc = random_codes((128, 2, 128), rng, 2.0)
        fill4(c, s, np.arange(128), codes, sc)
    table, lens = torch.arange(8, dtype=torch.int32, device="cuda")[None], i32([120])
    q = random_values((1, 8, 128), "bf16", rng)
    want = _attend(q, caches, table, lens, 0.1, lse=False)
    if exponent <= -100:
        got = _attend(q * 2.0 ** exponent, caches, table, lens, 0.1 * 2.0 ** 100, lse=False, ds=(f32([2.0 ** (-100 - exponent)]), None))
    else:
        got = _attend(q * 2.0 ** exponent, caches, table, lens, 0.1 * 2.0 ** -exponent, lse=False)
    if exponent == -130:                                                       # such queries have few bits in bf16 themselves
        q = (q * 2.0 ** exponent) * 2.0 ** 100 * 2.0 ** 30
        want = _attend(q, caches, table, lens, 0.1, lse=False)
    assert torch.equal(got, want)


def test_decode_rows_with_nan_and_infinities():
    rng = np.random.default_rng(5)
    caches = make_cache4(8, 16, 1, "64")
    for c, s in ((caches[0], caches[2]), (caches[1], caches[3])):
        codes, sc = random_codes((128, 1, 64), rng, 2.0)
        fill4(c, s, np.arange(128), codes, sc)
    table, lens = torch.arange(8, dtype=torch.int32, device="cuda")[None], i32([100])
    q = random_values((1, 3, 64), "bf16", rng)
    clean, clean_lse = _attend(q, caches, table, lens)
    bad = q.clone()
    bad[0, 1, 7] = math.nan
    out, lse = _attend(bad, caches, table, lens)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    assert torch.equal(out[0, [0, 2]], clean[0, [0, 2]]) and torch.equal(lse[0, [0, 2]], clean_lse[0, [0, 2]])
    ks, vs = caches[2].clone(), caches[3].clone()
    raw(ks)[3, 5, 0, 1] = 0x7F                                                  # a key's scale: every row
    out, lse = _attend(q, (caches[0], caches[1], ks, vs), table, lens)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    raw(vs)[3, 5, 0, 1] = 0x7F                                                  # a value's: its 16 channels
    out, lse = _attend(q, (caches[0], caches[1], caches[2], vs), table, lens)
    assert torch.isnan(out[0, :, 16:32]).all() and torch.equal(out[0, :, :16], clean[0, :, :16]) and torch.equal(out[0, :, 32:], clean[0, :, 32:])
    assert torch.equal(lse, clean_lse) and zyfa_check_errors() == 0


@pytest.mark.parametrize("page,width", [(16, 8), (16, 400), (7, 40)])
def test_decode_leaves_out_bad_pages(page, width):
    rng = np.random.default_rng(6)
    pages = 12
    caches = make_cache4(pages, page, 2, "128")
    for c, s in ((caches[0], caches[2]), (caches[1], caches[3])):
        codes, sc = random_codes((pages * page, 2, 128), rng, 2.0)
        fill4(c, s, np.arange(pages * page), codes, sc)
    table = np.full((3, width), -1, dtype=np.int32)
    table[0, :5], table[1, :5], table[2, :3] = [1, 2, -1, 3, 4], [5, pages, 6, 1 << 30, 7], [-5, pages + 3, -1]
    lens = [5 * page - 2, 5 * page, 3 * page]
    q = random_values((3, 4, 128), "bf16", rng)
    out, lse = _attend(q, caches, torch.from_numpy(table).cuda(), i32(lens))
    assert zyfa_check_errors() == BAD_PAGE and zyfa_check_errors() == 0
    assert (f64(out[2]) == 0).all() and torch.isinf(lse[2]).all()
    k64, v64 = held_of(caches[0], caches[2]), held_of(caches[1], caches[3])
    for b in range(2):
        at = [(table[b, t // page], t % page) for t in range(lens[b]) if 0 <= table[b, t // page] < pages]
        p, o = np.array(at).T
        for h in range(4):
            ref, _, w = P.decode_attention(f64(q[b, h]), k64[p, o, h // 2], v64[p, o, h // 2], 128 ** -0.5)
            tol, _ = decode_tolerance(f64(q[b, h]), k64[p, o, h // 2], v64[p, o, h // 2], 128 ** -0.5, 1.0, ref, w, "fp8")
            assert np.all(np.abs(f64(out[b, h]) - ref) <= tol)


def test_decode_lengths_beyond_the_table_and_below_zero():
    rng = np.random.default_rng(7)
    caches = make_cache4(4, 16, 1, "64")
    for c, s in ((caches[0], caches[2]), (caches[1], caches[3])):
        codes, sc = random_codes((64, 1, 64), rng, 2.0)
        fill4(c, s, np.arange(64), codes, sc)
    q, table = random_values((3, 2, 64), "bf16", rng), i32([[0, 1, 2, 3]] * 3)
    a, la = _attend(q, caches, table, i32([64, 1_000_000, -3]))
    b, lb = _attend(q, caches, table, i32([64, 64, 0]))
    assert torch.equal(a, b) and torch.equal(la, lb) and (f64(a[2]) == 0).all() and zyfa_check_errors() == 0


def test_decode_repeats_bit_for_bit():
    rng = np.random.default_rng(8)
    caches = make_cache4(300, 16, 4, "128")
    for c, s in ((caches[0], caches[2]), (caches[1], caches[3])):
        codes, sc = random_codes((4800, 4, 128), rng, 2.0)
        fill4(c, s, np.arange(4800), codes, sc)
    q = random_values((3, 16, 128), "bf16", rng)
    table = torch.arange(300, dtype=torch.int32, device="cuda").reshape(3, 100)
    first = _attend(q, caches, table, i32([1600, 900, 1333]))
    for _ in range(20):
        again = _attend(q, caches, table, i32([1600, 900, 1333]))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


# ------------------------------------------------------------------------------------------------
# together

class _Server:
    """Requests in a 4-bit cache of the 128/128 shape, 64 of whose channels turn."""

    def __init__(self, B, H, H_kv, page, width, pages, seed=0):
        self.rng, self.page, self.H, self.H_kv = np.random.default_rng(seed), page, H, H_kv
        self.caches = make_cache4(pages, page, H_kv, "128")
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.free, self.cursor, self.lens = i32(self.rng.permutation(pages)), i32([0]), i32([0] * B)
        self.inv = (10000.0 ** (-np.arange(0, 64, 2) / 64)).astype(np.float32)
        self.rope = Rope(torch.from_numpy(self.inv).cuda(), offset=64)
        self.ds = (f32([1 / 400]), f32([1 / 300]))

    def tokens(self, n):
        return [random_values((n, h, 128), "bf16", self.rng) for h in (self.H, self.H_kv, self.H_kv)]

    def store(self, x, new, rows, dense=False):
        plan = paged_plan(self.lens, new, self.table, self.free, self.cursor, self.page, rows)
        kw = dict(k_out=torch.empty_like(x[1]), v_out=torch.empty_like(x[2])) if dense else {}
        q = rope_paged_store(*x, self.caches[0], self.caches[1], plan.slots, plan.positions, self.rope, k_scales=self.caches[2],
                             v_scales=self.caches[3], k_descale=self.ds[0], v_descale=self.ds[1], **kw)
        self.lens.copy_(plan.seq_lens)
        self.cursor.copy_(plan.cursor)
        return q, plan, kw

    def attend(self, q, **kw):
        return _attend(q, self.caches, self.table, self.lens, lse=False, ds=self.ds, **kw)

    def read(self, cu, rows, starts=None, **kw):
        return paged_read(self.caches[0], self.caches[1], self.table, cu, rows, starts=starts, k_scales=self.caches[2], v_scales=self.caches[3],
                          k_descale=self.ds[0], v_descale=self.ds[1], **kw)


def test_prompts_steps_and_prompts_behind_cached_tokens():
    """Prompts, then steps of one token, then a prompt chunk behind what is cached: the chunk's attention is the prefill on the tokens
    read back, whose last row the single-token attention gives as well."""
    s = _Server(3, 4, 2, 16, 20, 60, seed=4)
    prompts = [37, 0, 130]
    s.store(s.tokens(170), i32(prompts), 170)
    for _ in range(5):
        q, _, _ = s.store(s.tokens(3), i32([1] * 3), 3)
        out = s.attend(q)
        lens = s.lens.tolist()
        cu = i32(np.cumsum([0] + lens))
        k, v = s.read(cu, sum(lens))
        for b, n in enumerate(lens):
            at = slice(sum(lens[:b]), sum(lens[:b]) + n)
            for h in range(4):
                # what was read is off by its bf16 rounding, 2^-8 of each value: scores of size 1 and V by that, and the output's own
                ref, _, _ = P.decode_attention(f64(q[b, h]), f64(k[at, h // 2]), f64(v[at, h // 2]), 128 ** -0.5)
                size = np.linalg.norm(f64(v[at, h // 2]), axis=1).max()
                assert np.linalg.norm(f64(out[b, h]) - ref) <= 4 * 2.0 ** -8 * size
    new = [50, 3, 0]
    had = s.lens.tolist()
    q, plan, _ = s.store(s.tokens(53), i32(new), 53)
    lens = s.lens.tolist()
    assert lens == [a + n for a, n in zip(had, new)]
    cu = i32(np.cumsum([0] + lens))
    k, v = s.read(cu, sum(lens))
    first = 0
    for b in range(2):
        at = slice(sum(lens[:b]), sum(lens[:b]) + lens[b])
        rows = torch.zeros((lens[b], 4, 128), dtype=torch.bfloat16, device="cuda")
        rows[had[b]:] = q[first: first + new[b]]                                # the cached tokens' queries are not asked for
        out = flash_attn_func(rows[None], k[at][None], v[at][None])[0, -1]
        last = _attend(q[first + new[b] - 1: first + new[b]], s.caches, s.table[b: b + 1], s.lens[b: b + 1], lse=False, ds=s.ds)[0]
        # keys and values read back off by 2^-8, weights and output of the prefill by 2^-8, the output here by 2^-8
        assert float((out - last).float().norm() / last.float().norm()) <= 6 * 2.0 ** -8
        first += new[b]
    # the new tokens alone, read from where they begin
    some, _ = s.read(i32(np.cumsum([0] + new)), 53, starts=i32(had))
    assert torch.equal(some[:50], k[had[0]: had[0] + 50]) and torch.equal(some[50:], k[lens[0] + had[1]: lens[0] + had[1] + 3])
    assert zyfa_check_errors() == 0


def test_stored_values_are_near_what_was_given():
    """4 bits with a scale for 16 channels: a normal block is off by about a tenth (a code's step is 1/8 to 1/3 of it, over sqrt(12))."""
    s = _Server(1, 2, 2, 16, 80, 80, seed=5)
    x = s.tokens(1000)
    _, plan, dense = s.store(x, i32([1000]), 1000, dense=True)
    k, v = s.read(i32([0, 1000]), 1000)
    for got, want in ((k, dense["k_out"]), (v, dense["v_out"])):
        off = float((got - want).float().norm() / want.float().norm())
        assert 0.03 < off < 0.15, off
    assert torch.equal(dense["v_out"], x[2])


def test_captured_step_replays():
    """One captured token step (plan, store, decode and read with their buffers) replayed over many steps equals eager steps."""
    B, steps = 5, 40
    a, b = (_Server(B, 4, 1, 8, 60, 300, seed=2) for _ in range(2))
    xs = [a.tokens(7) for _ in range(steps)]
    static = [torch.zeros_like(t) for t in xs[0]]
    new, cu = i32([1] * B), i32(range(B + 1))

    def step(s, x):
        q, plan, _ = s.store(x, new, 7)
        k, v = s.read(cu, B, starts=s.lens - 1, dtype=E4M3, k_out_descale=s.ds[0], v_out_descale=s.ds[1])
        return s.attend(q[:B]), bits(k), bits(v)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(_Server(B, 4, 1, 8, 60, 300, seed=3), static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(b, static)
    for x in xs:
        want = step(a, x)
        for t, v in zip(static, x):
            t.copy_(v)
        graph.replay()
        assert all(torch.equal(p, w) for p, w in zip(got, want))
    assert all(torch.equal(raw(p), raw(w)) for p, w in zip(a.caches, b.caches)) and zyfa_check_errors() == 0 and a.lens.tolist() == [steps] * B


def test_two_captured_graphs_with_their_own_workspaces():
    rng = np.random.default_rng(7)
    caches = make_cache4(64, 64, 2, "128")
    for c, s in ((caches[0], caches[2]), (caches[1], caches[3])):
        codes, sc = random_codes((4096, 2, 128), rng, 2.0)
        fill4(c, s, np.arange(4096), codes, sc)
    qs = [random_values((2, 8, 128), "bf16", rng) for _ in range(2)]
    table, lens = torch.arange(64, dtype=torch.int32, device="cuda").reshape(2, 32).contiguous(), i32([2048, 1500])
    want = [_attend(q, caches, table, lens, lse=False) for q in qs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        ws = torch.empty(paged_decode_workspace_bytes(2, 8, 2, 128, 2048), dtype=torch.uint8, device="cuda")
        with torch.cuda.graph(g):
            outs.append(_attend(q, caches, table, lens, lse=False, workspace=ws))
        graphs.append((g, ws))
    streams = [torch.cuda.Stream() for _ in graphs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(50):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
