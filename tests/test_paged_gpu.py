"""GPU tests of the paged serving operators against their float64 oracle: page plan, rotation and store,
single-token attention, and a run of them together."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from _paged_util import (E4M3, SHAPES, bits, decode_tolerance, dtype_of, f64, fill_tokens, make_cache, poisoned,
                         random_table, random_values)
from fp8_causal_prefill_gb300 import (PagedPlan, Rope, flash_attn_func, paged_decode_attn, paged_decode_workspace_bytes, paged_plan,
                                      rope_paged_store, zyfa_check_errors)
from oracle import paged as P

pytestmark = pytest.mark.gpu

CAPACITY, BAD_PAGE = 6, 7


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------
# page plan

def _plan(cached, new, page, max_tokens=None, pool=None, cursor=0, width=None, seed=0, wider=0):
    rng = np.random.default_rng(seed)
    need = [-(-(max(0, c) + max(0, n)) // page) for c, n in zip(cached, new)]
    width = max(need, default=0) if width is None else width
    total = sum(need) if pool is None else pool
    free = rng.permutation(total + 5).astype(np.int32)[:total]
    table = rng.integers(0, 1000, (len(cached), width)).astype(np.int32)
    max_tokens = sum(max(0, n) for n in new) if max_tokens is None else max_tokens
    want = P.paged_plan(cached, new, table, free, cursor, page, max_tokens)
    big = torch.full((len(cached), width + wider), 123456, dtype=torch.int32, device="cuda")
    big[:, :width] = torch.from_numpy(table).cuda()
    got = paged_plan(i32(cached), i32(new), big[:, :width], torch.from_numpy(free).cuda(), i32([cursor]), page, max_tokens)
    st = zyfa_check_errors()
    np.testing.assert_array_equal(big[:, :width].cpu().numpy(), want[0])
    assert bool((big[:, width:] == 123456).all())
    for g, w, name in zip(got, want[1:], PagedPlan._fields):
        np.testing.assert_array_equal(g.cpu().numpy().reshape(-1), np.atleast_1d(w), err_msg=name)
    assert st == (CAPACITY if want[6] else 0)


@pytest.mark.parametrize("page", [1, 7, 16, 48, 64, 4096])
@pytest.mark.parametrize("B", [1, 2, 33, 300])
def test_plan_matches(B, page):
    rng = np.random.default_rng(B * 100 + page)
    cached = rng.integers(0, 3 * page + 40, B).tolist()
    new = rng.integers(0, 2 * page + 9, B).tolist()
    cached[0] = 0
    new[-1] = max(1, new[-1])
    _plan(cached, new, page, seed=B, wider=3)
    _plan(cached, new, page, seed=B + 1, max_tokens=sum(new) + 13, cursor=0, pool=sum(-(-(c + n) // page) for c, n in zip(cached, new)) + 4)
    _plan(cached, [1] * B, page, seed=B + 2)                                   # a decode step


@pytest.mark.parametrize("cached,new,page,kw", [
    ([0], [1], 16, {}), ([15], [1], 16, {}), ([16], [1], 16, {}), ([0], [0], 16, {}), ([5], [0], 16, {}),
    ([3, -4, 2], [-1, 3, 2], 4, {}),                                           # negative lengths count as 0
    ([0, 0, 0], [0, 0, 0], 8, dict(max_tokens=5)),
    ([10, 20], [30, 7], 8, dict(pool=3)),                                      # the pool runs out inside request 0
    ([10, 20], [30, 7], 8, dict(cursor=100, pool=9)),                          # the cursor lies behind the pool
    ([10, 20], [30, 7], 8, dict(width=4)),                                     # a length passes the table's width
    ([40, 20], [3, 7], 8, dict(width=4)),                                      # already past it
    ([10, 20], [30, 7], 8, dict(max_tokens=31)),                               # more tokens than rows
    ([10, 20], [30, 7], 8, dict(max_tokens=0)),
    ([1], [70001], 64, dict(max_tokens=70100)),                                # one long prompt
    ([100000] * 4, [25000, 1, 0, 3], 128, {}),
])
def test_plan_edges(cached, new, page, kw):
    _plan(cached, new, page, **kw)


@pytest.mark.parametrize("B", [1023, 1024, 1025, 5000])
def test_plan_many_requests(B):
    rng = np.random.default_rng(B)
    _plan(rng.integers(0, 500, B).tolist(), rng.integers(0, 4, B).tolist(), 16, max_tokens=4 * B)


def test_plan_without_requests():
    p = paged_plan(i32([]), i32([]), torch.zeros((0, 4), dtype=torch.int32, device="cuda"), i32([1, 2]), i32([1]), 16, 3)
    assert p.cu_tokens.tolist() == [0] and p.slots.tolist() == [-1] * 3 and p.positions.tolist() == [0] * 3
    assert p.cursor.tolist() == [1] and zyfa_check_errors() == 0


def test_plan_updates_its_cursor_in_place():
    free, cursor = i32([4, 3, 2, 1]), i32([0])
    table, lens = torch.zeros((1, 4), dtype=torch.int32, device="cuda"), i32([0])
    for step in range(3):
        out = PagedPlan(i32([0]), i32([0, 0]), i32([0] * 5), torch.zeros(5, dtype=torch.int64, device="cuda"), cursor)
        p = paged_plan(lens, i32([5]), table, free, cursor, 4, 5, out=out)
        lens = p.seq_lens.clone()
    assert cursor.tolist() == [4] and table.tolist() == [[4, 3, 2, 1]] and lens.tolist() == [15] and zyfa_check_errors() == 0
    assert p.slots.tolist() == [2 * 4 + 2, 2 * 4 + 3, 4, 5, 6] and p.positions.tolist() == [10, 11, 12, 13, 14]


def test_plan_in_place_cursor_with_many_rows():
    # the rows take many blocks, all of which read the cursor before it moves
    rng = np.random.default_rng(3)
    B, page = 40, 16
    cached, new = rng.integers(0, 100, B), rng.integers(0, 900, B)
    need = int(sum(-(-(c + n) // page) for c, n in zip(cached, new)))
    free = rng.permutation(need + 9).astype(np.int32)
    table = np.full((B, 64), 5, dtype=np.int32)
    rows = int(new.sum()) + 31
    want = P.paged_plan(cached, new, table, free, 7, page, rows)
    t, cursor = torch.from_numpy(table).cuda(), i32([7])
    z = lambda n, d=torch.int32: torch.full((n,), -9, dtype=d, device="cuda")  # noqa: E731
    out = PagedPlan(z(B), z(B + 1), z(rows), z(rows, torch.int64), cursor)
    assert paged_plan(i32(cached), i32(new), t, torch.from_numpy(free).cuda(), cursor, page, rows, out=out) is out
    np.testing.assert_array_equal(t.cpu().numpy(), want[0])
    for g, w in zip(out, want[1:]):
        np.testing.assert_array_equal(g.cpu().numpy().reshape(-1), np.atleast_1d(w))
    assert zyfa_check_errors() == (CAPACITY if want[6] else 0)


# ------------------------------------------------------------------------------------------------
# rotation and store

def _store_case(kind, shape, N, H, H_kv, page=16, rot=None, offset=0, interleaved=False, pairs=None, layout="nhd", strided=False,
                pad=0, dense=False, per_head=False, descales=True, base=0, rope=True, parts="qkv", seed=0):
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
    kc, vc = make_cache(pages, page, H_kv, shape, kind, layout)
    slots = rng.permutation(pages * page)[:rows].astype(np.int64)
    padding = rng.permutation(rows)[:pad]                                     # padding rows anywhere
    slots[padding] = -1
    real = np.setdiff1d(np.arange(rows), padding)
    pairs = [rot // 2] if pairs is None else pairs
    positions = (base + rng.integers(0, 5000, (len(pairs), rows))).astype(np.int32)
    inv = (10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)
    ds = [None] * 3
    if kind == "fp8" and descales:
        ds = [torch.from_numpy((rng.random(H_kv if per_head else 1) + 1.0) / 64).float().cuda() for _ in range(3)]
    spin = Rope(torch.from_numpy(inv).cuda(), axis_pairs=pairs, offset=offset, interleaved=interleaved) if rope else None
    q_out = poisoned((rows, H, d_qk), kind) if "q" in parts else None
    k_out = poisoned((rows, H_kv, d_qk), kind) if dense else None
    v_out = poisoned((rows, H_kv, d_v), kind) if dense else None
    pos = torch.from_numpy(positions).cuda()
    rope_paged_store(q if "q" in parts else None, k if "k" in parts else None, v if "k" in parts else None, kc, vc,
                     torch.from_numpy(slots).cuda(), (pos[0] if len(pairs) == 1 else pos) if rope else None, spin, q_descale=ds[0],
                     k_descale=ds[1], v_descale=ds[2], q_out=q_out, k_out=k_out, v_out=v_out)
    assert zyfa_check_errors() == 0
    turn = (lambda x: P.rope_rotate(x, positions, inv, pairs, offset, interleaved)) if rope else (lambda x: x)
    group = H // H_kv

    def check(got, x64, y64, d, heads_per):
        """Against y64 / descale: fp32 rotation of u, w (sin, cos and products within 2^-20 of |u| + |w|), one rounding."""
        f = 1.0 if d is None else f64(d).repeat(heads_per)[:, None] if d.numel() > 1 else float(d.item())
        z = y64 / f
        # |u| + |w| <= 2 max over the row; the descale's reciprocal and product round once each
        slack = 2.0 ** -19 * np.abs(x64).max(-1, keepdims=True) / f + 2.0 ** -22 * np.abs(z)
        if kind == "fp8":
            assert np.all(np.abs(z) < 440)
            tol = 2.0 ** -4 * np.abs(z) + 2.0 ** -10 + 1.1 * slack
        else:
            tol = 2.0 ** -8 * np.abs(z) + 1.1 * slack
        err = np.abs(got - z)
        assert np.all(err <= tol), float((err / tol).max())

    if "q" in parts:
        check(f64(q_out)[real], q64[real], turn(q64)[real], ds[0], group)
        assert np.isnan(f64(q_out)[padding]).all()
    if "k" not in parts:
        assert np.isnan(f64(kc)).all() and np.isnan(f64(vc)).all()
        return
    y = turn(k64)
    s = slots[real]
    check(f64(kc)[s // page, s % page], k64[real], y[real], ds[1], 1)
    check(f64(vc)[s // page, s % page], v64[real], v64[real], ds[2], 1)
    other = np.setdiff1d(np.arange(pages * page), s)                           # every other slot is as it was
    assert np.isnan(f64(kc)[other // page, other % page]).all() and np.isnan(f64(vc)[other // page, other % page]).all()
    if dense:
        assert torch.equal(bits(k_out)[real], bits(kc)[s // page, s % page]) and torch.equal(bits(v_out)[real], bits(vc)[s // page, s % page])
        assert np.isnan(f64(k_out)[padding]).all() and np.isnan(f64(v_out)[padding]).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", ["64", "128", "mla"])
@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_store_shapes(kind, shape, interleaved):
    d = SHAPES[shape][0]
    _store_case(kind, shape, 37, 6, 2, interleaved=interleaved, dense=True, pad=4, seed=1)
    _store_case(kind, shape, 5, 3, 3, interleaved=interleaved, rot=32, offset=d - 32, seed=2)
    _store_case(kind, shape, 9, 4, 1, interleaved=interleaved, rot=48, offset=8, seed=3, strided=True)
    _store_case(kind, shape, 1, 1, 1, interleaved=interleaved, rot=16, offset=16, seed=4, page=1)


@pytest.mark.parametrize("shape", ["64", "128", "mla"])
@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_store_many_tokens(kind, shape):
    # several tokens per block, up to 32 where heads are few; the last block has fewer, and pairs do not divide the threads
    _store_case(kind, shape, 3001, 5, 1, pad=7, seed=13, pairs=[8, 16], rot=48, offset=8)
    _store_case(kind, shape, 9001, 2, 2, pad=100, seed=14, interleaved=True, dense=True, strided=True)
    _store_case(kind, shape, 20011, 1, 1, pad=3, seed=15, rot=64)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("pairs", [[16, 24, 24], [0, 64], [1, 2, 3, 58], [64, 0, 0]])
def test_store_axes(kind, pairs):
    _store_case(kind, "128", 23, 8, 2, pairs=pairs, pad=2, strided=True, seed=5)
    _store_case(kind, "128", 23, 8, 2, pairs=pairs, interleaved=True, seed=6)


@pytest.mark.parametrize("layout", ["nhd", "hnd", "joint"])
@pytest.mark.parametrize("page", [1, 7, 48])
def test_store_layouts(layout, page):
    _store_case("bf16", "64", 50, 8, 4, page=page, layout=layout, dense=True, seed=7)
    _store_case("fp8", "mla", 50, 4, 4, page=page, layout=layout, rot=64, offset=128, per_head=True, seed=8)


@pytest.mark.parametrize("base", [1_000_000, 2_147_000_000, -2_147_483_648])
def test_store_far_positions(base):
    _store_case("bf16", "128", 31, 4, 2, base=base, seed=9)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_store_parts(kind):
    _store_case(kind, "128", 11, 4, 2, parts="q", seed=10)
    _store_case(kind, "128", 11, 4, 2, parts="kv", seed=11, dense=True)
    _store_case(kind, "128", 11, 4, 2, rope=False, seed=12)
    _store_case(kind, "128", 11, 4, 2, descales=False, seed=13)
    _store_case(kind, "128", 11, 20, 20, per_head=True, seed=14)
    _store_case(kind, "64", 3, 71, 71, seed=15)
    _store_case(kind, "128", 700, 8, 2, seed=16, pad=60, dense=True)
    _store_case(kind, "64", 0, 4, 2, seed=17, pad=3)
    _store_case(kind, "mla", 2500, 3, 1, rot=64, offset=128, seed=18, pad=3)    # several tokens per block, a ragged last one
    _store_case(kind, "128", 5000, 2, 2, seed=19, strided=True, dense=True)


def test_store_without_tokens_or_rotation():
    kc, vc = make_cache(2, 4, 2, "64", "bf16")
    empty = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    assert rope_paged_store(empty, empty, empty, kc, vc, slots).shape == (0, 2, 64)
    assert rope_paged_store(None, empty, empty, kc, vc, slots) is None
    x = random_values((3, 2, 64), "bf16", np.random.default_rng(1))
    none = Rope(torch.empty(0, device="cuda"))
    at = torch.tensor([1, 5, 2], device="cuda")
    assert torch.equal(rope_paged_store(x, x, x, kc, vc, at, i32([9, 9, 9]), none), x)
    assert torch.equal(kc.flatten(0, 1)[at], x) and torch.equal(vc.flatten(0, 1)[at], x)


def test_store_tensor_refusals():
    kc, vc = make_cache(2, 4, 2, "64", "bf16")
    x, slots, pos = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda"), i32([0, 1, 2])
    rope = Rope(torch.ones(32, device="cuda"))
    for bad in (dict(q=x.float()), dict(q=x[:2]), dict(k=x[:, :1]), dict(v=None), dict(q=None, k=None, v=None), dict(slots=slots.int()),
                dict(slots=slots[:2]), dict(slots=slots.cpu()), dict(pos=pos.long()), dict(pos=pos[:2]), dict(pos=pos[None].repeat(2, 1)),
                dict(pos=None), dict(q_out=x), dict(q_out=x.to(E4M3)), dict(k_out=x[:2]), dict(q=x.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(q=x[..., ::2]), dict(kc=kc.float()), dict(kc=kc[:1]), dict(rope=Rope(torch.ones(32, device="cuda"), axis_pairs=(16, 16)))):
        a = dict(q=x, k=x, v=x, kc=kc, vc=vc, slots=slots, pos=pos, rope=rope, q_out=None, k_out=None)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            rope_paged_store(a["q"], a["k"], a["v"], a["kc"], a["vc"], a["slots"], a["pos"], a["rope"], q_out=a["q_out"], k_out=a["k_out"])
    with pytest.raises(RuntimeError):                                             # more rotated channels than there are
        rope_paged_store(x, x, x, kc, vc, slots, pos, Rope(torch.ones(40, device="cuda")))
    for pairs in ((31,), (16, 17), (40, -8), (8, 8, 8, 8, 0), ()):
        with pytest.raises(ValueError):
            Rope(torch.ones(32, device="cuda"), axis_pairs=pairs)
    assert np.isnan(f64(kc)).all()


def test_store_saturates_and_keeps_slots_outside_untouched():
    kc, vc = make_cache(2, 4, 1, "64", "fp8")
    x = torch.full((3, 1, 64), 1e4, dtype=torch.bfloat16, device="cuda")
    q = rope_paged_store(x, -x, x, kc, vc, torch.tensor([3, 8, 1 << 40], device="cuda"))
    assert zyfa_check_errors() == BAD_PAGE and zyfa_check_errors() == 0
    assert f64(q).tolist() == np.full((3, 1, 64), 448.0).tolist()
    k, v = f64(kc).reshape(8, 64), f64(vc).reshape(8, 64)
    assert (k[3] == -448.0).all() and (v[3] == 448.0).all() and np.isnan(np.delete(k, 3, 0)).all() and np.isnan(np.delete(v, 3, 0)).all()


def test_store_offsets_beyond_32_bits():
    kind, page, pages = "bf16", 16, 5
    far = (1 << 30) + 64                                                       # elements between pages: 2 GiB and a little
    store = torch.empty(far * (pages - 1) + page * 128, dtype=torch.bfloat16, device="cuda")
    kc = store.as_strided((pages, page, 2, 64), (far, 128, 64, 1))
    vc = poisoned((pages, page, 2, 64), kind)
    x = random_values((2, 2, 64), kind, np.random.default_rng(0))
    rope_paged_store(None, x, x, kc, vc, torch.tensor([4 * 16 + 15, 3], device="cuda"))
    assert torch.equal(kc[4, 15], x[0]) and torch.equal(kc[0, 3], x[1]) and torch.equal(vc[4, 15], x[0])
    lens, table = i32([80]), i32([[0, 1, 2, 3, 4]])
    for p in range(pages):
        kc[p] = random_values((page, 2, 64), kind, np.random.default_rng(p))
        vc[p] = random_values((page, 2, 64), kind, np.random.default_rng(p + 50))
    q = random_values((1, 2, 64), kind, np.random.default_rng(99))
    assert torch.equal(paged_decode_attn(q, kc, vc, table, lens), paged_decode_attn(q, kc.contiguous(), vc, table, lens))


# ------------------------------------------------------------------------------------------------
# single-token attention

def _decode_case(kind, shape, lens, H, H_kv, page=16, layout="nhd", per_head=False, scale=None, seed=0, loud=1.0, width=None,
                 strided_q=False, lse=True):
    rng = np.random.default_rng(seed)
    d_qk, d_v = SHAPES[shape]
    B = len(lens)
    table, pages = random_table(lens, page, rng, width)
    kc, vc = make_cache(pages, page, H_kv, shape, kind, layout)
    q = random_values((B, H, d_qk), kind, rng, loud)
    ks, vs = [], []
    for b, n in enumerate(lens):
        t = np.arange(n)
        slots = torch.from_numpy(table[b, t // page].astype(np.int64) * page + t % page).cuda()
        ks.append(random_values((n, H_kv, d_qk), kind, rng, loud))
        vs.append(random_values((n, H_kv, d_v), kind, rng))
        fill_tokens(kc, slots, ks[-1])
        fill_tokens(vc, slots, vs[-1])
    ds = [torch.from_numpy((rng.random(B * H_kv if per_head else 1) + 0.5) / 64).float().cuda() if kind == "fp8" else None for _ in range(3)]
    if strided_q:
        wide = poisoned((B, H + 3, d_qk), kind)
        bits(wide)[:, :H] = bits(q)
        q = wide[:, :H]
    got = paged_decode_attn(q, kc, vc, torch.from_numpy(table).cuda(), i32(lens), scale, q_descale=ds[0], k_descale=ds[1], v_descale=ds[2],
                            return_lse=lse)
    assert zyfa_check_errors() == 0
    out, got_lse = got if lse else (got, None)
    out, sc = f64(out), 1.0 / math.sqrt(d_qk) if scale is None else scale
    f = [np.ones((B, H_kv)) if d is None else np.broadcast_to(f64(d).reshape(-1, H_kv) if per_head else f64(d), (B, H_kv)) for d in ds]
    for b in range(B):
        k64, v64, q64 = f64(ks[b]), f64(vs[b]), f64(q[b])
        for h in range(H):
            hk = h // (H // H_kv)
            qr, kr = q64[h] * f[0][b, hk], k64[:, hk] * f[1][b, hk]
            ref, ref_lse, w = P.decode_attention(qr, kr, v64[:, hk] * f[2][b, hk], sc)
            if lens[b] <= 0:
                assert (out[b, h] == 0).all() and (not lse or float(got_lse[b, h]) == -math.inf)
                continue
            tol, lse_tol = decode_tolerance(qr, kr, v64[:, hk], sc, f[2][b, hk], ref, w, kind)
            assert np.all(np.abs(out[b, h] - ref) <= tol), (b, h, float((np.abs(out[b, h] - ref) / tol).max()))
            if lse:
                assert abs(float(got_lse[b, h]) - ref_lse) <= lse_tol + 2.0 ** -23 * abs(ref_lse), (b, h, float(got_lse[b, h]), ref_lse)
    return q, kc, vc, table, ds


@pytest.mark.parametrize("shape", ["64", "128", "mla"])
@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_decode_lengths(kind, shape):
    lens = [0, 1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 127, 128, 129, 191, 192, 255, 256, 257, 300, 0, 511, 513]
    _decode_case(kind, shape, lens, 4, 2, seed=1)
    _decode_case(kind, shape, lens, 3, 3, page=7, seed=2, width=80)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("H,H_kv", [(1, 1), (2, 1), (3, 1), (5, 1), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 1), (128, 1), (14, 2), (21, 7)])
def test_decode_groups(kind, H, H_kv):
    _decode_case(kind, "128", [77, 1, 300], H, H_kv, seed=H, per_head=True)
    _decode_case(kind, "64", [1000], H, H_kv, seed=H + 1)
    _decode_case(kind, "mla", [70, 140], H, H_kv, seed=H + 2)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("H,H_kv", [(10, 10), (20, 10), (11, 11), (12, 6), (32, 32), (24, 8), (32, 2), (96, 4)])
def test_decode_many_kv_heads(kind, H, H_kv):
    # heads that do and do not fill the blocks that take them side by side
    _decode_case(kind, "64", [37, 300], H, H_kv, seed=H, per_head=True, page=32)
    _decode_case(kind, "128", [290, 3], H, H_kv, seed=H + 1, page=8)
    _decode_case(kind, "mla", [64, 129], H, H_kv, seed=H + 2, page=64)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("B,page", [(128, 16), (129, 16), (200, 7), (700, 16), (1100, 24)])
def test_decode_many_requests(kind, B, page):
    # beyond 128 requests the schedule is formed by whole blocks, beyond a block's threads in several passes
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 90, B)
    lens[rng.permutation(B)[: B // 4]] = 0
    lens[3], lens[B - 1] = 800, 5
    _decode_case(kind, "64", lens.tolist(), 2, 1, seed=B, page=page)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("shape", ["64", "128", "mla"])
@pytest.mark.parametrize("B,H,H_kv", [(1, 8, 2), (7, 6, 3), (40, 20, 2), (300, 5, 5), (600, 2, 1)])
def test_decode_small_tables(kind, shape, B, H, H_kv):
    # tables that name few tokens, or many requests of one length: a request is one block's work
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 65, B)
    lens[:: 5] = 0
    lens[B // 2] = 64
    _decode_case(kind, shape, lens.tolist(), H, H_kv, seed=B, page=16, width=4, per_head=True)
    _decode_case(kind, shape, [0] * B, H, H_kv, seed=B, page=8, width=2)
    _decode_case(kind, shape, [130] * min(B, 300), H, H_kv, seed=B + 1, page=32)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_decode_broadcast_cache(kind):
    # strides of 0: every KV head (every page) reads the same rows
    rng = np.random.default_rng(8)
    q, table, lens = random_values((2, 8, 128), kind, rng), i32([[0, 1, 2], [2, 1, 0]]), i32([40, 47])
    k, v = random_values((3, 16, 1, 128), kind, rng), random_values((3, 16, 1, 128), kind, rng)
    wide = [bits(t).expand(-1, -1, 4, -1).view(t.dtype) for t in (k, v)]
    full = [bits(t).expand(-1, -1, 4, -1).contiguous().view(t.dtype) for t in (k, v)]
    a, b = paged_decode_attn(q, *wide, table, lens), paged_decode_attn(q, *full, table, lens)
    assert float((a - b).abs().max()) <= 2.0 ** -7 * float(b.abs().max())        # other tiles, other order: each within its roundings
    one = [bits(t)[:1].expand(3, -1, -1, -1).view(t.dtype) for t in (k, v)]
    c, d = paged_decode_attn(q, *one, table, lens), paged_decode_attn(q, k, v, torch.zeros_like(table), lens)
    assert float((c - d).abs().max()) <= 2.0 ** -7 * float(d.abs().max())


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_decode_very_long_context(kind):
    rng = np.random.default_rng(9)
    n, d = 300_001, 64
    table, pages = random_table([n], 64, rng)
    kc, vc = make_cache(pages, 64, 1, "64", kind)
    q, k, v = (random_values(s, kind, rng) for s in ((1, 2, d), (n, 1, d), (n, 1, d)))
    t = np.arange(n)
    slots = torch.from_numpy(table[0, t // 64].astype(np.int64) * 64 + t % 64).cuda()
    fill_tokens(kc, slots, k)
    fill_tokens(vc, slots, v)
    ds = [torch.tensor([1 / 64.0], device="cuda") if kind == "fp8" else None for _ in range(3)]
    f = 1 / 64.0 if kind == "fp8" else 1.0
    out, lse = paged_decode_attn(q, kc, vc, torch.from_numpy(table).cuda(), i32([n]), q_descale=ds[0], k_descale=ds[1], v_descale=ds[2], return_lse=True)
    for h in range(2):
        qr, kr, vr = f64(q)[0, h] * f, f64(k)[:, 0] * f, f64(v)[:, 0]
        ref, ref_lse, w = P.decode_attention(qr, kr, vr * f, d ** -0.5)
        tol, lse_tol = decode_tolerance(qr, kr, vr, d ** -0.5, f, ref, w, kind)
        assert np.all(np.abs(f64(out)[0, h] - ref) <= tol) and abs(float(lse[0, h]) - ref_lse) <= lse_tol + 2.0 ** -22 * abs(ref_lse)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "joint"])
@pytest.mark.parametrize("page", [1, 5, 8, 16, 48, 128, 1000])
def test_decode_layouts(kind, layout, page):
    _decode_case(kind, "128", [333, 5, 129, 0], 8, 2, page=page, layout=layout, seed=page, per_head=True)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_decode_long_and_ragged(kind):
    _decode_case(kind, "128", [20001], 8, 1, seed=1)
    _decode_case(kind, "64", [1, 9000, 3, 4000, 0, 0, 17], 4, 2, page=32, seed=2)
    _decode_case(kind, "mla", [5000, 1], 4, 4, page=64, seed=3)
    _decode_case(kind, "64", [6000, 40, 2500], 64, 16, page=32, seed=4)           # joins of 192 and 384 rows
    _decode_case(kind, "128", [900, 3000, 5, 1200, 700, 800], 64, 4, seed=5)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_decode_values(kind):
    _decode_case(kind, "128", [200, 700], 4, 1, seed=1, loud=4.0)               # peaked softmax
    _decode_case(kind, "128", [200, 700], 4, 1, seed=2, scale=1e-4)             # flat softmax
    _decode_case(kind, "64", [100], 4, 1, seed=3, scale=2.0, lse=False)
    _decode_case(kind, "128", [60, 61], 6, 2, seed=4, strided_q=True)


def test_decode_long_tail_of_light_weights():
    # one key far above the rest: 40,000 keys whose weights are 2^-14 of its weight carry most of the sum
    n, d = 40001, 128
    q = torch.zeros((1, 1, d), device="cuda")
    q[..., 0] = 1.0
    k = torch.zeros((1, n, 1, d), device="cuda")
    k[0, 777, 0, 0] = 14.0 * math.log(2) * math.sqrt(d)
    rng = np.random.default_rng(0)
    for kind in ("fp8", "bf16"):
        q8, k8 = q.to(dtype_of(kind)), k.to(dtype_of(kind))
        v = random_values((1, n, 1, d), kind, rng)
        out = f64(paged_decode_attn(q8, k8, v, i32([[0]]), i32([n])))[0, 0]
        k64, v64 = f64(k8)[0, :, 0], f64(v)[0, :, 0]
        ref, _, w = P.decode_attention(f64(q8)[0, 0], k64, v64, 1 / math.sqrt(d))
        tol, _ = decode_tolerance(f64(q8)[0, 0], k64, v64, 1 / math.sqrt(d), 1.0, ref, w, kind)
        assert np.all(np.abs(out - ref) <= tol)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_decode_bad_pages_are_left_out(kind):
    rng = np.random.default_rng(3)
    page, n, H_kv = 16, 100, 2
    kc = random_values((9, page, H_kv, 128), kind, rng)
    vc = random_values((9, page, H_kv, 128), kind, rng)
    q = random_values((2, 4, 128), kind, rng, 1 / 64 if kind == "fp8" else 1.0)
    table = np.array([[3, -1, 5, 9, 2_000_000_000, 0, 8], [-2, -5, 9, 77, 10, 11, 12]], dtype=np.int32)
    out, lse = paged_decode_attn(q, kc, vc, torch.from_numpy(table).cuda(), i32([n, n]), return_lse=True)
    assert zyfa_check_errors() == BAD_PAGE
    t = np.arange(n)
    t = t[np.isin(t // page, [0, 2, 5, 6])]
    k64, v64 = f64(kc)[table[0, t // page], t % page], f64(vc)[table[0, t // page], t % page]
    for h in range(4):
        ref, ref_lse, w = P.decode_attention(f64(q)[0, h], k64[:, h // 2], v64[:, h // 2], 128 ** -0.5)
        tol, lse_tol = decode_tolerance(f64(q)[0, h], k64[:, h // 2], v64[:, h // 2], 128 ** -0.5, 1.0, ref, w, kind)
        assert np.all(np.abs(f64(out)[0, h] - ref) <= tol) and abs(float(lse[0, h]) - ref_lse) <= lse_tol + 2.0 ** -22 * abs(ref_lse)
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())


@pytest.mark.parametrize("page", [7, 16])
@pytest.mark.parametrize("n", [70, 9000])
def test_decode_scores_of_minus_infinity(n, page):
    # keys whose score overflows to -inf weigh nothing, also as the first ones of a part; a row of only such keys is empty
    rng = np.random.default_rng(n + page)
    table, pages = random_table([n, n], page, rng)
    kc, vc = make_cache(pages, page, 1, "64", "bf16")
    q, k, v = (random_values(s, "bf16", rng) for s in ((2, 2, 64), (2, n, 1, 64), (2, n, 1, 64)))
    q[:, 0, 0], q[:, 1, 0] = 4.0, 0.0                                             # head 0: 4 * -3e38 is below any fp32 number
    low = np.zeros(n, dtype=bool)
    low[rng.permutation(n)[: n // 3]] = low[: n // 2] = True
    k[0, torch.from_numpy(low).cuda(), 0, 0] = -3e38
    k[1, :, 0, 0] = -3e38
    t = np.arange(n)
    for b in range(2):
        slots = torch.from_numpy(table[b, t // page].astype(np.int64) * page + t % page).cuda()
        fill_tokens(kc, slots, k[b])
        fill_tokens(vc, slots, v[b])
    out, lse = paged_decode_attn(q, kc, vc, torch.from_numpy(table).cuda(), i32([n, n]), return_lse=True)
    assert bool((out[1, 0] == 0).all()) and float(lse[1, 0]) == -math.inf
    for b, h in ((0, 0), (0, 1), (1, 1)):
        keep = ~low if h == 0 else low | True
        q64, k64, v64 = f64(q)[b, h], f64(k)[b, keep, 0], f64(v)[b, keep, 0]
        ref, ref_lse, w = P.decode_attention(q64, k64, v64, 0.125)
        tol, lse_tol = decode_tolerance(q64, k64, v64, 0.125, 1.0, ref, w, "bf16")
        assert np.all(np.abs(f64(out)[b, h] - ref) <= tol) and abs(float(lse[b, h]) - ref_lse) <= lse_tol + 2.0 ** -22 * abs(ref_lse)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_decode_lengths_outside_the_table(kind):
    rng = np.random.default_rng(4)
    kc, vc = random_values((4, 16, 1, 64), kind, rng), random_values((4, 16, 1, 64), kind, rng)
    q = random_values((3, 2, 64), kind, rng)
    table = i32([[0, 1], [2, 3], [1, 0]])
    got = paged_decode_attn(q, kc, vc, table, i32([-5, 1000, 32]))
    same = paged_decode_attn(q, kc, vc, table, i32([0, 32, 32]))
    assert torch.equal(got, same) and bool((got[0] == 0).all()) and zyfa_check_errors() == 0
    none = paged_decode_attn(q, kc, vc, table[:, :0], i32([3, 3, 3]))
    assert bool((none == 0).all())
    assert paged_decode_attn(q[:0], kc, vc, table[:0], i32([])).shape == (0, 2, 64)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_decode_shared_pages_streams_and_repeats(kind):
    rng = np.random.default_rng(5)
    kc, vc = random_values((300, 16, 2, 128), kind, rng), random_values((300, 16, 2, 128), kind, rng)
    q = random_values((6, 8, 128), kind, rng)
    q[3] = q[0]
    prefix = rng.permutation(300)[:250].astype(np.int32)
    table = torch.from_numpy(np.stack([prefix] * 6)).cuda()
    lens = i32([4000, 100, 3999, 4000, 0, 1])
    out = paged_decode_attn(q, kc, vc, table, lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        outs = [paged_decode_attn(q, kc, vc, table, lens) for _ in range(20)]
    side.synchronize()
    assert all(torch.equal(o, out) for o in outs)
    ws = torch.full((paged_decode_workspace_bytes(6, 8, 2, 128, 4000),), 0xFF, dtype=torch.uint8, device="cuda")
    mine = torch.empty_like(out)
    assert paged_decode_attn(q, kc, vc, table, lens, out=mine, workspace=ws) is mine and torch.equal(mine, out)
    assert torch.equal(paged_decode_attn(q, kc, vc, table, lens, workspace=ws), out)


def test_decode_tensor_refusals():
    kc = torch.zeros((4, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    q, table, lens = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device="cuda"), i32([[0]] * 3), i32([1] * 3)
    for bad in (dict(q=q.to(E4M3)), dict(q=q[:, :3]), dict(q=q[..., ::2]), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(lens=lens.long()), dict(lens=lens[:2]), dict(lens=lens.cpu()), dict(table=table.long()), dict(table=table[:2]),
                dict(table=i32([[0, 1]] * 6).T[:, ::2][:, :3]), dict(v=kc[:3]), dict(v=kc.cpu()), dict(kc=kc.transpose(2, 3)),
                dict(out=torch.empty((3, 4, 128), device="cuda")), dict(ws=torch.empty(1 << 20, device="cuda"))):
        a = dict(q=q, kc=kc, v=kc, table=table, lens=lens, out=None, ws=None)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            paged_decode_attn(a["q"], a["kc"], a["v"], a["table"], a["lens"], out=a["out"], workspace=a["ws"])
    with pytest.raises(RuntimeError):
        paged_decode_attn(q, kc, kc, table, lens, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    for scale in (1e-60, -1.0, math.nan, math.inf):                               # the first would round to 0, which selects the default
        with pytest.raises((ValueError, RuntimeError)):
            paged_decode_attn(q, kc, kc, table, lens, scale)
    k8 = kc.to(E4M3)
    one, many = torch.ones(1, device="cuda"), torch.ones(6, device="cuda")
    for kw in (dict(q_descale=one, k_descale=many), dict(q_descale=torch.ones(5, device="cuda")), dict(v_descale=one.cpu())):
        with pytest.raises(ValueError):
            paged_decode_attn(q.to(E4M3), k8, k8, table, lens, **kw)


# ------------------------------------------------------------------------------------------------
# the operators together

class _Server:
    """A small serving loop over the three operators, with buffers of fixed sizes as a captured step needs them."""

    def __init__(self, kind, B, H, H_kv, shape, page, pages, width, seed):
        self.rng = np.random.default_rng(seed)
        self.kind, self.B, self.H, self.H_kv, self.shape, self.page = kind, B, H, H_kv, shape, page
        self.d_qk, self.d_v = SHAPES[shape]
        self.kc, self.vc = make_cache(pages, page, H_kv, shape, kind)
        self.free = torch.from_numpy(self.rng.permutation(pages).astype(np.int32)).cuda()
        self.cursor, self.lens = i32([0]), i32([0] * B)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        rot = 64
        self.inv = (10000.0 ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)
        self.rope = Rope(torch.from_numpy(self.inv).cuda(), offset=self.d_qk - rot)
        self.ds = [torch.tensor([1 / 64.0], device="cuda") if kind == "fp8" else None for _ in range(3)]

    def store(self, x, plan, dense=False):
        q, k, v = x
        n = q.shape[0]
        outs = {}
        if dense:
            outs = dict(k_out=torch.empty((n, self.H_kv, self.d_qk), dtype=dtype_of(self.kind), device="cuda"),
                        v_out=torch.empty((n, self.H_kv, self.d_v), dtype=dtype_of(self.kind), device="cuda"))
        q = rope_paged_store(q, k, v, self.kc, self.vc, plan.slots, plan.positions, self.rope, q_descale=self.ds[0], k_descale=self.ds[1],
                             v_descale=self.ds[2], **outs)
        return q, outs

    def plan(self, new, rows):
        p = paged_plan(self.lens, new, self.table, self.free, self.cursor, self.page, rows)
        self.cursor.copy_(p.cursor)
        self.lens.copy_(p.seq_lens)
        return p

    def attend(self, q):
        return paged_decode_attn(q, self.kc, self.vc, self.table, self.lens, q_descale=self.ds[0], k_descale=self.ds[1], v_descale=self.ds[2])

    def tokens(self, n):
        return [torch.from_numpy(self.rng.standard_normal((n, h, d))).to(torch.bfloat16).cuda()
                for h, d in ((self.H, self.d_qk), (self.H_kv, self.d_qk), (self.H_kv, self.d_v))]


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_prompt_then_tokens(kind):
    """Prompts through plan, store and prefill, then token steps through plan, store and decode: each step's
    output equals float64 attention over all tokens so far, within the quantisation of Q, K and V."""
    prompts, steps = [37, 1, 0, 64], 5
    s = _Server(kind, 4, 4, 2, "128", 16, 40, 8, seed=1)
    x = s.tokens(sum(prompts))
    plan = s.plan(i32(prompts), sum(prompts))
    q, dense = s.store(x, plan, dense=True)
    history = [[[t[a: a + n]] for t in x] for a, n in zip(np.cumsum([0] + prompts), prompts)]
    a = 0
    for b, n in enumerate(prompts):                                             # the prompt's own attention, on the dense copies
        if n:
            one = lambda t: t[a: a + n].unsqueeze(0)  # noqa: E731
            out = flash_attn_func(one(q), one(dense["k_out"]), one(dense["v_out"]), q_descale=s.ds[0], k_descale=s.ds[1], v_descale=s.ds[2])
            last = paged_decode_attn(q[a + n - 1: a + n], s.kc, s.vc, s.table[b: b + 1], i32([n]), q_descale=s.ds[0], k_descale=s.ds[1],
                                     v_descale=s.ds[2])
            # the two differ by the weights' roundings (prefill: e4m3 codes up to 7.5% off; bf16: 2^-8 on either side)
            # and the output's (2^-8 on either side)
            assert float((out[0, -1] - last[0]).float().norm() / last.float().norm()) < (0.075 + 2 * 2.0 ** -8 if kind == "fp8" else 4 * 2.0 ** -8)
        a += n
    for step in range(steps):
        x = s.tokens(4)
        plan = s.plan(i32([1] * 4), 4)
        q, _ = s.store(x, plan)
        out = f64(s.attend(q))
        assert zyfa_check_errors() == 0
        for b in range(4):
            for t, row in zip(history[b], x):
                t.append(row[b: b + 1])
            qs, ks, vs = (f64(torch.cat(t)) for t in history[b])
            n = len(ks)
            assert n == prompts[b] + step + 1 == int(s.lens[b])
            pos = [np.arange(n)]
            kr = P.rope_rotate(ks, pos, s.inv, [32], offset=64)
            qr = P.rope_rotate(qs[-1:], [[n - 1]], s.inv, [32], offset=64)[0]
            for h in range(4):
                ref, _, _ = P.decode_attention(qr[h], kr[:, h // 2], vs[:, h // 2], 128 ** -0.5)
                # each input off by half a step: scores of size ~1 by ~2 half steps, V by one, relative to |out| ~ |V|
                tol = 4 * (2.0 ** -4 if kind == "fp8" else 2.0 ** -8)
                assert np.linalg.norm(out[b, h] - ref) <= tol * np.linalg.norm(vs[:, h // 2], axis=1).max()


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_captured_step_replays(kind):
    """One captured token step (plan, store, decode with its buffers) replayed over many steps equals eager steps."""
    B, rows, steps = 5, 7, 40
    a = _Server(kind, B, 4, 1, "mla", 8, 60, 10, seed=2)
    b = _Server(kind, B, 4, 1, "mla", 8, 60, 10, seed=2)
    new = i32([1] * B)
    xs = [a.tokens(rows) for _ in range(steps)]
    static = [torch.zeros_like(t) for t in xs[0]]

    def step(s, x):
        plan = s.plan(new, rows)
        q, _ = s.store(x, plan)
        return s.attend(q[:B]), plan

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(_Server(kind, B, 4, 1, "mla", 8, 60, 10, seed=3), static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, plan = step(b, static)
    for x in xs:
        want, want_plan = step(a, x)
        for t, v in zip(static, x):
            t.copy_(v)
        graph.replay()
        assert all(torch.equal(p, w) for p, w in zip(plan, want_plan))
        assert torch.equal(out, want)
    assert torch.equal(bits(a.kc), bits(b.kc)) and torch.equal(a.table, b.table) and zyfa_check_errors() == 0
    assert a.lens.tolist() == [steps] * B


def test_two_captured_graphs_with_their_own_workspaces():
    rng = np.random.default_rng(7)
    kc, vc = random_values((64, 64, 2, 128), "bf16", rng), random_values((64, 64, 2, 128), "bf16", rng)
    qs = [random_values((2, 8, 128), "bf16", rng) for _ in range(2)]
    table, lens = torch.arange(64, dtype=torch.int32, device="cuda").reshape(2, 32).contiguous(), i32([2048, 1500])
    want = [paged_decode_attn(q, kc, vc, table, lens) for q in qs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        ws = torch.empty(paged_decode_workspace_bytes(2, 8, 2, 128, 2048), dtype=torch.uint8, device="cuda")
        with torch.cuda.graph(g):
            outs.append(paged_decode_attn(q, kc, vc, table, lens, workspace=ws))
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


_FIRST_IN_CAPTURE = """
import torch
from fp8_causal_prefill_gb300 import Rope, paged_decode_attn, paged_plan, rope_paged_store, zyfa_check_errors
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
n, page = 50, 16
x = [torch.randn(n, h, 128, device="cuda").bfloat16() for h in (8, 2, 2)]
kc, vc = (torch.zeros(6, page, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
table, lens, new, free, cursor = i32([[-1] * 4]), i32([0]), i32([n]), i32([4, 1, 5, 0, 2]), i32([0])
rope = Rope(torch.rand(64, device="cuda"))
def step():
    plan = paged_plan(lens, new, table, free, cursor, page, n)
    q = rope_paged_store(*x, kc, vc, plan.slots, plan.positions, rope)
    return paged_decode_attn(q[n - 1:], kc, vc, table, plan.seq_lens)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
got = out.clone()
kc.zero_(); vc.zero_(); table.fill_(-1)
assert torch.equal(step(), got) and bool((got != 0).any()) and zyfa_check_errors() == 0
"""


def test_first_calls_of_a_process_inside_a_capture():
    # nothing that a call does once per process or device (symbol addresses, kernel attributes) is forbidden in a capture
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_IN_CAPTURE], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0, r.stderr[-2000:]
