"""GPU tests of the paged serving operators where their numbers, checks or choices could go wrong beside the ordinary cases:
the bits that the weights keep, values that are not finite, steps over capacity, batches of every size."""
import ctypes
import math
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

from _paged_util import SHAPES, bits, decode_tolerance, dtype_of, f64, fill_tokens, make_cache, random_table, random_values
from fp8_causal_prefill_gb300 import Rope, api, paged_decode_attn, paged_decode_workspace_bytes, paged_plan, rope_paged_store, zyfa_check_errors
from oracle import paged as P
from test_paged_gpu import _FIRST_IN_CAPTURE, _Server

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class _Batch:
    """A decode batch over a paged cache: q, the caches, the table and each request's keys and values."""

    def __init__(self, kind, shape, lens, H, H_kv, page=16, width=None, seed=0):
        rng = np.random.default_rng(seed)
        d_qk, d_v = SHAPES[shape]
        table, pages = random_table(lens, page, rng, width)
        self.kind, self.lens, self.page, self.table = kind, list(lens), page, table
        self.kc, self.vc = make_cache(pages, page, H_kv, shape, kind)
        self.q = random_values((len(lens), H, d_qk), kind, rng)
        self.k = [random_values((n, H_kv, d_qk), kind, rng) for n in lens]
        self.v = [random_values((n, H_kv, d_v), kind, rng) for n in lens]
        for b in range(len(lens)):
            self.fill(b)
        self.scale = 1.0 / math.sqrt(d_qk)
        self.descale = torch.tensor([1 / 64.0], device="cuda") if kind == "fp8" else None

    def fill(self, b):
        """Writes request b's keys and values into its pages."""
        t = np.arange(self.lens[b])
        slots = torch.from_numpy(self.table[b, t // self.page].astype(np.int64) * self.page + t % self.page).cuda()
        fill_tokens(self.kc, slots, self.k[b])
        fill_tokens(self.vc, slots, self.v[b])

    def attend(self, **kw):
        d = self.descale
        out, lse = paged_decode_attn(self.q, self.kc, self.vc, torch.from_numpy(self.table).cuda(), i32(self.lens), q_descale=d, k_descale=d,
                                     v_descale=d, return_lse=True, **kw)
        assert zyfa_check_errors() == 0
        return f64(out), f64(lse)

    def rows(self):
        """(b, h, query, keys, values) of every row, in float64 and real units (values without their descale)."""
        f = 1 / 64.0 if self.kind == "fp8" else 1.0
        H, H_kv = self.q.shape[1], self.kc.shape[2]
        q = f64(self.q) * f
        for b in range(len(self.lens)):
            k, v = f64(self.k[b]) * f, f64(self.v[b])
            for h in range(H):
                yield b, h, q[b, h], k[:, h * H_kv // H], v[:, h * H_kv // H]


# ------------------------------------------------------------------------------------------------
# the bits that the weights keep

@pytest.mark.parametrize("shape", ["64", "128", "mla"])
@pytest.mark.parametrize("page", [7, 16])
def test_decode_bf16_weights_keep_16_bits(shape, page):
    """Weights multiply a bf16 V as a sum of two bf16 numbers, the second the rest of the first: a rounding is off by 2^-8 of what
    it rounds, so the two are off by 2^-16.  Rows whose values nearly cancel show a weight of 8 bits; the tolerance is that of the other tests
    with 2^-16 in place of 2^-8."""
    x = _Batch("bf16", shape, [2, 5, 64, 300, 5000], 8, 2, page=page, seed=page)
    out, lse = x.attend()
    worst = 0.0
    for b, h, q, k, v in x.rows():
        ref, ref_lse, w = P.decode_attention(q, k, v, x.scale)
        tol, lse_tol = decode_tolerance(q, k, v, x.scale, 1.0, ref, w, "bf16")
        tol = tol - 2 * (2.0 ** -8 - 2.0 ** -16) * (w @ np.abs(v)) * 1.01
        worst = max(worst, float((np.abs(out[b, h] - ref) / tol).max()))
        assert abs(lse[b, h] - ref_lse) <= lse_tol + 2.0 ** -22 * abs(ref_lse)
    assert worst <= 1.0, worst


# ------------------------------------------------------------------------------------------------
# values that are not finite

# (requests, query heads, KV heads, tokens): rows in one block; few rows (16 warps a row, by channels and whole); 8 and 4 warps a row;
# a warp a row
SPLITS = [(2, 4, 2, 40), (1, 4, 2, 9000), (2, 32, 8, 9000), (6, 64, 4, 5000), (16, 32, 8, 2000), (48, 32, 8, 700)]


@pytest.mark.parametrize("kind,what", [(kind, what) for kind in ("fp8", "bf16") for what in ("query", "key", "value")] +
                         [("bf16", "infinite score")])                        # (e4m3 products do not overflow)
@pytest.mark.parametrize("page", [7, 16])
@pytest.mark.parametrize("B,H,H_kv,n", SPLITS)
def test_decode_shows_values_that_are_not_finite(kind, B, H, H_kv, n, page, what):
    """A NaN in a query, a key or a value, and a score of +inf, make NaN of the rows that they belong to, however these are split, and
    change no other row."""
    x = _Batch(kind, "128", [n + i % 3 for i in range(B)], H, H_kv, page=page, width=None if n < 100 else -(-(n + 40) // page) + 64, seed=n)
    clean, clean_lse = x.attend()
    assert np.isfinite(clean).all() and np.isfinite(clean_lse).all()
    b, head, token, group = B - 1, H_kv - 1, n // 3, H // H_kv
    nan = bits(torch.full((1,), math.nan, device="cuda").to(dtype_of(kind)))
    rows, channels = np.zeros((B, H), dtype=bool), slice(None)
    rows[b, head * group:] = True
    if what == "query":
        bits(x.q)[b, head * group, 5] = nan
        rows[b] = False
        rows[b, head * group] = True
    elif what == "key":
        bits(x.k[b])[token, head, 5] = nan
    elif what == "infinite score":
        x.q[b, head * group:, 5] = 4.0
        x.k[b][token, head, 5] = 3e38
    else:
        bits(x.v[b])[token, head, 5] = nan
        channels = 5
    x.fill(b)
    out, lse = x.attend()
    assert np.isnan(out[rows][:, channels]).all()
    if what == "value":
        out[rows, 5] = clean[rows, 5]
        assert np.array_equal(out, clean) and np.array_equal(lse, clean_lse)
    else:
        assert not np.isfinite(lse[rows]).any() and not (lse[rows] == -math.inf).any()
        assert np.array_equal(out[~rows], clean[~rows]) and np.array_equal(lse[~rows], clean_lse[~rows])


@pytest.mark.parametrize("page", [7, 16])
@pytest.mark.parametrize("n", [40, 5000])
def test_decode_of_scores_near_the_lowest_number(n, page):
    """Scores between -3e38 and the lowest fp32 number, in units of log2, are scores like others: their weights go by their differences."""
    x = _Batch("bf16", "64", [n], 1, 1, page=page, seed=n)
    x.scale = 1.0 / math.log2(math.e)
    x.q.zero_()
    x.q[..., 0] = 1.0
    x.k[0].zero_()
    x.k[0][..., 0] = -3.2e38                                                   # one score for all: equal weights
    x.fill(0)
    out, lse = x.attend(softmax_scale=x.scale)
    assert np.isfinite(lse).all()
    v = f64(x.v[0])[:, 0]
    # equal weights are exact powers of two; n products and weights summed in fp32, out rounded once
    assert np.all(np.abs(out[0, 0] - v.mean(0)) <= 2.0 ** -8 * np.abs(v.mean(0)) + 2 * n * 2.0 ** -24 * np.abs(v).mean(0) * 1.01)


# ------------------------------------------------------------------------------------------------
# a step over capacity

@pytest.mark.parametrize("over", [1, 5000])
@pytest.mark.parametrize("above", [1, 300])
def test_plan_of_more_tokens_than_rows(above, over):
    """Tokens behind the last row are dropped, not their pages: they are in the table, whatever number of rows the blocks take."""
    blocks = 8 * torch.cuda.get_device_properties(0).multi_processor_count      # each takes 256 rows, or more where there are more
    rows, page, B = blocks * 256 + above, 16, 7
    rng = np.random.default_rng(above + over)
    cached = rng.integers(0, 100, B)
    new = np.full(B, (rows + over) // B)
    new[-1] += rows + over - new.sum()
    need = int(sum(-(-int(c + n) // page) for c, n in zip(cached, new)))
    free = rng.permutation(need + 9).astype(np.int32)
    table = np.full((B, -(-int(max(cached + new)) // page)), 5, dtype=np.int32)
    want = P.paged_plan(cached, new, table, free, 2, page, rows)
    t = torch.from_numpy(table).cuda()
    got = paged_plan(i32(cached), i32(new), t, torch.from_numpy(free).cuda(), i32([2]), page, rows)
    assert zyfa_check_errors() == 6                                             # ZYFA_ERR_CAPACITY
    np.testing.assert_array_equal(t.cpu().numpy(), want[0])
    for g, w in zip(got, want[1:]):
        np.testing.assert_array_equal(g.cpu().numpy().reshape(-1), np.atleast_1d(w))


@pytest.mark.parametrize("B,page,width,rows", [(3, 16, 9, 500), (3, 1, 40, 0), (1500, 5, 3, 4000)])
def test_plan_of_lengths_as_large_as_int32_holds(B, page, width, rows):
    # lengths that no program means end in an error, at once
    most, cap, cursor = 2 ** 31 - 1, width * page, 4
    pool = cursor + B * width - 1                                               # the last page is missing
    free = np.random.default_rng(B).permutation(pool).astype(np.int32)
    table = torch.full((B, width + 2), 5, dtype=torch.int32, device="cuda")
    got = paged_plan(i32([0] * B), i32([most] * B), table[:, :width], torch.from_numpy(free).cuda(), i32([cursor]), page, rows)
    assert zyfa_check_errors() == 6
    pages = np.append(free[cursor:], -1).reshape(B, width)
    np.testing.assert_array_equal(table.cpu().numpy(), np.pad(pages, ((0, 0), (0, 2)), constant_values=5))
    t = np.arange(rows)                                                         # all of request 0
    slots = np.where(t < cap, pages[0, np.minimum(t // page, width - 1)].astype(np.int64) * page + t % page, -1)
    assert got.seq_lens.tolist() == [cap] * B and got.cu_tokens.tolist() == [min(b * most, most) for b in range(B + 1)]
    assert got.positions.tolist() == t.tolist() and got.slots.tolist() == slots.tolist() and got.cursor.tolist() == [pool]


# ------------------------------------------------------------------------------------------------
# batches of every size

@pytest.mark.parametrize("kind,H,H_kv,B", [("bf16", 32, 32, 28), ("bf16", 32, 8, 114), ("fp8", 32, 8, 228), ("fp8", 16, 16, 114)])
def test_decode_of_one_long_request_where_whole_ones_would_fill_the_gpu(kind, H, H_kv, B):
    lens = [1 + 7 * b % 30 for b in range(B)]
    lens[B // 3], lens[5], lens[6] = 3000, 0, 0
    x = _Batch(kind, "64" if H_kv == 16 else "128", lens, H, H_kv, seed=B)
    out, lse = x.attend()
    f = 1 / 64.0 if kind == "fp8" else 1.0
    for b, h, q, k, v in x.rows():
        ref, ref_lse, w = P.decode_attention(q, k, v * f, x.scale)
        if lens[b] == 0:
            assert (out[b, h] == 0).all() and lse[b, h] == -math.inf
            continue
        tol, lse_tol = decode_tolerance(q, k, v, x.scale, f, ref, w, kind)
        assert np.all(np.abs(out[b, h] - ref) <= tol) and abs(lse[b, h] - ref_lse) <= lse_tol + 2.0 ** -22 * abs(ref_lse)


# ------------------------------------------------------------------------------------------------
# steps whose attention is split and joined, captured

def _cache_of(kc, vc):
    return api.PagedCache(kc.data_ptr(), vc.data_ptr(), 0 if kc.element_size() == 1 else 1, kc.shape[1], kc.shape[0], kc.shape[2], kc.shape[3],
                          vc.shape[3], *kc.stride()[:3], *vc.stride()[:3])


def _launches(kc, vc, width, B, H):
    return api.load_library().zyfa_attn_decode_paged_launches(ctypes.byref(_cache_of(kc, vc)), width, B, H, 0)


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("B", [5, 40, 140, 300])
def test_captured_step_of_wide_tables_replays(kind, B):
    """A captured token step over a table of 800 tokens a request, some of them idle, replayed equals eager steps: the join finds the lengths
    that the step's plan has written, at every number of requests that reads them in a way of its own."""
    H, H_kv, page, width, steps = 4, 2, 8, 100, 6
    rng = np.random.default_rng(B)
    prompts = rng.integers(0, 60, B)
    prompts[0], prompts[B // 2], prompts[B - 1] = 500, 0, 0
    new = np.ones(B, dtype=int)
    new[rng.permutation(B)[: B // 4]] = 0
    pages = int(sum(-(-(p + steps) // page) for p in prompts)) + 8
    a, b = (_Server(kind, B, H, H_kv, "128", page, pages, width, seed=B) for _ in range(2))
    assert _launches(a.kc, a.vc, width, B, H) == 2
    for s in (a, b):
        s.store(s.tokens(int(prompts.sum())), s.plan(i32(prompts), int(prompts.sum())))
    new_t = i32(new)
    static = [torch.zeros_like(t) for t in a.tokens(B)]

    def step(s, x):
        plan = s.plan(new_t, B)
        q, _ = s.store(x, plan)
        rows = plan.cu_tokens[:B].long().clamp(max=int(new.sum()) - 1)          # an idle request takes any row
        return s.attend(q[rows]), plan

    step(_Server(kind, B, H, H_kv, "128", page, pages, width, seed=1), static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, plan = step(b, static)
    for _ in range(steps):
        x = a.tokens(B)
        want, want_plan = step(a, x)
        for t, v in zip(static, x):
            t.copy_(v)
        out.fill_(math.nan)
        graph.replay()
        assert all(torch.equal(p, w) for p, w in zip(plan, want_plan))
        assert torch.equal(out, want) and bool(torch.isfinite(want).all())
    assert torch.equal(bits(a.kc), bits(b.kc)) and torch.equal(a.table, b.table) and zyfa_check_errors() == 0
    assert a.lens.tolist() == (prompts + steps * new).tolist()


def test_first_calls_of_a_process_inside_a_capture_of_a_wide_table():
    # kernel attributes of both kernels and the dependent launch of the join are set up within the capture
    text = _FIRST_IN_CAPTURE.replace("[[-1] * 4]", "[[-1] * 64]")
    assert text != _FIRST_IN_CAPTURE
    assert _launches(torch.empty((6, 16, 2, 128), dtype=torch.bfloat16), torch.empty((6, 16, 2, 128), dtype=torch.bfloat16), 64, 1, 8) == 2
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", text], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("B", [256, 257, 700, 1100])
def test_decode_of_many_requests_is_split(kind, B):
    # up to 256 requests warps form the schedule, beyond that blocks, beyond a block's threads in several passes
    lens = [b * 37 % 90 if b % 4 else 0 for b in range(B)]
    lens[3], lens[B - 1] = 800, 5
    x = _Batch(kind, "64", lens, 2, 1, page=16, width=200, seed=B)
    assert _launches(x.kc, x.vc, 200, B, 2) == 2
    out, lse = x.attend()
    f = 1 / 64.0 if kind == "fp8" else 1.0
    for b, h, q, k, v in x.rows():
        ref, ref_lse, w = P.decode_attention(q, k, v * f, x.scale)
        if lens[b] == 0:
            assert (out[b, h] == 0).all() and lse[b, h] == -math.inf
            continue
        tol, lse_tol = decode_tolerance(q, k, v, x.scale, f, ref, w, kind)
        assert np.all(np.abs(out[b, h] - ref) <= tol) and abs(lse[b, h] - ref_lse) <= lse_tol + 2.0 ** -22 * abs(ref_lse)


# ------------------------------------------------------------------------------------------------
# descales per head through the whole step

@pytest.mark.parametrize("page", [7, 16])
@pytest.mark.parametrize("width", [None, 90])
def test_descales_of_a_head_serve_the_store_and_the_attention(page, width):
    """The H_kv values that the store divides by are those that the attention multiplies by, for any number of requests."""
    B, H, H_kv, d, n = 3, 8, 4, 128, 41
    rng = np.random.default_rng(page)
    table, pages = random_table([n] * B, page, rng, width)
    kc, vc = make_cache(pages, page, H_kv, "128", "fp8")
    ds = [torch.from_numpy((rng.random(H_kv) + 0.5) / 64).float().cuda() for _ in range(3)]
    q, k, v = (torch.from_numpy(rng.standard_normal((B * n, h, d))).to(torch.bfloat16).cuda() for h in (H, H_kv, H_kv))
    t = np.arange(n)
    slots = torch.from_numpy(np.concatenate([table[b, t // page].astype(np.int64) * page + t % page for b in range(B)])).cuda()
    kw = dict(q_descale=ds[0], k_descale=ds[1], v_descale=ds[2])
    q8 = rope_paged_store(q, k, v, kc, vc, slots, **kw)[n - 1:: n]
    lens, table_t = i32([n] * B), torch.from_numpy(table).cuda()
    out = paged_decode_attn(q8, kc, vc, table_t, lens, **kw)
    wide = {name: x.repeat(B) for name, x in kw.items()}
    assert torch.equal(out, paged_decode_attn(q8, kc, vc, table_t, lens, **wide)) and zyfa_check_errors() == 0
    for b in range(B):                                                          # one request by itself
        one = paged_decode_attn(q8[b: b + 1], kc, vc, table_t[b: b + 1], lens[:1], **kw)
        ref = [P.decode_attention(f64(q8)[b, h] * f64(ds[0])[h // 2], f64(kc)[table[b, t // page], t % page, h // 2] * f64(ds[1])[h // 2],
                                  f64(vc)[table[b, t // page], t % page, h // 2] * f64(ds[2])[h // 2], d ** -0.5)[0] for h in range(H)]
        for got in (out[b], one[0]):
            # within the tolerance of the weights and the output's rounding (2^-11 and 2^-8), with |v| of some units
            assert np.all(np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * np.abs(f64(v)[b * n: (b + 1) * n]).max())
    with pytest.raises(ValueError):                                             # two forms at once
        paged_decode_attn(q8, kc, vc, table_t, lens, q_descale=ds[0], k_descale=wide["k_descale"])
    with pytest.raises(ValueError):
        paged_decode_attn(q8, kc, vc, table_t, lens, q_descale=ds[0][:2])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_store_shows_frequencies_that_are_not_finite(kind, interleaved):
    """A pair whose frequency is infinite or NaN is NaN, as its angle is; every other channel is as with finite ones."""
    n, H, H_kv, d = 40, 4, 2, 128
    rng = np.random.default_rng(11)
    q, k, v = (torch.from_numpy(rng.standard_normal((n, h, d))).to(torch.bfloat16).cuda() for h in (H, H_kv, H_kv))
    inv = torch.from_numpy((10000.0 ** (-np.arange(0, d, 2) / d)).astype(np.float32)).cuda()
    bad = inv.clone()
    bad[3], bad[17], bad[63] = math.inf, math.nan, -math.inf
    slots, positions = torch.arange(n, device="cuda"), i32(np.arange(n))
    got = []
    for f in (inv, bad):
        kc, vc = make_cache(3, 16, H_kv, "128", kind)
        out = rope_paged_store(q, k, v, kc, vc, slots, positions, Rope(f, interleaved=interleaved))
        got.append([f64(t) for t in (out, kc.flatten(0, 1)[:n], vc.flatten(0, 1)[:n])])
    lost = np.zeros(d, dtype=bool)
    for i in (3, 17, 63):
        lost[[2 * i, 2 * i + 1] if interleaved else [i, i + 64]] = True
    for clean, x in zip(*got):
        assert np.isfinite(clean).all() and np.array_equal(x[..., ~lost], clean[..., ~lost])
    assert np.isnan(got[1][0][..., lost]).all() and np.isnan(got[1][1][..., lost]).all() and np.array_equal(got[1][2], got[0][2])


# ------------------------------------------------------------------------------------------------
# waits that run out

@pytest.mark.parametrize("kind", ["fp8", "bf16"])
@pytest.mark.parametrize("shape,H,H_kv,lens,width", [
    ("128", 32, 8, [64, 0, 17], 4),                                             # a request a block, no join
    ("128", 32, 8, [900, 0, 17, 400], 64),                                      # split and joined
    ("64", 2, 1, [900, 5], 64),                                                 # warps that share a head's tokens and would meet
    ("mla", 20, 2, [300], 64)])
def test_decode_without_its_loads_times_out_and_the_next_call_is_right(kind, shape, H, H_kv, lens, width):
    """Every wait of the kernel is bounded: without a load it ends, with a status that the host reads once, and the context, the status
    word and the workspace serve the next call as ever."""
    x = _Batch(kind, shape, lens, H, H_kv, width=width, seed=3)
    B, d_v = len(lens), x.vc.shape[3]
    ws = torch.empty(paged_decode_workspace_bytes(B, H, H_kv, d_v, width * x.page), dtype=torch.uint8, device="cuda")
    want, want_lse = x.attend(workspace=ws)
    out = torch.empty((B, H, d_v), dtype=torch.bfloat16, device="cuda")
    table, lens_t, c = torch.from_numpy(x.table).cuda(), i32(lens), _cache_of(x.kc, x.vc)
    stream = torch.cuda.current_stream().cuda_stream
    st = api.load_library().zyfa_selftest_stalled_decode(x.q.data_ptr(), x.q.stride(0), ctypes.byref(c), table.data_ptr(), width, width,
                                                         lens_t.data_ptr(), out.data_ptr(), B, H, ws.data_ptr(), ws.numel(), stream)
    assert st == 0
    assert zyfa_check_errors(stream) == 5 and zyfa_check_errors(stream) == 0    # ZYFA_ERR_TIMEOUT, read and cleared
    got, got_lse = x.attend(workspace=ws)
    assert np.array_equal(got, want) and np.array_equal(got_lse, want_lse)


# ------------------------------------------------------------------------------------------------
# several callers

def test_steps_of_several_threads_and_streams():
    """Threads that each run their own steps on their own stream get what they get alone."""
    def run(seed, stream):
        with torch.cuda.stream(stream):
            s = _Server("fp8" if seed % 2 else "bf16", 40, 8, 2, "128", 16, 400, 100, seed=seed)
            outs = []
            for step in range(12):
                new = [(37 * b + step) % 60 if step == 0 else 1 for b in range(40)]
                plan = s.plan(i32(new), sum(new))
                q, _ = s.store(s.tokens(sum(new)), plan)
                if step:
                    outs.append(s.attend(q))
            stream.synchronize()
            return outs

    alone = [run(seed, torch.cuda.Stream()) for seed in range(4)]
    with ThreadPoolExecutor(4) as pool:
        for _ in range(3):
            together = list(pool.map(run, range(4), [torch.cuda.Stream() for _ in range(4)]))
            assert all(torch.equal(x, y) for a, b in zip(alone, together) for x, y in zip(a, b))
    assert zyfa_check_errors() == 0
