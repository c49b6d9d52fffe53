"""GPU tests of the 4-bit paged cache at its edges: any bytes in the cache, addresses far apart or shared, waits that run out, several
callers, first calls inside a capture."""
import ctypes
import math
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import test_paged4_gpu as base
from _paged4_util import make_cache4, raw
from _paged_util import E4M3, SHAPES, bits, poisoned, random_table, random_values
from fp8_causal_prefill_gb300 import api, paged_decode_attn, paged_decode_workspace_bytes, paged_read, rope_paged_store, zyfa_check_errors
from oracle import paged4 as Q

pytestmark = pytest.mark.gpu

i32, f32 = base.i32, base.f32
FAR = (1 << 31) + 4096                                                          # bytes between pages


def _random(cache, scales, seed):
    """Codes of any bits, and scales about 1 with a sign."""
    rng = np.random.default_rng(seed)
    raw(cache).copy_(torch.from_numpy(rng.integers(0, 256, tuple(cache.shape), dtype=np.uint8)))
    raw(scales).copy_(torch.from_numpy((rng.integers(0x2C, 0x40, tuple(scales.shape)) | rng.integers(0, 2, tuple(scales.shape)) << 7).astype(np.uint8)))


def _any_bytes(shape, rng, about=None):
    """Any codes, and any scales that are no NaN."""
    codes = rng.integers(0, 256, (*shape[:-1], shape[-1] // 2), dtype=np.uint8)
    scales = (rng.integers(0, 127, (*shape[:-1], shape[-1] // 16)) | rng.integers(0, 2, (*shape[:-1], shape[-1] // 16)) << 7).astype(np.uint8)
    return codes, scales


# ------------------------------------------------------------------------------------------------
# what the cache holds need not come from the store

@pytest.mark.parametrize("shape", ["64", "128", "mla"])
@pytest.mark.parametrize("page", [7, 16])
def test_any_codes_and_scales_are_read_and_attended_to(monkeypatch, shape, page):
    monkeypatch.setattr(base, "random_codes", _any_bytes)
    for out in ("bf16", "fp8"):
        base._read_case("e2m1", out, shape, 3, base.RAGGED, page=page, per_head=1, seed=1)
    base._decode_case(shape, [1, 40, 333, 0], 6, 2, page=page, seed=2, per_head=True)
    base._decode_case(shape, [130, 64], 24, 2, page=page, seed=3)


@pytest.mark.parametrize("group", [1, 3, 9, 16, 17])
def test_decode_of_queries_that_requests_share(group):
    # q_batch_stride 0: one token's queries for every request
    H_kv, page, lens = 2, 16, [100, 0, 33]
    caches = make_cache4(16, page, H_kv, "128")
    for c, s, seed in ((caches[0], caches[2], 1), (caches[1], caches[3], 2)):
        _random(c, s, seed)
    table, _ = random_table(lens, page, np.random.default_rng(0))
    table = torch.from_numpy(table % 16).cuda()
    q = random_values((1, group * H_kv, 128), "bf16", np.random.default_rng(3))
    shared, one_each = (base._attend(x, caches, table, i32(lens)) for x in (q.expand(3, -1, -1), q.repeat(3, 1, 1)))
    assert torch.equal(shared[0], one_each[0]) and torch.equal(shared[1], one_each[1]) and zyfa_check_errors() == 0


# ------------------------------------------------------------------------------------------------
# addresses

@pytest.mark.parametrize("shape,H_kv", [("128", 2), ("64", 1), ("mla", 4)])
def test_offsets_beyond_32_bits(shape, H_kv):
    """Pages more than 2 GiB apart, of codes and of scales: stored, read back and attended to as in a dense cache."""
    page, pages = 16, 4
    sizes = [w // n for n in (2, 16) for w in SHAPES[shape]]
    buffers = [torch.empty(FAR * (pages - 1) + page * H_kv * n, dtype=torch.uint8, device="cuda") for n in (sizes[0], sizes[2])]
    near = make_cache4(pages, page, H_kv, shape)
    far = list(near)
    for at, buffer in zip((0, 2), buffers):
        far[at] = buffer.as_strided(near[at].shape, (FAR, H_kv * sizes[at], sizes[at], 1))
        far[at].fill_(0x7F)
    far[1], far[3] = near[1].clone(), near[3].clone()
    rng = np.random.default_rng(0)
    n, lens, table = 60, i32([60]), i32([[3, 0, 1, 2]])
    k, v = (random_values((n, H_kv, d), "bf16", rng) for d in SHAPES[shape])
    t = torch.arange(n, device="cuda")
    slots = table[0].long()[t // page] * page + t % page
    q = random_values((1, 2 * H_kv, SHAPES[shape][0]), "bf16", rng)
    got = []
    for caches in (far, near):
        rope_paged_store(None, k, v, caches[0], caches[1], slots, k_scales=caches[2], v_scales=caches[3])
        rows = paged_read(caches[0], caches[1], table, i32([0, n]), n, k_scales=caches[2], v_scales=caches[3])
        got.append([*rows, *base._attend(q, caches, table, lens)])
    assert zyfa_check_errors() == 0 and all(torch.equal(x, y) for x, y in zip(*got)) and bool(torch.isfinite(got[0][2]).all())
    assert all(torch.equal(x, y) for x, y in zip(far, near))
    far[0] = far[0].clone()                                                     # only the scales far apart
    assert torch.equal(base._attend(q, far, table, lens)[0], got[0][2])


@pytest.mark.parametrize("shape,group", [("128", 2), ("64", 12), ("mla", 1)])
def test_caches_that_repeat_a_head_or_a_page(shape, group):
    """Strides of 0, which only reading allows."""
    one = make_cache4(3, 16, 1, shape)
    for c, s, seed in ((one[0], one[2], 1), (one[1], one[3], 2)):
        _random(c, s, seed)
    table, lens, cu = i32([[0, 1, 2], [2, 1, 0]]), i32([40, 47]), i32([0, 40, 87])
    q = random_values((2, 4 * group, SHAPES[shape][0]), "bf16", np.random.default_rng(4))
    heads = [t.expand(-1, -1, 4, -1) for t in one]
    full = [t.contiguous() for t in heads]
    page = [t[:1].expand(3, -1, -1, -1) for t in full]
    same = [t[:1].repeat(3, 1, 1, 1) for t in full]
    for a, b in ((heads, full), (page, same)):
        x, y = base._attend(q, a, table, lens)[0], base._attend(q, b, table, lens)[0]
        assert float((x - y).abs().max()) <= 2.0 ** -7 * float(y.abs().max())   # tiles may differ: each within its roundings
        x, y = (paged_read(c[0], c[1], table, cu, 87, k_scales=c[2], v_scales=c[3]) for c in (a, b))
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    for t in (0, 2):
        with pytest.raises(RuntimeError):                                       # rows that would be written twice
            caches = [heads[i] if i == t else full[i] for i in range(4)]
            k, v = (torch.zeros((1, 4, d), dtype=torch.bfloat16, device="cuda") for d in SHAPES[shape])
            rope_paged_store(None, k, v, caches[0], caches[1], torch.zeros(1, dtype=torch.int64, device="cuda"), k_scales=caches[2], v_scales=caches[3])
    assert zyfa_check_errors() == 0


@pytest.mark.parametrize("out", ["bf16", "fp8"])
@pytest.mark.parametrize("kind", ["e2m1", "fp8", "bf16"])
def test_read_rows_aligned_to_16_bytes_only(kind, out):
    caches = make_cache4(4, 16, 3, "64") if kind == "e2m1" else None
    if caches:
        for c, s, seed in ((caches[0], caches[2], 1), (caches[1], caches[3], 2)):
            _random(c, s, seed)
    else:
        rng = np.random.default_rng(5)
        caches = (random_values((4, 16, 3, 64), kind, rng), random_values((4, 16, 3, 64), kind, rng), None, None)
    table, cu, n = i32([[2, 0, 3], [1, 1, 1]]), i32([0, 45, 50]), 50
    kw = dict(k_scales=caches[2], v_scales=caches[3])
    got = []
    for shift in (0, 16):
        size = n * 3 * 64
        rows = []
        for _ in range(2):
            whole = poisoned((size + 64,), out)
            at = shift // whole.element_size()
            assert whole.data_ptr() % 32 == 0
            rows.append((whole, whole[at:at + size].view(n, 3, 64), at))
        paged_read(caches[0], caches[1], table, cu, k_out=rows[0][1], v_out=rows[1][1], **kw)
        for whole, _, at in rows:
            rest = torch.cat([whole[:at], whole[at + size:]]).float()
            assert bool(torch.isnan(rest).all())
        got.append([bits(r[1]).clone() for r in rows])
    assert all(torch.equal(x, y) for x, y in zip(*got)) and zyfa_check_errors() == 0


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("H_kv", [1, 2, 3, 5, 6, 7])
def test_pages_of_8_tokens_and_numbers_of_heads(layout, H_kv):
    # boxes of the fewest tokens, and blocks whose last heads are missing
    for shape, group in (("64", 1), ("128", 10), ("mla", 3)):
        base._decode_case(shape, [77, 8, 130], group * H_kv, H_kv, page=8, layout=layout, seed=H_kv, per_head=True)


# ------------------------------------------------------------------------------------------------
# waits that run out

def _structs(caches):
    k, v, ks, vs = caches
    return (api.PagedCache(k.data_ptr(), v.data_ptr(), api.ZYFA_DTYPE_E2M1, k.shape[1], k.shape[0], k.shape[2], 2 * k.shape[3], 2 * v.shape[3],
                           *k.stride()[:3], *v.stride()[:3]),
            api.PagedScales(ks.data_ptr(), vs.data_ptr(), *ks.stride()[:3], *vs.stride()[:3]))


@pytest.mark.parametrize("page", [16, 5])                                       # boxes, and pieces
@pytest.mark.parametrize("shape,H,H_kv,lens,width", [
    ("128", 32, 8, [64, 0, 17], 80), ("128", 32, 8, [900, 0, 17, 400], 1000),   # whole requests; split and joined
    ("64", 2, 1, [900, 5], 1000), ("128", 32, 2, [300, 70], 1000),              # warps that would meet; two sets of heads
    ("mla", 20, 2, [300], 1000)])
def test_decode_without_its_loads_times_out_and_the_next_call_is_right(shape, H, H_kv, lens, width, page):
    width = -(-width // page)
    d_qk, d_v = SHAPES[shape]
    B = len(lens)
    table, pages = random_table(lens, page, np.random.default_rng(1), width)
    table = torch.from_numpy(table).cuda()
    caches = make_cache4(pages, page, H_kv, shape)
    for c, s, seed in ((caches[0], caches[2], 1), (caches[1], caches[3], 2)):
        _random(c, s, seed)
    q, lens_t = random_values((B, H, d_qk), "bf16", np.random.default_rng(2)), i32(lens)
    ws = torch.empty(paged_decode_workspace_bytes(B, H, H_kv, d_v, width * page), dtype=torch.uint8, device="cuda")
    want, want_lse = base._attend(q, caches, table, lens_t, workspace=ws)
    out = torch.empty_like(want)
    cache, scales = _structs(caches)
    stream = torch.cuda.current_stream().cuda_stream
    st = api.load_library().zyfa_selftest_stalled_decode_e2m1(q.data_ptr(), q.stride(0), ctypes.byref(cache), ctypes.byref(scales), table.data_ptr(),
                                                              width, width, lens_t.data_ptr(), out.data_ptr(), B, H, ws.data_ptr(), ws.numel(), stream)
    assert st == 0
    assert zyfa_check_errors(stream) == 5 and zyfa_check_errors(stream) == 0    # ZYFA_ERR_TIMEOUT, read and cleared
    got, got_lse = base._attend(q, caches, table, lens_t, workspace=ws)
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)


# ------------------------------------------------------------------------------------------------
# several callers

def test_steps_of_several_threads_and_streams():
    """Threads that each run their own steps on their own stream get what they get alone."""
    def run(seed, stream):
        with torch.cuda.stream(stream):
            s = base._Server(30, 8, 2, 16, 40, 300, seed=seed)
            outs = []
            for step in range(8):
                new = [(37 * b + step) % 60 if step == 0 else 1 for b in range(30)]
                q, plan, _ = s.store(s.tokens(sum(new)), i32(new), sum(new))
                if step:
                    outs.append(s.attend(q))
            cu = i32(np.cumsum([0] + s.lens.tolist()))
            outs.extend(s.read(cu, int(cu[-1])))
            stream.synchronize()
            return outs

    alone = [run(seed, torch.cuda.Stream()) for seed in range(4)]
    with ThreadPoolExecutor(4) as pool:
        for _ in range(3):
            together = list(pool.map(run, range(4), [torch.cuda.Stream() for _ in range(4)]))
            assert all(torch.equal(x, y) for a, b in zip(alone, together) for x, y in zip(a, b))
    assert zyfa_check_errors() == 0


_FIRST_IN_CAPTURE = """
import torch
from fp8_causal_prefill_gb300 import Rope, paged_decode_attn, paged_plan, paged_read, rope_paged_store, zyfa_check_errors
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
n, page = 50, 16
x = [torch.randn(n, h, 128, device="cuda").bfloat16() for h in (8, 2, 2)]
kc, vc = (torch.zeros(6, page, 2, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
ks, vs = (torch.zeros(6, page, 2, 8, dtype=torch.uint8, device="cuda") for _ in range(2))
kw = dict(k_scales=ks, v_scales=vs)
table, lens, new, free, cursor = i32([[-1] * WIDTH]), i32([0]), i32([n]), i32([4, 1, 5, 0, 2]), i32([0])
rope = Rope(torch.rand(64, device="cuda"))
def step():
    plan = paged_plan(lens, new, table, free, cursor, page, n)
    q = rope_paged_store(*x, kc, vc, plan.slots, plan.positions, rope, **kw)
    return paged_decode_attn(q[n - 1:], kc, vc, table, plan.seq_lens, **kw), *paged_read(kc, vc, table, plan.cu_tokens, n, **kw)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in out]
kc.zero_(); vc.zero_(); ks.zero_(); vs.zero_(); table.fill_(-1)
for a, b in zip(step(), got):
    assert torch.equal(a, b) and bool((b != 0).any())
assert zyfa_check_errors() == 0
"""


@pytest.mark.parametrize("width", [4, 64])                                      # one launch, and two
def test_first_calls_of_a_process_inside_a_capture(width):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_IN_CAPTURE.replace("WIDTH", str(width))], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------------------------------------------
# refusals

def test_tensor_refusals():
    kc, vc, ks, vs = make_cache4(4, 16, 2, "128")
    kw = dict(k_scales=ks, v_scales=vs)
    q, table, lens = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device="cuda"), i32([[0]] * 3), i32([1] * 3)
    one = f32([1.0])
    attend = dict(q=q, k_cache=kc, v_cache=vc, block_table=table, seq_lens=lens, **kw)
    read = dict(k_cache=kc, v_cache=vc, block_table=table, cu_tokens=i32([0, 1, 2, 3]), max_tokens=3, **kw)
    kv = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    store = dict(q=q, k=kv, v=kv.clone(), k_cache=kc, v_cache=vc, slots=torch.arange(3, device="cuda"), **kw)
    caches = [dict(k_cache=kc.to(torch.bfloat16)), dict(v_cache=vc.view(E4M3)), dict(k_scales=ks.float()), dict(v_scales=vs[..., :4]), dict(k_scales=ks[:3]),
              dict(v_scales=vs.cpu()), dict(k_cache=kc[..., ::2]), dict(k_scales=None), dict(v_scales=None), dict(k_cache=kc[:, :8]),
              dict(k_cache=kc[:, :, :1]), dict(k_scales=ks.transpose(2, 3)), dict(k_scales=ks[..., 1:]), dict(k_cache=kc[..., 8:])]
    for call, a, more in (
            (paged_decode_attn, attend, [dict(q=q.to(E4M3)), dict(q=q.float()), dict(q=q[..., :64]), dict(q_descale=one), dict(k_descale=f32([1, 1, 1])),
                                         dict(k_descale=one.cpu()), dict(out=q.float())]),
            (paged_read, read, [dict(dtype=torch.float16), dict(dtype=torch.uint8), dict(max_tokens=None), dict(max_tokens=-1), dict(k_out=kv), dict(v_out=kv),
                                dict(k_out=kv, v_out=kv), dict(k_out=kv, v_out=kv[:2]), dict(k_out=kv.float(), v_out=kv), dict(k_out_descale=one),
                                dict(k_out=kv, v_out=kv.to(E4M3)), dict(cu_tokens=i32([0, 1, 2])), dict(cu_tokens=torch.arange(4, device="cuda")),
                                dict(cu_tokens=i32([])), dict(starts=i32([0, 0])), dict(starts=lens.long()), dict(starts=lens.cpu()),
                                dict(k_descale=f32([1, 1, 1])), dict(dtype=E4M3, v_out_descale=f32([1, 1, 1]))]),
            (rope_paged_store, store, [dict(q_descale=one), dict(k_descale=f32([1, 1, 1])), dict(q_out=torch.empty(q.shape, dtype=E4M3, device="cuda")),
                                       dict(k_out=torch.empty(kv.shape, dtype=E4M3, device="cuda")), dict(k=kv.float()), dict(v=None), dict(k=kv[:2])])):
        call(**a)
        for bad in caches + more:
            with pytest.raises((TypeError, ValueError, RuntimeError)):
                call(**{**a, **bad})
    assert zyfa_check_errors() == 0


def test_stored_codes_do_not_depend_on_the_layout():
    """The same tokens in caches of every layout hold the same bytes, whichever way keys take through the store."""
    rng = np.random.default_rng(0)
    x = [random_values((77, h, d), "bf16", rng) for h, d in ((6, 192), (3, 192), (3, 128))]
    slots = torch.from_numpy(rng.permutation(96)[:77]).cuda()
    want = None
    for layout in ("nhd", "hnd", "row", "joint"):
        caches = make_cache4(6, 16, 3, "mla", layout)
        rope_paged_store(*x, caches[0], caches[1], slots, k_scales=caches[2], v_scales=caches[3])
        got = [raw(t).contiguous() for t in caches]
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    codes, scales = Q.quantise(x[1].double().cpu().numpy(), 1.0)
    at = slots.cpu().numpy()
    assert np.array_equal(want[0].cpu().numpy()[at // 16, at % 16], codes) and np.array_equal(want[2].cpu().numpy()[at // 16, at % 16], scales)
    assert math.prod(want[0].shape) > 0 and zyfa_check_errors() == 0
