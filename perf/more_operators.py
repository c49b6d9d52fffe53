"""Measured cases of the 4-bit paged key/value cache: quantising a step's tokens as they are written, reading tokens of the
cache back as dense rows, and the attention of one new token per request over the 4-bit pages.

The cache holds e2m1 codes, two channels a byte (channel 2i in the low half), and one e4m3 scale for each 16 channels of a
token and head; a value is code * scale * descale.  ``store`` rotates a step's queries and keys, writes keys and values
as codes and scales and reads what it wrote back as e4m3 rows, which is also how its values can be returned.  ``read``
gathers runs of tokens of several requests, of any cache type, as bf16 or e4m3 rows.  ``decode`` lets one bf16 query per
request attend over its pages.  Head shapes are those of the prefill attention.

``run`` computes each operator in elementary torch operations, or with ``own`` through the package.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
SHAPES = {"64": (64, 64), "128": (128, 128), "mla": (192, 128)}
GROUP = 16                                                                   # channels of a scale


# ------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one chat session takes one more token: latency of every layer and token
        dict(name="store_token", op="store", B=1, N=1, cached=1000, H=32, H_kv=8, shape="128", axes=1, interleaved=False,
             page=64, dense=False, pad=0, strided=False),
        # a decode batch of the 192/128 head shape: 64 rotary channels behind 128 plain ones, interleaved pairs
        dict(name="store_decode_mla", op="store", B=128, N=1, cached=2000, H=8, H_kv=8, shape="mla", axes=1,
             interleaved=True, page=16, dense=False, pad=5, strided=False),
        # a text and image prompt: three position axes, an odd number of tokens, slices of one QKV projection, padded rows
        dict(name="store_image_4099", op="store", B=1, N=4099, cached=0, H=16, H_kv=4, shape="64", axes=3,
             interleaved=False, page=48, dense=False, pad=29, strided=True),
        # a long prompt: cache, and the rotated rows as the bf16 prefill reads them, from the same pass
        dict(name="store_prompt_32k", op="store", B=1, N=32768, cached=0, H=32, H_kv=8, shape="128", axes=1,
             interleaved=False, page=64, dense=True, pad=0, strided=True),
        # a short context read back before a prompt that begins with it: latency
        dict(name="read_prefix_700", op="read", B=1, lo=700, hi=700, H_kv=8, shape="128", kind="e2m1", page=16, fp8=False,
             late=False, pad=0, per_head=False),
        # ragged contexts of a batch, from a place within each on, as e4m3 rows for the FP8 prefill; rows padded for a graph
        dict(name="read_ragged_fp8", op="read", B=37, lo=1, hi=9001, H_kv=4, shape="mla", kind="e2m1", page=64, fp8=True,
             late=True, pad=117, per_head=True),
        # a document's context read back whole: the bandwidth of the pass
        dict(name="read_document_128k", op="read", B=1, lo=131072, hi=131072, H_kv=8, shape="128", kind="e2m1", page=64,
             fp8=False, late=False, pad=0, per_head=False),
        # one short context, a small model: latency
        dict(name="decode_b1_256", op="decode", B=1, lo=256, hi=256, H=2, H_kv=2, shape="64", page=16, lse=False,
             per_head=False, outliers=False),
        # one long context: few rows, so the cache's length has to fill the card
        dict(name="decode_b1_32k", op="decode", B=1, lo=32768, hi=32768, H=32, H_kv=8, shape="128", page=64, lse=False,
             per_head=False, outliers=True),
        # a ragged batch, 16 query heads on each key head: the arithmetic of a byte counts
        dict(name="decode_b64_ragged_g16", op="decode", B=64, lo=1, hi=8192, H=64, H_kv=4, shape="128", page=32, lse=True,
             per_head=False, outliers=False),
        # the 192/128 head shape without shared key heads: one query row per key
        dict(name="decode_b9_mla", op="decode", B=9, lo=3001, hi=15000, H=16, H_kv=16, shape="mla", page=16, lse=False,
             per_head=True, outliers=False),
        # a large serving batch: the bandwidth of the cache read
        dict(name="decode_b128", op="decode", B=128, lo=513, hi=16384, H=32, H_kv=8, shape="128", page=64, lse=False,
             per_head=False, outliers=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["store", "read", "decode", "decode"])
    page = rng.choice([8, 16, 32, 48, 64, 128])
    shape = rng.choice(list(SHAPES))
    H_kv = rng.choice([1, 2, 3, 4, 8, 16])
    group = 1 if shape == "mla" else rng.choice([1, 2, 3, 4, 7, 8, 16])
    while group * H_kv > 64:
        group = max(1, group // 2)
    d_qk, d_v = SHAPES[shape]
    if op == "store":
        most = min(20000, 32768 * 48 * 128 // ((group + 2) * H_kv * d_qk))
        B = rng.choice([1, _log(rng, 2, 192)])
        return dict(op="store", B=B, N=1 if rng.random() < 0.3 else _log(rng, 1, max(1, most // B)), cached=_log(rng, 1, 4000) - 1,
                    H=group * H_kv, H_kv=H_kv, shape=shape, axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.5, page=page,
                    dense=rng.random() < 0.3, pad=rng.choice([0, _log(rng, 1, 100)]), strided=rng.random() < 0.5)
    B = _log(rng, 1, 192)
    most = int(2.0e9 / (B * H_kv * (d_qk + d_v)))
    if op == "read":
        hi = _log(rng, 1, min(65536, most // 8))
        return dict(op="read", B=B, lo=_log(rng, 1, hi), hi=hi, H_kv=H_kv, shape=shape, kind=rng.choice(["e2m1", "e2m1", "e4m3", "bf16"]),
                    page=page, fp8=rng.random() < 0.5, late=rng.random() < 0.5, pad=rng.choice([0, _log(rng, 1, 300)]),
                    per_head=rng.random() < 0.5)
    hi = _log(rng, 1, min(65536, most))
    return dict(op="decode", B=B, lo=_log(rng, 1, hi), hi=hi, H=group * H_kv, H_kv=H_kv, shape=shape, page=page,
                lse=rng.random() < 0.5, per_head=rng.random() < 0.5, outliers=rng.random() < 0.3)


# ------------------------------------------------------------------------------------------------
# inputs

def _spread(lo, hi, n):
    """n whole numbers spread evenly over the logarithm from lo to hi: their sum is the case's, not the seed's."""
    if n == 1:
        return [hi]
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** (i / (n - 1)))))) for i in range(n)]


def _runs(case):
    """(first token, number of tokens) of each request's run that a read takes."""
    ends = _spread(case["lo"], case["hi"], case["B"])
    first = [n // 3 if case["late"] and i % 2 else 0 for i, n in enumerate(ends)]
    return first, [n - f for n, f in zip(ends, first)]


def _table(lens, page, gen, spare):
    """A block table for requests of these lengths: random pages, each used once, and their number."""
    need = (lens + page - 1) // page
    total = int(need.sum())
    order = torch.randperm(total + spare, generator=gen, device=DEV, dtype=torch.int32)
    width = max(1, int(need.max()))
    first = torch.cumsum(need, 0) - need
    col = torch.arange(width, device=DEV)
    have = col[None, :] < need[:, None]
    at = (first[:, None] + col[None, :]).clamp(max=total + spare - 1)
    return torch.where(have, order[at], torch.full_like(at, -1, dtype=torch.int32)), total + spare


def _quantise(z):
    """Codes (two a byte) and e4m3 scales of values over their descale: a block's scale is its largest magnitude over 6."""
    blocks = z.unflatten(-1, (-1, GROUP))
    scale = (blocks.abs().amax(-1) * (1.0 / 6.0)).clamp(max=448.0).to(E4M3)
    s = scale.float()
    x = blocks * torch.where(s > 0, 1.0 / s, torch.zeros_like(s))[..., None]
    a = x.abs()
    code = (a > 0.25).byte()                                                 # ties go to the even code
    for limit, tie_up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= limit) if tie_up else (a > limit)
    code = (code | ((x < 0).byte() << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _values(codes, scales):
    """code * scale, exact in 32 bits."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    e, half = (c >> 1) & 3, (c & 1).float() * 0.5
    x = torch.where(e == 0, half, (1.0 + half) * 0.5 * torch.bitwise_left_shift(torch.ones_like(e), e).float())
    x = torch.where(c > 7, -x, x)
    return (x.unflatten(-1, (-1, GROUP)) * scales.float()[..., None]).flatten(-2)


def _cache(x, kind, descale):
    """Values [pages, page, H_kv, D] as a cache of this kind: (codes or values, scales or None)."""
    if kind == "bf16":
        return x.to(torch.bfloat16), None
    x = x / descale
    return _quantise(x) if kind == "e2m1" else (x.clamp_(-448.0, 448.0).to(E4M3), None)


def _positive(n, gen, about):
    return (torch.rand((n,), generator=gen, device=DEV) * 0.4 + 0.8) * about


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)
    op, page, H_kv, (d_qk, d_v) = case["op"], case["page"], case["H_kv"], SHAPES[case["shape"]]
    i32 = dict(dtype=torch.int32, device=DEV)
    if op == "store":
        B, N, H, pad, axes = case["B"], case["N"], case["H"], case["pad"], case["axes"]
        cached = (case["cached"] - torch.arange(B, device=DEV) % 7).clamp(min=0)  # some begin, some end a page
        table, pages = _table(cached + N, page, gen, 3)
        rows = B * N + pad
        sizes = [H * d_qk, H_kv * d_qk, H_kv * d_v]
        if case["strided"]:                                                  # slices of one projection's rows
            x = torch.randn((rows, sum(sizes)), generator=gen, device=DEV).to(torch.bfloat16)
            parts = torch.split(x, sizes, dim=1)
        else:
            parts = [torch.randn((rows, n), generator=gen, device=DEV).to(torch.bfloat16) for n in sizes]
        q, k, v = (t.unflatten(1, (h, d)) for t, h, d in zip(parts, (H, H_kv, H_kv), (d_qk, d_qk, d_v)))
        place = (cached[:, None] + torch.arange(N, device=DEV)[None, :]).flatten()
        request = torch.arange(B, device=DEV).repeat_interleave(N)
        slots = table[request, place // page].long() * page + place % page
        slots = torch.cat([slots, torch.full((pad,), -1, dtype=torch.int64, device=DEV)])
        place = torch.cat([place, torch.zeros((pad,), dtype=torch.int64, device=DEV)])
        far = torch.randint(0, 131072, (1,), generator=gen, device=DEV)
        positions = (place + far)[None, :].repeat(axes, 1)
        if axes > 1:                                                         # image patches: rows and columns of a grid
            positions[1], positions[-1] = far + place // 61, far + place % 61
        rot = 64 if case["shape"] == "mla" else d_qk
        inv = (10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)).to(torch.float32)
        third = rot // 2 // axes
        blank = lambda *s, d=torch.uint8: torch.zeros(s, dtype=d, device=DEV)  # noqa: E731
        state = dict(case=case, q=q, k=k, v=v, slots=slots, positions=positions.to(torch.int32), inv=inv,
                     pairs=[rot // 2 - third * (axes - 1)] + [third] * (axes - 1), offset=d_qk - rot,
                     kc=blank(pages, page, H_kv, d_qk // 2), vc=blank(pages, page, H_kv, d_v // 2),
                     ks=blank(pages, page, H_kv, d_qk // GROUP).view(E4M3), vs=blank(pages, page, H_kv, d_v // GROUP).view(E4M3),
                     kd=_positive(1, gen, 0.002), vd=_positive(1, gen, 0.002), q_out=blank(rows, H, d_qk, d=torch.bfloat16),
                     k_dense=None, v_dense=None, k_out=blank(rows, H_kv, d_qk).view(E4M3), v_out=blank(rows, H_kv, d_v).view(E4M3),
                     ko=_positive(1, gen, 1 / 64), vo=_positive(1, gen, 1 / 64), table=table, starts=cached.to(torch.int32),
                     cu=torch.arange(0, B * N + 1, N, **i32))
        if case["dense"]:
            state.update(k_dense=blank(rows, H_kv, d_qk, d=torch.bfloat16), v_dense=blank(rows, H_kv, d_v, d=torch.bfloat16))
        return state
    B = case["B"]
    mix = torch.randperm(B, generator=gen, device=DEV)
    kind = case.get("kind", "e2m1")
    if op == "read":
        starts, counts = (torch.tensor(x, device=DEV)[mix] for x in _runs(case))
        lens = starts + counts
    else:
        lens = torch.tensor(_spread(case["lo"], case["hi"], B), device=DEV)[mix]
    table, pages = _table(lens, page, gen, 2)
    n = (B * H_kv if op == "decode" else H_kv) if case["per_head"] else 1
    about = {"e2m1": 0.002, "e4m3": 1 / 64, "bf16": 1.0}[kind]
    kd, vd = (_positive(n, gen, about) if kind != "bf16" else None for _ in range(2))
    k = torch.randn((pages, page, H_kv, d_qk), generator=gen, device=DEV)
    q = torch.randn((B, case["H"], d_qk), generator=gen, device=DEV) if op == "decode" else None
    if op == "decode" and case["outliers"]:                                  # a few strong channels, as captured activations have
        loud = torch.randperm(d_qk, generator=gen, device=DEV)[:4]
        q[..., loud] *= 4.0
        k[..., loud] *= 4.0
    kc, ks = _cache(k, kind, about)
    del k
    vc, vs = _cache(torch.randn((pages, page, H_kv, d_v), generator=gen, device=DEV), kind, about)
    state = dict(case=case, kc=kc, vc=vc, ks=ks, vs=vs, table=table, kd=kd, vd=vd)
    if op == "decode":
        state.update(q=q.to(torch.bfloat16), lens=lens.to(torch.int32))
        return state
    cu = torch.cat([torch.zeros((1,), dtype=torch.int64, device=DEV), torch.cumsum(counts, 0)])
    rows = int(cu[-1]) + case["pad"]
    out = lambda d: torch.zeros((rows, H_kv, d), dtype=torch.uint8, device=DEV).view(E4M3) if case["fp8"] else torch.zeros(  # noqa: E731
        (rows, H_kv, d), dtype=torch.bfloat16, device=DEV)
    ko, vo = (_positive(1, gen, 1 / 64) if case["fp8"] else None for _ in range(2))
    state.update(starts=starts.to(torch.int32), cu=cu.to(torch.int32), k_out=out(d_qk), v_out=out(d_v), ko=ko, vo=vo)
    return state


# ------------------------------------------------------------------------------------------------
# the passes

def run(state):
    op = state["case"]["op"]
    if own:
        return {"store": _own_store, "read": _own_read, "decode": _own_decode}[op](state)
    return {"store": _plain_store, "read": _plain_read, "decode": _plain_decode}[op](state)


def _own_store(s):
    from fp8_causal_prefill_gb300 import Rope, paged_read, rope_paged_store
    rope = Rope(s["inv"], axis_pairs=s["pairs"], offset=s["offset"], interleaved=s["case"]["interleaved"])
    rope_paged_store(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["positions"], rope, k_scales=s["ks"], v_scales=s["vs"],
                     k_descale=s["kd"], v_descale=s["vd"], q_out=s["q_out"], k_out=s["k_dense"], v_out=s["v_dense"])
    paged_read(s["kc"], s["vc"], s["table"], s["cu"], starts=s["starts"], k_scales=s["ks"], v_scales=s["vs"], k_descale=s["kd"],
               v_descale=s["vd"], k_out_descale=s["ko"], v_out_descale=s["vo"], k_out=s["k_out"], v_out=s["v_out"])
    return _stored(s)


def _own_read(s):
    from fp8_causal_prefill_gb300 import paged_read
    return paged_read(s["kc"], s["vc"], s["table"], s["cu"], starts=s["starts"], k_scales=s["ks"], v_scales=s["vs"], k_descale=s["kd"],
                      v_descale=s["vd"], k_out_descale=s["ko"], v_out_descale=s["vo"], k_out=s["k_out"], v_out=s["v_out"])


def _own_decode(s):
    from fp8_causal_prefill_gb300 import paged_decode_attn
    return paged_decode_attn(s["q"], s["kc"], s["vc"], s["table"], s["lens"], k_scales=s["ks"], v_scales=s["vs"], k_descale=s["kd"],
                             v_descale=s["vd"], return_lse=s["case"]["lse"])


def _stored(s):
    out = dict(q=s["q_out"], k=s["k_out"], v=s["v_out"])
    if s["case"]["dense"]:
        out.update(k_dense=s["k_dense"], v_dense=s["v_dense"])
    return out


def _plain_rotate(x, angle, offset, interleaved):
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    rot = 2 * cos.shape[-1]
    x = x.float()
    part = x[..., offset: offset + rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., : rot // 2], part[..., rot // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    both = torch.stack([a, b], dim=-1).flatten(-2) if interleaved else torch.cat([a, b], dim=-1)
    return torch.cat([x[..., :offset], both, x[..., offset + rot:]], dim=-1)


def _bits(x):
    return x.view(torch.uint8) if x.dtype == E4M3 else x


def _plain_store(s):
    case = s["case"]
    axis = torch.repeat_interleave(torch.arange(len(s["pairs"]), device=DEV), torch.tensor(s["pairs"], device=DEV))
    angle = s["positions"].double()[axis].T * s["inv"].double()
    n = case["B"] * case["N"]                                                # the rows behind are padding: left as they were
    q, k = (_plain_rotate(s[x][:n], angle[:n], s["offset"], case["interleaved"]) for x in "qk")
    v = s["v"][:n].float()
    s["q_out"][:n] = q.to(torch.bfloat16)
    for x, d, codes, scales in ((k, "kd", "kc", "ks"), (v, "vd", "vc", "vs")):
        c, sc = _quantise(x * (1.0 / s[d]))
        s[codes].flatten(0, 1)[s["slots"][:n]] = c
        _bits(s[scales]).flatten(0, 1)[s["slots"][:n]] = _bits(sc)
    if case["dense"]:
        s["k_dense"][:n], s["v_dense"][:n] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    _plain_read(s)
    return _stored(s)


def _plain_read(s):
    cu, rows = s["cu"].long(), s["k_out"].shape[0]
    page, H_kv = s["kc"].shape[1], s["kc"].shape[2]
    n = torch.arange(rows, device=DEV)
    b = torch.searchsorted(cu[1:], n, right=True).clamp(max=cu.numel() - 2)
    place = (s["starts"].long()[b] + n - cu[b]).clamp(min=0)
    page_at = s["table"][b, (place // page).clamp(max=s["table"].shape[1] - 1)].long().clamp(min=0)
    real = (n < cu[-1])[:, None, None]
    for codes, scales, d, o, out in (("kc", "ks", "kd", "ko", "k_out"), ("vc", "vs", "vd", "vo", "v_out")):
        x = _bits(s[codes])[page_at, place % page]
        x = _values(x, _bits(s[scales])[page_at, place % page].view(E4M3)) if s[scales] is not None else x.view(s[codes].dtype).float()
        f = torch.ones((1,), device=DEV) if s[d] is None else s[d]
        f = f if s[o] is None else f * (1.0 / s[o])
        y = x * f.reshape(1, -1, 1)
        y = y.to(torch.bfloat16) if s[out].dtype == torch.bfloat16 else y.clamp(-448.0, 448.0).to(E4M3)
        s[out].copy_(torch.where(real, _bits(y), _bits(s[out])).view(s[out].dtype))
    return s["k_out"], s["v_out"]


def _plain_decode(s):
    q, table, lens = s["q"], s["table"], s["lens"].long()
    B, H, d_qk = q.shape
    page, H_kv = s["kc"].shape[1], s["kc"].shape[2]
    t = torch.arange(table.shape[1] * page, device=q.device)
    slot = table[:, t // page].long().clamp(min=0) * page + t % page         # [B, L]
    k, v = (_values(s[c], s[x]).flatten(0, 1)[slot].permute(0, 2, 1, 3) for c, x in (("kc", "ks"), ("vc", "vs")))
    dk, dv = (d.reshape(-1, H_kv) if d.numel() > 1 else d.reshape(1, 1) for d in (s["kd"], s["vd"]))
    x = torch.matmul(q.float().unflatten(1, (H_kv, -1)), k.transpose(2, 3)) * (dk / math.sqrt(d_qk))[:, :, None, None]
    x = x.masked_fill((t[None, :] >= lens[:, None])[:, None, None, :], float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    out = (torch.matmul(p, v) / total * dv[:, :, None, None]).flatten(1, 2).to(torch.bfloat16)
    if s["case"]["lse"]:
        return out, (top + torch.log(total)).squeeze(-1).flatten(1, 2)
    return out


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits

def _held_bytes(values, kind):
    return values * {"e2m1": 9 / 16, "e4m3": 1, "bf16": 2}[kind]             # half a byte and a sixteenth of a scale


def work(case):
    d_qk, d_v = SHAPES[case["shape"]]
    H_kv, page = case["H_kv"], case["page"]
    if case["op"] == "store":
        n, q, kv = case["B"] * case["N"], case["H"] * d_qk, H_kv * (d_qk + d_v)
        rot = 64 if case["shape"] == "mla" else d_qk
        back = _held_bytes(kv, "e2m1") + kv + 4 / page                       # read again, as e4m3 rows
        return {"bytes": n * (2 * (q + kv) + 2 * q + _held_bytes(kv, "e2m1") + (2 * kv if case["dense"] else 0) + 8 + 4 * case["axes"] + back)
                + 2 * rot + 12 * case["B"], "flops": 3 * n * (case["H"] + H_kv) * rot}
    if case["op"] == "read":
        n, kv = sum(_runs(case)[1]), H_kv * (d_qk + d_v)
        return {"bytes": n * (_held_bytes(kv, case["kind"]) + kv * (1 if case["fp8"] else 2) + 4 / page) + 12 * case["B"], "flops": n * kv}
    tokens = sum(_spread(case["lo"], case["hi"], case["B"]))
    rows = case["B"] * case["H"] * (2 * d_qk + 2 * d_v + (4 if case["lse"] else 0))
    return {"bytes": _held_bytes(tokens * H_kv * (d_qk + d_v), "e2m1") + rows + 4 * (tokens // page + case["B"]),
            "flops": 2 * tokens * case["H"] * (d_qk + d_v)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "read": _exact_read, "decode": _exact_decode}[case["op"]](s)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nearest(x, values):
    """The nearest of ascending `values` to each x >= 0, in 64 bits."""
    at = torch.tensor(values, dtype=torch.float64, device=x.device)
    return at[torch.bucketize(x, (at[1:] + at[:-1]) / 2)]


def _as_held(y, descale):
    """What a 4-bit cache holds of y, over the descale: the nearest code times the block's scale."""
    z = y.double().unflatten(-1, (-1, GROUP)) / descale.double()
    finite = torch.arange(127, dtype=torch.uint8, device=y.device).view(E4M3).double().tolist()
    scale = _nearest(z.abs().amax(-1, keepdim=True) / 6.0, finite)
    x = z / torch.where(scale > 0, scale, torch.ones_like(scale))
    return (torch.sign(x) * _nearest(x.abs(), E2M1) * scale).flatten(-2)


def _exact_store(s):
    case = s["case"]
    n = case["B"] * case["N"]
    turn = torch.zeros((n, len(s["inv"])), dtype=torch.float64, device=DEV)
    at = 0
    for axis, m in enumerate(s["pairs"]):
        turn[:, at: at + m] = torch.outer(s["positions"][axis, :n].double(), s["inv"][at: at + m].double())
        at += m
    phase = torch.polar(torch.ones_like(turn), turn)[:, None, :]             # each pair as one complex number
    half, lo = len(s["inv"]), s["offset"]

    def rotated(x):
        y = x[:n].double().clone()
        if case["interleaved"]:
            first, second = slice(lo, lo + 2 * half, 2), slice(lo + 1, lo + 2 * half, 2)
        else:
            first, second = slice(lo, lo + half), slice(lo + half, lo + 2 * half)
        z = torch.complex(y[..., first], y[..., second]) * phase
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def rows(y, like):
        z = torch.zeros(like.shape, dtype=torch.float64, device=DEV)
        z[:n] = y
        return z

    k, v = rotated(s["k"]), s["v"][:n].double()
    back = lambda y, d, o: (_as_held(y, s[d]) * (s[d].double() / s[o].double())).clamp(-448.0, 448.0)  # noqa: E731
    out = dict(q=rows(rotated(s["q"]), s["q_out"]), k=rows(back(k, "kd", "ko"), s["k_out"]), v=rows(back(v, "vd", "vo"), s["v_out"]))
    if case["dense"]:
        out.update(k_dense=rows(k, s["k_dense"]), v_dense=rows(v, s["v_dense"]))
    return out


def _decoded(codes, scales):
    """The values of a cache, over its descale, in 64 bits."""
    if scales is None:
        return codes.double()
    both = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=codes.device)
    x = torch.stack([both[(codes & 15).long()], both[(codes >> 4).long()]], dim=-1).flatten(-2)
    return x * scales.double().repeat_interleave(GROUP, -1)


def _exact_read(s):
    case, page, outs = s["case"], s["case"]["page"], []
    first, cu = s["starts"].tolist(), s["cu"].tolist()
    for codes, scales, d, o, like in (("kc", "ks", "kd", "ko", "k_out"), ("vc", "vs", "vd", "vo", "v_out")):
        z = torch.zeros(s[like].shape, dtype=torch.float64, device=DEV)
        for b in range(case["B"]):
            t = torch.arange(first[b], first[b] + cu[b + 1] - cu[b], device=DEV)
            at = s["table"][b, t // page].long()
            x = _decoded(_bits(s[codes])[at, t % page].view(s[codes].dtype), None if s[scales] is None else _bits(s[scales])[at, t % page].view(E4M3))
            if s[d] is not None:
                x = x * s[d].double().reshape(1, -1, 1)
            if s[o] is not None:
                x = (x / s[o].double()).clamp(-448.0, 448.0)
            z[cu[b]: cu[b + 1]] = x
        outs.append(z)
    return tuple(outs)


def _exact_decode(s):
    """One request at a time, its pages one after another, in 64 bits."""
    case = s["case"]
    (B, H, d_qk), H_kv = s["q"].shape, case["H_kv"]
    group = H // H_kv
    outs, lses = [], []
    for b in range(B):
        n = int(s["lens"][b])
        pages = s["table"][b, : -(-n // case["page"])].long()
        k, v = (_decoded(s[c][pages], _bits(s[x])[pages].view(E4M3)).flatten(0, 1)[:n] for c, x in (("kc", "ks"), ("vc", "vs")))
        dk, dv = (d.double().reshape(-1, H_kv)[b] if d.numel() > 1 else d.double().repeat(H_kv) for d in (s["kd"], s["vd"]))
        k, v = k * dk[None, :, None], v * dv[None, :, None]
        q = s["q"][b].double()
        x = torch.stack([q[h] @ k[:, h // group].T for h in range(H)]) / d_qk ** 0.5
        lses.append(torch.logsumexp(x, -1))
        w = torch.softmax(x, -1)
        outs.append(torch.stack([w[h] @ v[:, h // group] for h in range(H)]))
    out, lse = torch.stack(outs), torch.stack(lses)
    return (out, lse) if case["lse"] else out
