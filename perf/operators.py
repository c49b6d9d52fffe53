"""Measured cases of the paged serving operators: the page plan of a step, the rotation and store of its
new tokens, and the attention of one new token per request over the paged cache.

A serving step runs the three in this order.  ``plan`` turns request lengths into cache pages, slots and
positions; ``store`` rotates the step's queries and keys and writes keys and values into their slots;
``decode`` lets one query token per request attend over its pages.  Head shapes, group sizes and the two
cache types (e4m3 and bf16) are those of the prefill attention beside them.

``run`` computes each operator in elementary torch operations, or with ``own`` through the package.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
SHAPES = {"64": (64, 64), "128": (128, 128), "mla": (192, 128)}


# ------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one request takes one more token: what a single chat session pays in latency for every token
        dict(name="plan_step_b1", op="plan", B=1, page=16, cached=1000, decode=1.0, chunk=1, pad=0),
        # a full decode batch: one token each, contexts of very different lengths
        dict(name="plan_decode_b256", op="plan", B=256, page=64, cached=32768, decode=1.0, chunk=1, pad=0),
        # a mixed step of a busy server: half the requests bring a prompt chunk; token rows padded for a graph
        dict(name="plan_mixed_b96", op="plan", B=96, page=32, cached=16384, decode=0.5, chunk=2048, pad=777),
        # one token of one request, FP8 cache, all channels rotated: latency
        dict(name="store_token_fp8", op="store", N=1, H=32, H_kv=8, shape="128", fp8=True, axes=1, interleaved=False,
             page=64, dense=False, pad=0, strided=False),
        # a decode batch of the 192/128 head shape: 64 rotary channels behind 128 plain ones, interleaved pairs
        dict(name="store_decode_mla_bf16", op="store", N=128, H=16, H_kv=16, shape="mla", fp8=False, axes=1,
             interleaved=True, page=16, dense=False, pad=5, strided=False),
        # a text and image prompt: three position axes, an odd number of tokens, slices of one QKV projection
        dict(name="store_image_bf16_4099", op="store", N=4099, H=16, H_kv=4, shape="64", fp8=False, axes=3,
             interleaved=False, page=48, dense=False, pad=29, strided=True),
        # a long prompt quantised for the FP8 prefill: cache and dense tensors from the same pass
        dict(name="store_prompt_fp8_32k", op="store", N=32768, H=32, H_kv=8, shape="128", fp8=True, axes=1,
             interleaved=False, page=64, dense=True, pad=0, strided=True),
        # one short context, a small model: latency
        dict(name="decode_b1_256_bf16", op="decode", B=1, lo=256, hi=256, H=2, H_kv=2, shape="64", fp8=False, page=16,
             lse=False, per_head=False, outliers=False),
        # one long context, FP8 cache: few rows, so the cache's length has to fill the card
        dict(name="decode_b1_32k_fp8", op="decode", B=1, lo=32768, hi=32768, H=32, H_kv=8, shape="128", fp8=True,
             page=64, lse=False, per_head=False, outliers=True),
        # a ragged batch in BF16 with small pages: contexts from one token to thousands
        dict(name="decode_b64_ragged_bf16", op="decode", B=64, lo=1, hi=8192, H=32, H_kv=8, shape="128", fp8=False,
             page=16, lse=True, per_head=False, outliers=False),
        # the 192/128 head shape without shared key heads: one query row per key
        dict(name="decode_b9_mla_fp8", op="decode", B=9, lo=3001, hi=15000, H=16, H_kv=16, shape="mla", fp8=True,
             page=32, lse=False, per_head=True, outliers=False),
        # a large serving batch, FP8 cache: the bandwidth of the cache read
        dict(name="decode_b128_fp8", op="decode", B=128, lo=513, hi=16384, H=32, H_kv=8, shape="128", fp8=True, page=64,
             lse=False, per_head=False, outliers=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["plan", "store", "decode", "decode"])
    page = rng.choice([8, 16, 32, 48, 64, 128])
    if op == "plan":
        B = _log(rng, 1, 512)
        return dict(op="plan", B=B, page=page, cached=_log(rng, 1, 40000), decode=rng.choice([0.0, 0.5, 0.9, 1.0]),
                    chunk=_log(rng, 1, max(1, 100000 // B)), pad=rng.choice([0, _log(rng, 1, 1000)]))
    shape = rng.choice(list(SHAPES))
    H_kv = rng.choice([1, 2, 3, 4, 8, 16])
    group = 1 if shape == "mla" else rng.choice([1, 2, 3, 4, 7, 8, 16])
    while group * H_kv > 64:
        group = max(1, group // 2)
    d_qk, d_v = SHAPES[shape]
    fp8 = rng.random() < 0.5
    if op == "store":
        most = 32768 * 48 * 128 // ((group + 2) * H_kv * d_qk)
        return dict(op="store", N=_log(rng, 1, min(20000, most)), H=group * H_kv, H_kv=H_kv, shape=shape, fp8=fp8,
                    axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.5, page=page, dense=rng.random() < 0.3,
                    pad=rng.choice([0, _log(rng, 1, 100)]), strided=rng.random() < 0.5)
    B = _log(rng, 1, 192)
    most = int(2.0e9 / (B * H_kv * (d_qk + d_v) * (1 if fp8 else 2)))
    hi = _log(rng, 1, min(65536, most))
    return dict(op="decode", B=B, lo=_log(rng, 1, hi), hi=hi, H=group * H_kv, H_kv=H_kv, shape=shape, fp8=fp8, page=page,
                lse=rng.random() < 0.5, per_head=fp8 and rng.random() < 0.5, outliers=rng.random() < 0.3)


# ------------------------------------------------------------------------------------------------
# inputs

def _spread(lo, hi, n):
    """n whole numbers spread evenly over the logarithm from lo to hi: their sum is the case's, not the seed's."""
    if n == 1:
        return [hi]
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** (i / (n - 1)))))) for i in range(n)]


def _plan_lengths(case):
    B = case["B"]
    cached = _spread(1, case["cached"], B)
    cached = [c - 1 if i % 7 == 0 else c for i, c in enumerate(cached)]      # some begin, some end a page
    steps = int(round(case["decode"] * B))
    new = [1] * steps + _spread(1, case["chunk"], B - steps) if B > steps else [1] * B
    return cached, new


def _decode_lengths(case):
    return _spread(case["lo"], case["hi"], case["B"])


def _pages_of(lens, page, gen, spare):
    """A block table for requests of these lengths: random pages, each used once, and the page order."""
    need = (lens + page - 1) // page
    total = int(need.sum())
    order = torch.randperm(total + spare, generator=gen, device=DEV, dtype=torch.int32)
    width = int(need.max())
    first = torch.cumsum(need, 0) - need
    col = torch.arange(width, device=DEV)
    have = col[None, :] < need[:, None]
    at = (first[:, None] + col[None, :]).clamp(max=total + spare - 1)
    table = torch.where(have, order[at], torch.full_like(at, -1, dtype=torch.int32))
    return table, order, total


def _codes(x):
    return x.mul_(64.0).clamp_(-448.0, 448.0).to(E4M3)


def _normal(shape, gen, fp8):
    """N(0, 1) values in the case's type; e4m3 codes carry a descale of 1/64."""
    x = torch.randn(shape, generator=gen, device=DEV)
    return _codes(x) if fp8 else x.to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)
    op = case["op"]
    if op == "plan":
        cached, new = (torch.tensor(x, device=DEV) for x in _plan_lengths(case))
        mix = torch.randperm(case["B"], generator=gen, device=DEV)
        cached, new = cached[mix], new[torch.randperm(case["B"], generator=gen, device=DEV)]
        page = case["page"]
        spare = int(((cached + new + page - 1) // page).sum())
        table, order, used = _pages_of(cached, page, gen, spare)
        width = -(-(max(_plan_lengths(case)[0]) + max(_plan_lengths(case)[1])) // page)
        wide = torch.full((case["B"], width), -1, dtype=torch.int32, device=DEV)
        wide[:, : table.shape[1]] = table[:, :width]
        return dict(case=case, cached=cached.to(torch.int32), new=new.to(torch.int32), table=wide, free=order,
                    cursor=torch.tensor([used], dtype=torch.int32, device=DEV), max_tokens=sum(_plan_lengths(case)[1]) + case["pad"])
    d_qk, d_v = SHAPES[case["shape"]]
    H, H_kv, fp8, page = case["H"], case["H_kv"], case["fp8"], case["page"]
    typ = E4M3 if fp8 else torch.bfloat16
    if op == "store":
        N, pad = case["N"], case["pad"]
        sizes = [H * d_qk, H_kv * d_qk, H_kv * d_v]
        rows = N + pad
        if case["strided"]:                                                  # slices of one projection's rows
            x = torch.randn((rows, sum(sizes)), generator=gen, device=DEV).to(torch.bfloat16)
            parts = torch.split(x, sizes, dim=1)
        else:
            parts = [torch.randn((rows, n), generator=gen, device=DEV).to(torch.bfloat16) for n in sizes]
        q, k, v = (t.unflatten(1, (h, d)) for t, h, d in zip(parts, (H, H_kv, H_kv), (d_qk, d_qk, d_v)))
        pages = (N + page - 1) // page + 3
        slots = torch.randperm(pages * page, generator=gen, device=DEV)[:N]
        if N > 64:                                                           # a prompt fills page after page
            order = torch.randperm(pages, generator=gen, device=DEV)
            t = torch.arange(N, device=DEV)
            slots = order[t // page] * page + t % page
        slots = torch.cat([slots, torch.full((pad,), -1, dtype=torch.int64, device=DEV)])
        axes = case["axes"]
        base = torch.randint(0, 131072, (1,), generator=gen, device=DEV)
        positions = (base + torch.arange(rows, device=DEV))[None, :].repeat(axes, 1)
        if axes > 1:                                                         # image patches: rows and columns of a grid
            positions[1] = base + torch.arange(rows, device=DEV) // 61
            positions[-1] = base + torch.arange(rows, device=DEV) % 61
        rot = 64 if case["shape"] == "mla" else d_qk
        inv = (10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)).to(torch.float32)
        third = rot // 2 // axes
        pairs = [rot // 2 - third * (axes - 1)] + [third] * (axes - 1)
        blank = lambda *s: torch.zeros(s, dtype=torch.uint8 if fp8 else torch.bfloat16, device=DEV).view(typ)  # noqa: E731
        descales = [torch.tensor([c / 64.0], device=DEV) if fp8 else None for c in (1.0, 0.9, 1.1)]
        state = dict(case=case, q=q, k=k, v=v, slots=slots, positions=positions.to(torch.int32), inv=inv, pairs=pairs,
                     offset=d_qk - rot, kc=blank(pages, page, H_kv, d_qk), vc=blank(pages, page, H_kv, d_v),
                     descales=descales, q_out=blank(rows, H, d_qk), k_out=None, v_out=None)
        if case["dense"]:
            state.update(k_out=blank(rows, H_kv, d_qk), v_out=blank(rows, H_kv, d_v))
        return state
    B = case["B"]
    lens = torch.tensor(_decode_lengths(case), device=DEV)[torch.randperm(B, generator=gen, device=DEV)]
    table, _, used = _pages_of(lens, page, gen, 2)
    q = torch.randn((B, H, d_qk), generator=gen, device=DEV)
    k = torch.randn((used + 2, page, H_kv, d_qk), generator=gen, device=DEV)
    if case["outliers"]:                                                     # a few strong channels, as captured activations have
        loud = torch.randperm(d_qk, generator=gen, device=DEV)[:4]
        q[..., loud] *= 4.0
        k[..., loud] *= 4.0
    q, k = (_codes(x) if fp8 else x.to(torch.bfloat16) for x in (q, k))
    v = _normal((used + 2, page, H_kv, d_v), gen, fp8)
    n = B * H_kv if case["per_head"] else 1
    descales = [torch.rand((n,), generator=gen, device=DEV) * 0.004 + 0.0136 if fp8 else None for _ in range(3)]
    return dict(case=case, q=q, kc=k, vc=v, table=table, lens=lens.to(torch.int32), descales=descales)


# ------------------------------------------------------------------------------------------------
# the passes

def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "store": _own_store, "decode": _own_decode}[op](state)
    return {"plan": _plain_plan, "store": _plain_store, "decode": _plain_decode}[op](state)


def _own_plan(s):
    from fp8_causal_prefill_gb300 import paged_plan
    p = paged_plan(s["cached"], s["new"], s["table"], s["free"], s["cursor"], page_size=s["case"]["page"],
                   max_tokens=s["max_tokens"])
    return dict(table=s["table"], seq_lens=p.seq_lens, cu_tokens=p.cu_tokens, positions=p.positions, slots=p.slots,
                cursor=p.cursor)


def _own_store(s):
    from fp8_causal_prefill_gb300 import Rope, rope_paged_store
    rope = Rope(s["inv"], axis_pairs=s["pairs"], offset=s["offset"], interleaved=s["case"]["interleaved"])
    rope_paged_store(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["positions"], rope,
                     q_descale=s["descales"][0], k_descale=s["descales"][1], v_descale=s["descales"][2],
                     q_out=s["q_out"], k_out=s["k_out"], v_out=s["v_out"])
    return _stored(s)


def _own_decode(s):
    from fp8_causal_prefill_gb300 import paged_decode_attn
    return paged_decode_attn(s["q"], s["kc"], s["vc"], s["table"], s["lens"], q_descale=s["descales"][0],
                             k_descale=s["descales"][1], v_descale=s["descales"][2], return_lse=s["case"]["lse"])


def _stored(s):
    out = dict(q=s["q_out"], k_cache=s["kc"], v_cache=s["vc"])
    if s["case"]["dense"]:
        out.update(k=s["k_out"], v=s["v_out"])
    return out


def _plain_plan(s):
    page, n_max = s["case"]["page"], s["max_tokens"]
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"]
    lens = cached + new
    had, has = (cached + page - 1) // page, (lens + page - 1) // page
    need = has - had
    first = torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    fresh = (col >= had[:, None]) & (col < has[:, None])
    at = (s["cursor"].long() + first[:, None] + col - had[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][at], table))
    ends = torch.cumsum(new, 0)
    t = torch.arange(n_max, device=table.device)
    b = torch.searchsorted(ends, t, right=True)
    real = b < lens.numel()
    b = b.clamp(max=lens.numel() - 1)
    pos = cached[b] + t - (ends - new)[b]
    pos = torch.where(real, pos, torch.zeros_like(pos))
    slots = table[b, pos // page].long() * page + pos % page
    cu = torch.cat([torch.zeros_like(ends[:1]), ends])
    return dict(table=table, seq_lens=lens.int(), cu_tokens=cu.int(), positions=pos.int(),
                slots=torch.where(real, slots, torch.full_like(slots, -1)), cursor=s["cursor"] + need.sum().int())


def _pair_angles(s):
    axis = torch.repeat_interleave(torch.arange(len(s["pairs"]), device=DEV), torch.tensor(s["pairs"], device=DEV))
    return s["positions"].double()[axis].T * s["inv"].double()               # [N, rot / 2]


def _plain_rotate(x, cos, sin, offset, interleaved):
    rot = 2 * cos.shape[-1]
    x = x.float()
    part = x[..., offset: offset + rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., : rot // 2], part[..., rot // 2:])
    c, d = cos[:, None, :], sin[:, None, :]
    a, b = a * c - b * d, a * d + b * c
    both = torch.stack([a, b], dim=-1).flatten(-2) if interleaved else torch.cat([a, b], dim=-1)
    return torch.cat([x[..., :offset], both, x[..., offset + rot:]], dim=-1)


def _plain_round(x, descale):
    if descale is None:
        return x.to(torch.bfloat16)
    return (x * (1.0 / descale)).clamp(-448.0, 448.0).to(E4M3)


def _bits(x):
    return x.view(torch.uint8) if x.dtype == E4M3 else x


def _plain_store(s):
    angle = _pair_angles(s)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    dq, dk, dv = s["descales"]
    turn = (cos, sin, s["offset"], s["case"]["interleaved"])
    q = _plain_round(_plain_rotate(s["q"], *turn), dq)
    k = _plain_round(_plain_rotate(s["k"], *turn), dk)
    v = _plain_round(s["v"].float(), dv)
    n = s["case"]["N"]                                                       # the rows behind are padding: left as they were
    slots = s["slots"][:n]
    _bits(s["q_out"])[:n] = _bits(q)[:n]
    _bits(s["kc"]).flatten(0, 1)[slots] = _bits(k)[:n]
    _bits(s["vc"]).flatten(0, 1)[slots] = _bits(v)[:n]
    if s["case"]["dense"]:
        _bits(s["k_out"])[:n] = _bits(k)[:n]
        _bits(s["v_out"])[:n] = _bits(v)[:n]
    return _stored(s)


def _plain_decode(s):
    q, kc, vc, table, lens = s["q"], s["kc"], s["vc"], s["table"], s["lens"].long()
    B, H, d_qk = q.shape
    page, H_kv = kc.shape[1], kc.shape[2]
    most = table.shape[1] * page
    t = torch.arange(most, device=q.device)
    slot = table[:, t // page].long().clamp(min=0) * page + t % page         # [B, L]
    k = _bits(kc).flatten(0, 1)[slot].view(kc.dtype).float().permute(0, 2, 1, 3)
    v = _bits(vc).flatten(0, 1)[slot].view(vc.dtype).float().permute(0, 2, 1, 3)
    dq, dk, dv = (torch.ones((1, 1), device=q.device) if d is None else d.reshape(-1, H_kv) if d.numel() > 1 else d.reshape(1, 1)
                  for d in s["descales"])
    scale = (dq * dk / math.sqrt(d_qk))[:, :, None, None]
    x = torch.matmul(q.float().unflatten(1, (H_kv, -1)), k.transpose(2, 3)) * scale
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

def work(case):
    if case["op"] == "plan":
        cached, new = _plan_lengths(case)
        fresh = sum(new) // case["page"]                                     # read from the pool, written to the table
        return {"bytes": 12 * (sum(new) + case["pad"]) + 16 * case["B"] + 8 * fresh + 12, "flops": 0}
    d_qk, d_v = SHAPES[case["shape"]]
    H, H_kv, es = case["H"], case["H_kv"], 1 if case["fp8"] else 2
    if case["op"] == "store":
        N, q, k, v = case["N"], H * d_qk, H_kv * d_qk, H_kv * d_v
        rot = 64 if case["shape"] == "mla" else d_qk
        written = q + (k + v) * (2 if case["dense"] else 1)
        return {"bytes": N * (2 * (q + k + v) + es * written + 8 + 4 * case["axes"]) + 2 * rot, "flops": 3 * N * (H + H_kv) * rot}
    tokens = sum(_decode_lengths(case))
    cache = tokens * H_kv * (d_qk + d_v) * es
    rows = case["B"] * H * (d_qk * es + 2 * d_v + (4 if case["lse"] else 0))
    return {"bytes": cache + rows + 4 * (tokens // case["page"] + case["B"]), "flops": 2 * tokens * H * (d_qk + d_v)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "store": _exact_store, "decode": _exact_decode}[case["op"]](s)


def _exact_plan(s):
    """Whole numbers: nothing to say about rounding."""
    return None


def _exact_store(s):
    case, out = s["case"], {}
    turn = torch.zeros((s["positions"].shape[1], len(s["inv"])), dtype=torch.float64, device=DEV)
    at = 0
    for axis, n in enumerate(s["pairs"]):
        turn[:, at: at + n] = torch.outer(s["positions"][axis].double(), s["inv"][at: at + n].double())
        at += n
    phase = torch.polar(torch.ones_like(turn), turn)[:, None, :]             # each pair as one complex number
    half, lo = len(s["inv"]), s["offset"]

    def rotated(x):
        y = x.double().clone()
        if case["interleaved"]:
            first, second = slice(lo, lo + 2 * half, 2), slice(lo + 1, lo + 2 * half, 2)
        else:
            first, second = slice(lo, lo + half), slice(lo + half, lo + 2 * half)
        z = torch.complex(y[..., first], y[..., second]) * phase
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def held(y, descale):
        return y if descale is None else (y / descale.double()).clamp(-448.0, 448.0)

    n = case["N"]
    q, k, v = (held(y, d) for y, d in zip((rotated(s["q"]), rotated(s["k"]), s["v"].double()), s["descales"]))
    for name, y, like in (("q", q, s["q_out"]), ("k", k, s["k_out"]), ("v", v, s["v_out"])):
        if like is not None:
            z = torch.zeros(like.shape, dtype=torch.float64, device=DEV)
            z[:n] = y[:n]
            out[name] = z
    for name, y, like in (("k_cache", k, s["kc"]), ("v_cache", v, s["vc"])):
        z = torch.zeros(like.shape, dtype=torch.float64, device=DEV)
        z.view(-1, *like.shape[2:])[s["slots"][:n]] = y[:n]
        out[name] = z
    return out


def _exact_decode(s):
    """One request at a time, its pages one after another, in 64 bits."""
    case = s["case"]
    (B, H, d_qk), H_kv, d_v = s["q"].shape, s["kc"].shape[2], s["vc"].shape[3]
    group = H // H_kv
    outs, lses = [], []
    for b in range(B):
        n = int(s["lens"][b])
        pages = s["table"][b, : -(-n // case["page"])].long()
        k = _bits(s["kc"])[pages].view(s["kc"].dtype).double().reshape(-1, H_kv, d_qk)[:n]
        v = _bits(s["vc"])[pages].view(s["vc"].dtype).double().reshape(-1, H_kv, d_v)[:n]
        q = s["q"][b].double()
        for d, name in zip(s["descales"], "qkv"):
            if d is not None:
                f = d.double().reshape(-1, H_kv)[b] if d.numel() > 1 else d.double().repeat(H_kv)
                if name == "q":
                    q = q * f.repeat_interleave(group)[:, None]
                elif name == "k":
                    k = k * f[None, :, None]
                else:
                    v = v * f[None, :, None]
        x = torch.stack([q[h] @ k[:, h // group].T for h in range(H)]) / d_qk ** 0.5
        lses.append(torch.logsumexp(x, -1))
        w = torch.softmax(x, -1)
        outs.append(torch.stack([w[h] @ v[:, h // group] for h in range(H)]))
    out, lse = torch.stack(outs), torch.stack(lses)
    return (out, lse) if case["lse"] else out
