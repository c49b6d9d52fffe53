"""GPU tests of single-token attention where scores are turned around or far from 0: descales below 0, and a few equal keys beyond all
others by more than fp32 resolves next to them."""
import math

import numpy as np
import pytest
import torch

from _paged4_util import fill4, make_cache4
from _paged_util import E4M3, SHAPES, decode_tolerance, f64, fill_tokens, make_cache, random_table, random_values
from fp8_causal_prefill_gb300 import paged_decode_attn, zyfa_check_errors
from oracle import paged as P
from oracle import paged4 as Q

pytestmark = pytest.mark.gpu


class _Cache:
    """A paged cache of any type, filled request by request with the nearest values that it holds; `rows` are those, in 64 bits."""

    def __init__(self, kind, shape, lens, H_kv, page, width, rng):
        self.kind, self.rows, self.lens = kind, ([], []), lens
        self.table, pages = random_table(lens, page, rng, width)
        self.slots = [self.table[b, np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page for b, n in enumerate(lens)]
        if kind == "e2m1":
            kc, vc, ks, vs = make_cache4(pages, page, H_kv, shape)
            self.caches, self.scales = (kc, vc), dict(k_scales=ks, v_scales=vs)
        else:
            self.caches, self.scales = make_cache(pages, page, H_kv, shape, kind), {}

    def put(self, which, b, x):
        cache = self.caches[which]
        if self.kind == "e2m1":
            codes, scales = Q.quantise(x, 1.0)
            fill4(cache, self.scales["v_scales" if which else "k_scales"], self.slots[b], codes, scales)
            held = Q.held(codes, scales)
        else:
            t = torch.from_numpy(x).float().to(E4M3 if self.kind == "fp8" else torch.bfloat16).cuda()
            fill_tokens(cache, torch.as_tensor(self.slots[b], device="cuda"), t)
            held = f64(t)
        self.rows[which].append(held)

    def attend(self, q, of, scale, **kw):
        """Row b of q attends over the tokens that request of[b] was filled with (requests may share pages)."""
        table, lens = (torch.from_numpy(np.array(x, dtype=np.int32)).cuda() for x in (self.table[of], [self.lens[i] for i in of]))
        out, lse = paged_decode_attn(q, *self.caches, table, lens, scale, return_lse=True, **self.scales, **kw)
        assert zyfa_check_errors() == 0
        return f64(out), f64(lse)


# 64 and 128 channels with one and two sets of 8 query heads, and heads that are not shared; the tokens of a tile.
FORMS = [("64", 4, 1, 128), ("64", 12, 1, 128), ("128", 8, 2, 64), ("128", 24, 2, 64), ("mla", 3, 3, 32)]


def _ways(tile):
    """(lengths, width of the table, which request each row of q takes): requests as one block's work, parts of a tile each, and parts of
    many tiles."""
    lens = [5 * tile - 3, 1, 3 * tile + 5, 37]
    return [(lens, None, range(4)), (lens, 120, range(4)), ([1000, 1, 777, 64], 300, [0, 2, 3, 1, 0, 2] * 40)]


@pytest.mark.parametrize("per_head", [0, 1, 3])
@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("shape,H,H_kv,tile", FORMS)
@pytest.mark.parametrize("kind", ["e2m1", "fp8"])
def test_descales_below_zero(kind, shape, H, H_kv, tile, page, per_head):
    """A descale's sign turns the order of a row's scores around (K) or its output (V)."""
    rng = np.random.default_rng(page + per_head)
    d_qk, d_v = SHAPES[shape]
    for lens, width, of in _ways(tile):
        c, B = _Cache(kind, shape, lens, H_kv, page, width, rng), len(of)
        for b, n in enumerate(lens):
            c.put(0, b, rng.standard_normal((n, H_kv, d_qk)) * 64.0)
            c.put(1, b, rng.standard_normal((n, H_kv, d_v)) * 64.0)
        q = random_values((B, H, d_qk), "fp8" if kind == "fp8" else "bf16", rng)
        n = {0: 1, 1: B * H_kv, 3: H_kv}[per_head]
        sign = rng.choice([-1.0, 1.0], (2, n))
        sign[0, 0] = -1.0
        ds = [torch.tensor((rng.random(n) + 0.5) / 64 * s, dtype=torch.float32, device="cuda") for s in sign]
        dq = torch.tensor([1 / 64], dtype=torch.float32, device="cuda").repeat(n) if kind == "fp8" else None
        out, lse = c.attend(q, of, None, q_descale=dq, k_descale=ds[0], v_descale=ds[1])
        dk, dv = (np.broadcast_to(f64(d).reshape(-1, H_kv) if n > 1 else f64(d), (B, H_kv)) for d in ds)
        q64, sc = f64(q) * (1 / 64 if kind == "fp8" else 1.0), d_qk ** -0.5
        for b in range(0, B, 1 + B // 20):
            for h in range(H):
                hk = h // (H // H_kv)
                k, v, f = c.rows[0][of[b]][:, hk] * dk[b, hk], c.rows[1][of[b]][:, hk], dv[b, hk]
                ref, ref_lse, w = P.decode_attention(q64[b, h], k, v * f, sc)
                tol, lse_tol = decode_tolerance(q64[b, h], k, v, sc, abs(f), ref, w, "fp8")
                # a query beside a 4-bit cache loses bits below 2^-28 of its row's largest channel: 2^-39 of that
                more = d_qk * 2.0 ** -39 * np.abs(q64[b, h]).max() * np.abs(k).max() * sc if kind == "e2m1" else 0.0
                assert np.all(np.abs(out[b, h] - ref) <= tol + 2 * more * (w @ np.abs(v)) * abs(f)), (width, b, h)
                assert abs(lse[b, h] - ref_lse) <= lse_tol + more + 2.0 ** -23 * abs(ref_lse), (width, b, h)
        assert np.isfinite(out).all() and np.isfinite(lse).all()


# Levels of the loud channel, which e4m3 and bf16 hold; what e2m1 blocks hold of them is as far apart
LEVELS = {"e2m1": np.array([1.0, 2.0, 3.0, 4.0, 6.0]) * 448.0, "fp8": np.array([64.0, 128.0, 192.0, 256.0, 448.0]),
          "bf16": np.array([64.0, 128.0, 192.0, 256.0, 448.0])}


@pytest.mark.parametrize("away", [1, -1])
@pytest.mark.parametrize("exponent", [12, 20, 24, 25, 26, 27, 30, 40, 100])
@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("kind,kd", [("e2m1", 1.0), ("e2m1", -1.0), ("fp8", 1.0), ("fp8", -1.0), ("bf16", 1.0)])
def test_scores_far_from_zero(kind, kd, page, exponent, away):
    """The greatest scores lie at about `away` 2^exponent in units of log2 and the next ones a tenth of that and more away: all weight
    is on those keys, equal ones share it, wherever they are among tiles, parts and the other heads of a warp.

    Their weights and V are exact, so only a few sums and the quotient round (2^-24 each, 2^-22 in exp2) before out does to bf16 (2^-8).
    A score is an fp32 sum of D products, rounded three times after.  Rows of queries of 0 weigh all keys alike.
    """
    rng = np.random.default_rng(exponent + page)
    for i, (shape, H, H_kv, tile) in enumerate(FORMS):
        d_qk, d_v = SHAPES[shape]
        for lens, width, of in _ways(tile)[:2] if (i + exponent) % 3 else _ways(tile)[2:]:
            c, B, levels, winners = _Cache(kind, shape, lens, H_kv, page, width, rng), len(of), LEVELS[kind], []
            for b, n in enumerate(lens):
                k = rng.standard_normal((n, H_kv, d_qk))
                # three equal rows at the greatest level of channel 0, a few at each other one, most at the lowest
                level = np.zeros(n, dtype=np.int64)
                for j, t in enumerate(rng.permutation(n)[:12]):
                    level[t] = j % 4
                best = rng.permutation(n)[:3]
                level[best] = 4
                k[:, :, 0] = (levels[level] if away > 0 else -levels[4 - level])[:, None]
                k[best] = k[best[0]]
                c.put(0, b, k)
                c.put(1, b, rng.standard_normal((n, H_kv, d_v)) * 64.0)
                winners.append(best)
            q64 = rng.standard_normal((B, H, d_qk)) / 8.0
            q64[:, :, 0] = rng.integers(8, 16, (B, H)) * 8.0 * kd
            quiet = rng.random((B, H)) < 0.2
            q64[quiet] = 0.0
            q = torch.from_numpy(q64).float().to(E4M3 if kind == "fp8" else torch.bfloat16).cuda()
            q64 = f64(q)
            scale = float(np.float32(2.0 ** exponent * math.log(2.0) / (96.0 * levels[4 if away > 0 else 0])))
            out, lse = c.attend(q, of, scale, k_descale=None if kind == "bf16" else torch.tensor([kd], dtype=torch.float32, device="cuda"))
            for b in range(0, B, 1 + B // 10):
                for h in range(H):
                    hk, best = h // (H // H_kv), winners[of[b]]
                    k, v = c.rows[0][of[b]][:, hk], c.rows[1][of[b]][:, hk]
                    n, where = len(k), (shape, H, width, b, h)
                    if quiet[b, h]:
                        ref, ref_lse = v.mean(0), math.log(n)
                        tol = 2.0 ** -8 * np.abs(ref) * 1.01 + (n + 8) * 2.0 ** -23 * np.abs(v).mean(0)
                        lse_tol = (n + 8) * 2.0 ** -23 + 2.0 ** -19
                    else:
                        x = k @ q64[b, h] * kd * scale
                        rest = np.setdiff1d(np.arange(n), best)
                        assert len(rest) == 0 or x[best].min() - x[rest].max() > 0.05 * 2.0 ** exponent, where  # e^-200: no weight
                        ref, ref_lse = v[best].mean(0), x[best[0]] + math.log(len(best))
                        tol = 2.0 ** -8 * np.abs(ref) * 1.01 + 2.0 ** -20 * np.abs(v[best]).mean(0)
                        lse_tol = (d_qk + 8) * 2.0 ** -24 * (np.abs(k[best[0]]) @ np.abs(q64[b, h])) * scale + 2.0 ** -20
                    err = np.abs(out[b, h] - ref)
                    assert np.all(err <= tol), (where, out[b, h][:4], ref[:4])
                    assert abs(lse[b, h] - ref_lse) <= lse_tol, (where, float(lse[b, h]), ref_lse)
            assert np.isfinite(out).all() and np.isfinite(lse).all()


@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("shape,H,H_kv,tile", FORMS)
@pytest.mark.parametrize("kind", ["e2m1", "fp8", "bf16"])
def test_one_score_beyond_float32(kind, shape, H, H_kv, tile, page):
    """One key's score overflows, anywhere among the tiles; all others are 0.  +inf makes the row NaN, -inf weighs nothing."""
    rng = np.random.default_rng(page)
    d_qk, d_v = SHAPES[shape]
    for lens, width, of in _ways(tile):
        c, B = _Cache(kind, shape, lens, H_kv, page, width, rng), len(of)
        where = rng.integers(0, np.array(lens))
        for b, n in enumerate(lens):
            k = np.zeros((n, H_kv, d_qk))
            k[where[b], :, 0] = 448.0
            c.put(0, b, k)
            c.put(1, b, rng.standard_normal((n, H_kv, d_v)) * 64.0)
        sign = rng.choice([-1.0, 0.0, 1.0], (B, H))
        q = torch.zeros((B, H, d_qk))
        q[:, :, 0] = torch.from_numpy(sign * 448.0).float()
        q[:, :, 1] = 0.5
        out, lse = c.attend(q.to(E4M3 if kind == "fp8" else torch.bfloat16).cuda(), of, 1e37)
        for b in range(0, B, 1 + B // 20):
            for h in range(H):
                v, at = c.rows[1][of[b]][:, h // (H // H_kv)], where[of[b]]
                if sign[b, h] > 0:
                    assert np.isnan(out[b, h]).all() and np.isnan(lse[b, h]), (width, b, h)
                    continue
                v = np.delete(v, at, axis=0) if sign[b, h] < 0 else v
                if len(v) == 0:
                    assert (out[b, h] == 0).all() and lse[b, h] == -math.inf, (width, b, h)
                    continue
                # equal weights are exact; n of them and of their products are summed in fp32, then out rounds to bf16
                tol = 2.0 ** -8 * np.abs(v.mean(0)) * 1.01 + (len(v) + 8) * 2.0 ** -23 * np.abs(v).mean(0)
                assert np.all(np.abs(out[b, h] - v.mean(0)) <= tol), (width, b, h)
                assert abs(lse[b, h] - math.log(len(v))) <= (len(v) + 8) * 2.0 ** -23 + 2.0 ** -19, (width, b, h)
