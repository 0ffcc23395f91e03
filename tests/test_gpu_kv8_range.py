"""Attention and votes over 8-bit caches at the ends of the range: logits far past fp32's integers, tokens that
tie there, all logits far below zero."""
import math

import numpy as np
import pytest
import torch

from oracle import kv8 as O8
from query_aware_sparse_decode_b200 import tb as TB

from harness import mask_from_sets
from test_gpu_kv8 import DT, MODES, Case, dev, host, random_sets

pytestmark = pytest.mark.gpu


def one_hot_case(fmt, dtype, up, sign, L=(700, 90)):
    """Logits without any rounding before the scale: query h has one element, +-1 at dim h, and the keys hold j 2^up
    (j one of 64, 72 .. 120: four significant bits, exact in both formats) there.  V blocks differ by up to 2^24."""
    gs = 4
    c = Case(fmt, dtype, B=2, Hq=8, Hkv=2, D=128 if dtype == "bf16" else 64, max_len=768, seed=up)
    n = max(L)
    k = np.zeros((2, 2, n, c.D))
    k[..., :gs] = sign * c.rng.integers(8, 16, size=(2, 2, n, gs)) * 8.0 * 2.0 ** up
    v = c.rng.normal(size=k.shape) * np.exp2(np.repeat(c.rng.integers(-12, 12, size=(n + 15) // 16), 16)[:n])[:, None]
    c.append(L, k=k, v=v)
    q = np.zeros((2, 8, c.D))
    for h in range(8):
        q[:, h, h % gs] = 1.0 if h < 6 or sign < 0 else -1.0
    return c, q


@pytest.mark.parametrize("mode", ["head", "dense"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("up", [4, 13, 20, 27, 40, 100])
@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("int8", "bf16"), ("e4m3", "f32"), ("int8", "f32")])
def test_attention_with_large_logits(fmt, dtype, up, sign, mode):
    """Equal keys have equal logits, bit for bit, and others are at least 2^up apart: the softmax is even over the
    largest ones, and its error is that of the weights (fp16: half a step, 2^-11) and of the output's type."""
    c, q = one_hot_case(fmt, dtype, up, sign)
    sets, mask = c.all_tokens(), None
    if mode == "head":
        sets = random_sets(c, c.Hq, 0.3, empty={(1, 2)})
        mask = mask_from_sets(sets, c.B, c.Hq, c.max_len)
    out = torch.full((c.B, c.Hq, c.D), 9.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((c.B, c.Hq), 9.0, device="cuda")
    c.ctx.sparse_attn(0, dev(q, dtype), mask, MODES[mode], out, lse)
    torch.cuda.synchronize()
    assert c.ctx.check_status() == 0
    half, w = (2.0 ** -8, 2.0 ** -11) if dtype == "bf16" else (2.0 ** -24, 0.0)
    for b in range(c.B):
        for h in range(c.Hq):
            o, z, weight, _ = O8.attend(q[b, h], c.val["k"][b, h // c.gs], c.val["v"][b, h // c.gs], sets[b, h])
            # z's terms: the product with log2e / sqrt(D) and its own rounding, log2 and the way back, half a step each
            assert float(lse[b, h]) == z if z == -math.inf else abs(float(lse[b, h]) - z) <= 8 * 2.0 ** -24 * abs(z) + 2e-6
            tol = half * np.abs(o) + (w + 1e-5) * weight + 1e-36
            assert np.all(np.abs(host(out)[b, h] - o) <= tol), f"b{b} h{h}"


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("up", [4, 20, 27, 40, 100])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_votes_with_large_logits(fmt, up, sign):
    c, q = one_hot_case(fmt, "bf16", up, sign)
    votes = torch.full((c.B, c.max_len), 3.0, device="cuda")
    c.ctx.softvote_scores(0, dev(q, "bf16"), votes)
    torch.cuda.synchronize()
    for b, L in enumerate(c.lens):
        ref, slack = np.zeros(L), np.zeros(L)
        for h in range(c.Hq):
            a = c.val["k"][b, h // c.gs, :L] @ q[b, h] / math.sqrt(c.D)
            p = np.exp(a - a.max())
            ref += p / p.sum()
            # a logit below the largest: three roundings (log2e / sqrt(D), its product with the scale, the logit) of
            # each of the two, half a step 2^-24 each, move their distance; equal ones move together
            slack += np.where(a < a.max(), p / p.sum() * 6 * 2.0 ** -24 * np.abs(a).max(), 0.0)
        assert np.all(np.abs(host(votes)[b, :L] - ref) <= 4e-6 * ref + slack + 1e-30), f"b{b}"


@pytest.mark.parametrize("mode", ["head", "dense"])
@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("int8", "bf16"), ("e4m3", "f32")])
def test_large_queries_beside_large_scales(fmt, dtype, mode):
    """Keys with 2^120 in a dimension that the queries, 2^60 elsewhere, do not read: the products are zero in those
    blocks and ordinary in the others, though query times scale passes fp32."""
    c = Case(fmt, dtype, B=1, Hq=4, Hkv=1, D=64, max_len=256, seed=7)
    k = c.rng.normal(size=(1, 1, 90, 64)) * 2.0 ** -60
    k[0, 0, [20, 70], 5] = 2.0 ** 120, -1.5 * 2.0 ** 119
    c.append([90], k=k, v=c.rng.normal(size=k.shape))
    q = c.rng.normal(size=(1, 4, 64)) * 2.0 ** 60
    q[..., 5] = 0.0
    q = dev(q, dtype)
    sets, mask = c.all_tokens(), None
    if mode == "head":
        sets = random_sets(c, c.Hq, 0.5)
        mask = mask_from_sets(sets, 1, c.Hq, c.max_len)
    out, lse = torch.zeros((1, 4, 64), dtype=DT[dtype], device="cuda"), torch.zeros((1, 4), device="cuda")
    c.ctx.sparse_attn(0, q, mask, MODES[mode], out, lse)
    votes = torch.zeros((1, 256), device="cuda")
    if dtype == "bf16":
        c.ctx.softvote_scores(0, q, votes)
    torch.cuda.synchronize()
    assert c.ctx.check_status() == 0
    c.check_attention(q, sets, out, lse)
    if dtype == "bf16":
        ref, slack = np.zeros(90), 0.0
        for h in range(4):
            a = c.val["k"][0, 0, :90] @ host(q)[0, h] / 8.0
            p = np.exp(a - a.max())
            ref += p / p.sum()
            slack = max(slack, 72 * 2.0 ** -24 * float((np.abs(c.val["k"][0, 0, :90]) @ np.abs(host(q)[0, h])).max()) / 8.0)
        assert np.all(np.abs(host(votes)[0, :90] - ref) <= (2 * slack + 4e-6) * ref + 1e-30)


@pytest.mark.parametrize("mode", ["head", "dense"])
@pytest.mark.parametrize("spread", [0, 30, 70])
@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("int8", "bf16"), ("int8", "f32")])
def test_scales_that_are_not_powers_of_two(fmt, dtype, spread, mode):
    """Caches that another program quantised: any positive finite scales.  log2 of a V scale is off by at most 3 units
    of its last place (2^-16 for |log2| in [64, 128)), its sums with the references by half a step each: a weight is off
    by less than 2^-14 of itself, beside the rest."""
    c = Case(fmt, dtype, B=2, Hq=8, Hkv=2, max_len=512, seed=spread)
    c.append((300, 37))
    torch.cuda.synchronize()
    for x, t, up in (("k", c.ks, 0), ("v", c.vs, spread)):
        f = c.rng.uniform(1, 2, size=t.shape) * np.exp2(c.rng.integers(-up, up + 1, size=t.shape))
        t.copy_(torch.from_numpy(host(t) * f).float())
        codes, s = c.cached()["kv".index(x)]
        c.val[x] = codes * np.repeat(s, 16, axis=2)[..., None]
    q = dev(c.rng.normal(size=(2, 8, c.D)), dtype)
    sets, mask = c.all_tokens(), None
    if mode == "head":
        sets = random_sets(c, c.Hq, 0.4, empty={(1, 0)})
        mask = mask_from_sets(sets, 2, c.Hq, c.max_len)
    out, lse = torch.zeros((2, 8, c.D), dtype=DT[dtype], device="cuda"), torch.zeros((2, 8), device="cuda")
    c.ctx.sparse_attn(0, q, mask, MODES[mode], out, lse)
    ko, vo = (torch.zeros((2, 2, 300, c.D), dtype=DT[dtype], device="cuda") for _ in range(2))
    c.ctx.read_kv(0, 0, 300, ko, vo)
    torch.cuda.synchronize()
    half, w = (2.0 ** -8, 2.0 ** -11) if dtype == "bf16" else (2.0 ** -24, 0.0)
    for b in range(2):
        for h in range(8):
            o, z, weight, dot = O8.attend(host(q)[b, h], c.val["k"][b, h // c.gs], c.val["v"][b, h // c.gs], sets[b, h])
            dl = (c.D + 8) * 2.0 ** -24 * dot / math.sqrt(c.D)
            tol = half * np.abs(o) + (w + 2.0 ** -14 + 2 * dl + 1e-5) * weight + 1e-36
            assert np.all(np.abs(host(out)[b, h] - o) <= tol), f"b{b} h{h}"
            got = float(lse[b, h])
            assert got == z if z == -math.inf else abs(got - z) <= dl + 2e-6 * (1 + abs(z)), f"lse b{b} h{h}"
        L = c.lens[b]
        for x, t in (("k", ko), ("v", vo)):
            assert np.all(np.abs(host(t)[b, :, :L] - c.val[x][b, :, :L]) <= half * np.abs(c.val[x][b, :, :L]))
