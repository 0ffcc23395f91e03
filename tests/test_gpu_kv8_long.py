"""8-bit attention and votes where a CTA walks long chunks: batches with more (sequence, KV head) pairs than one wave
has CTAs, so that a warp lists several segments of 256 tokens, carries tokens from one to the next, takes dozens of
tiles and moves its softmax references many times.  The reference is the formula in float64 over the cached values
(read back; exact in bf16)."""
import math

import pytest
import torch

from query_aware_sparse_decode_b200 import tb as TB

from test_gpu_kv8 import MODES

pytestmark = pytest.mark.gpu
SHARES = (0.005, 0.05, 0.4, 1.0)


class Wide:
    """B sequences of 1025 to 4500 tokens (three of them short or empty), rows from `rows(generator, which, shape)`."""

    def __init__(self, fmt, gs, D, page=0, B=80, Hkv=8, max_len=4608, seed=0, rows=None):
        self.B, self.Hkv, self.gs, self.Hq, self.D, self.max_len, self.page = B, Hkv, gs, gs * Hkv, D, max_len, page
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.cfg = TB.make_config(1, B, self.Hq, Hkv, D, 16, 1, max_len, "bf16", 100, 4, 16)
        self.ctx = TB.Context(self.cfg)
        self.kimp = TB.kimp_cache(self.cfg)
        w = torch.zeros((D, 16), dtype=torch.bfloat16, device="cuda")
        code = TB.KV8_FORMATS[fmt][1]
        if page:
            n = B * max_len // page
            self.table = torch.randperm(n + 5, device="cuda", generator=self.g)[:n].reshape(B, -1).int()
            k, v = (torch.zeros((n + 5, Hkv, page, D), dtype=torch.int8, device="cuda").view(code) for _ in range(2))
            ks, vs = (torch.zeros((n + 5, Hkv, page // 16), device="cuda") for _ in range(2))
            self.ctx.bind_layer_kv8_paged(0, k, v, ks, vs, self.table, self.kimp, w)
        else:
            self.ctx.bind_layer_kv8(0, *TB.kv8_cache(self.cfg, fmt), self.kimp, w)
        rng = torch.Generator()
        rng.manual_seed(seed)
        self.lens = torch.randint(1025, min(4501, max_len + 1), (B,), generator=rng).tolist()
        self.lens[1], self.lens[5], self.lens[B - 1] = 0, 17, 1
        n = max(self.lens)
        shape = (B, Hkv, n, D)
        k, v = (rows(self.g, x, shape) if rows else torch.randn(shape, device="cuda", generator=self.g).bfloat16() for x in "kv")
        self.ctx.append_kv_rows(0, k, v, self.lens)
        self.k, self.v = torch.zeros_like(k), torch.zeros_like(v)
        self.ctx.read_kv(0, 0, n, self.k, self.v)
        torch.cuda.synchronize()
        assert self.ctx.check_status() == 0

    def mask(self, mode, share):
        """A bit mask with `share` of the tokens for each row, bits past the length among them, and one row empty."""
        rows = {"head": self.Hq, "group": self.Hkv, "shared": 1}[mode]
        bits = torch.rand((self.B, rows, self.max_len), device="cuda", generator=self.g) < share
        bits[2, rows - 1] = False
        weight = torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
        words = (bits.view(self.B, rows, -1, 32) * weight).sum(-1)
        return (words - (words >> 31 << 32)).to(torch.int32), bits

    def check(self, mode, share, q=None):
        if q is None:
            q = torch.randn((self.B, self.Hq, self.D), device="cuda", generator=self.g).bfloat16()
        mask, bits = (None, None) if mode == "dense" else self.mask(mode, share)
        out, lse = torch.full_like(q, 9.0), torch.full((self.B, self.Hq), 9.0, device="cuda")
        self.ctx.sparse_attn(0, q, mask, MODES[mode], out, lse)
        torch.cuda.synchronize()
        assert self.ctx.check_status() == 0
        for b, L in enumerate(self.lens):
            qq = q[b].double().view(self.Hkv, self.gs, self.D)
            k, v = self.k[b, :, :L].double(), self.v[b, :, :L].double()
            a = qq @ k.transpose(1, 2) / math.sqrt(self.D)
            dot = qq.abs() @ k.abs().transpose(1, 2)
            if bits is not None:
                per = self.gs if mode == "head" else 1
                kept = bits[b, :, :L].view(bits.shape[1] // per, per, L)
                a, dot = a.masked_fill(~kept, -math.inf), dot.masked_fill(~kept, 0.0)
            top = a.amax(-1, keepdim=True) if L else a.new_full((*a.shape[:2], 1), -math.inf)
            p = torch.exp(a - top.clamp(min=-1e300))
            z = p.sum(-1, keepdim=True)
            p = p / z.clamp(min=1e-300)
            want, weight = (p @ v).view(-1, self.D), (p @ v.abs()).view(-1, self.D)
            lse_want = (torch.log(z) + top).view(-1)
            # logits: fp32 sums of D products; weights: fp16, half a step 2^-11; outputs: bf16, half a step 2^-8
            dl = (self.D + 8) * 2.0 ** -24 / math.sqrt(self.D) * (dot.amax(-1) if L else dot.sum(-1)).view(-1)
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * dl + 1e-5)[:, None] * weight + 1e-36
            assert bool(((out[b].double() - want).abs() <= tol).all()), f"{mode} {share} b{b}"
            empty = lse_want == -math.inf
            assert bool((lse[b].double()[empty] == -math.inf).all())
            near = (lse[b].double() - lse_want).abs() <= dl + 2e-6 * (1 + lse_want.abs())
            assert bool(near[~empty].all()), f"lse {mode} {share} b{b}"


@pytest.mark.parametrize("page", [0, 16, 256])
@pytest.mark.parametrize("fmt,gs,D", [("e4m3", 4, 64), ("int8", 2, 64), ("e4m3", 8, 64), ("int8", 8, 128), ("int8", 1, 64)])
def test_long_chunks_against_the_formula(fmt, gs, D, page):
    c = Wide(fmt, gs, D, page, seed=gs + page)
    for share in SHARES:
        c.check("head", share)
    c.check("group", 0.1)
    c.check("shared", 0.3)
    c.check("dense", 1.0)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_long_chunks_of_blocks_of_very_different_scale(fmt):
    """V blocks 2^-20 to 2^20 apart: the weights' own reference moves apart from the softmax's."""
    def rows(g, which, shape):
        x = torch.randn(shape, device="cuda", generator=g)
        if which == "v":
            up = torch.randint(-20, 20, (*shape[:2], (shape[2] + 15) // 16), device="cuda", generator=g)
            x *= torch.exp2(up.float()).repeat_interleave(16, 2)[:, :, :shape[2], None]
        return (x * 3.0 if which == "k" else x).bfloat16()
    c = Wide(fmt, 4, 64, seed=3, rows=rows)
    for mode, share in (("head", 0.02), ("head", 0.5), ("group", 0.3), ("dense", 1.0)):
        c.check(mode, share)


@pytest.mark.parametrize("mode", ["head", "dense"])
def test_references_that_move_at_every_tile(mode):
    """Keys along one direction whose logits rise, fall and jump over a warp's dozens of tiles."""
    def rows(g, which, shape):
        x = torch.randn(shape, device="cuda", generator=g)
        if which == "k":
            t = torch.arange(shape[2], device="cuda") / shape[2]
            up = torch.stack([60 * (2 * t - 1), 60 * (1 - 2 * t), 60 * torch.cos(12 * t), 40 * t * torch.sign(torch.cos(99 * t))])
            x *= 0.1
            x[..., 0] += up.repeat(shape[1] // 4, 1)[None]
        return x.bfloat16()
    c = Wide("e4m3", 2, 64, seed=4, rows=rows)
    q = torch.zeros((c.B, c.Hq, c.D), device="cuda")
    q[..., 0] = torch.tensor([3.0, -3.0], device="cuda").repeat(c.Hkv)
    q += 0.05 * torch.randn(q.shape, device="cuda", generator=c.g)
    c.check(mode, 0.3, q.bfloat16())


@pytest.mark.parametrize("B,fmt,gs,D,page", [(80, "e4m3", 4, 64, 0), (8, "int8", 4, 128, 64), (20, "int8", 8, 64, 16), (8, "e4m3", 1, 128, 0)])
def test_votes_of_long_chunks(B, fmt, gs, D, page):
    """Chunks of 288 to 2048 tokens (the smallest is 256)."""
    c = Wide(fmt, gs, D, page, B=B, seed=B)
    q = torch.randn((B, c.Hq, D), device="cuda", generator=c.g).bfloat16()
    votes = torch.full((B, c.max_len), 3.0, device="cuda")
    c.ctx.softvote_scores(0, q, votes)
    torch.cuda.synchronize()
    for b, L in enumerate(c.lens):
        qq, k = q[b].double().view(c.Hkv, gs, D), c.k[b, :, :L].double()
        want = torch.softmax(qq @ k.transpose(1, 2) / math.sqrt(D), -1).sum((0, 1))
        dot = qq.abs() @ k.abs().transpose(1, 2)
        slack = (D + 8) * 2.0 ** -24 * (float(dot.max()) if L else 0.0) / math.sqrt(D)
        assert bool(((votes[b, :L].double() - want).abs() <= (2 * slack + 4e-6) * want + 1e-30).all()), f"b{b}"
        assert bool((votes[b, L:] == 3.0).all())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_calls_repeat_themselves_bit_for_bit(fmt):
    c = Wide(fmt, 4, 64, page=64, B=12, seed=9)
    q = torch.randn((c.B, c.Hq, c.D), device="cuda", generator=c.g).bfloat16()
    mask, _ = c.mask("head", 0.3)
    got = []
    for _ in range(5):
        outs = [torch.zeros_like(q) for _ in range(2)]
        lse, votes = torch.zeros((c.B, c.Hq), device="cuda"), torch.zeros((c.B, c.max_len), device="cuda")
        part = torch.zeros(c.B * c.Hq * (c.D + 1), device="cuda")
        c.ctx.sparse_attn(0, q, mask, TB.TB_MASK_PER_HEAD, outs[0], lse)
        c.ctx.sparse_attn(0, q, None, TB.TB_MASK_DENSE, outs[1])
        c.ctx.sparse_attn_partial(0, q, mask, TB.TB_MASK_PER_HEAD, part)
        c.ctx.softvote_scores(0, q, votes)
        got.append((*outs, lse, votes, part))
    torch.cuda.synchronize()
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
