"""8-bit K/V caches on the GPU against the float64 oracle (oracle/kv8.py):
codes and scales exactly, K_imp within fp32 rounding, attention and votes
over the cached values within derived bounds."""
import math

import numpy as np
import pytest
import torch

from oracle import kv8 as O8
from oracle import tokenbutler as O
from query_aware_sparse_decode_b200 import tb as TB
from query_aware_sparse_decode_b200.shard import ShardBuffers, run_lockstep, shard_step

from harness import KIMP_REL, kimp_rows, mask_from_sets, sets_from_mask

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rng_rows(rng, shape, wide=False):
    x = rng.normal(size=shape)
    if wide:  # blocks of very different size, rows too
        x = x * np.exp2(rng.integers(-30, 30, size=shape[:2] + (shape[2], 1)))
    return x


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(DT[dtype])


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


class Case:
    """A context with one 8-bit layer and the oracle's copy of its cache."""

    def __init__(self, fmt="e4m3", dtype="bf16", B=2, Hq=8, Hkv=2, D=128, dimp=32, max_len=512, page=0, seed=0,
                 variant=TB.TB_BUTLER, dense=False, keep=30, kimp_dtype="f32", G=1, layers=1, spare=3, fill=None):
        self.fmt, self.dtype, self.B, self.Hq, self.Hkv, self.D, self.dimp = fmt, dtype, B, Hq, Hkv, D, dimp
        self.gs, self.max_len, self.page = Hq // Hkv, max_len, page
        self.rng = np.random.default_rng(seed)
        self.cfg = TB.make_config(layers, B, Hq, Hkv, D, dimp, G, max_len, dtype, keep, 4, 16,
                                  dense_layers=(0,) if dense else (), variant=variant, kimp_dtype=kimp_dtype)
        self.ctx = TB.Context(self.cfg)
        self.W = host(dev(self.rng.normal(size=(D, dimp)) / math.sqrt(D), dtype))
        self.w = dev(self.W, dtype)
        self.kimp = TB.kimp_cache(self.cfg, fill=7.0)
        self.k, self.v, self.ks, self.vs = TB.kv8_cache(self.cfg, fmt)
        if page:
            n = max_len // page
            self.table = torch.from_numpy(self.rng.permutation(B * n + spare)[: B * n].reshape(B, n).astype(np.int32)).cuda()
            pool = lambda: torch.zeros((B * n + spare, Hkv, page, D), dtype=torch.int8, device="cuda").view(self.k.dtype)  # noqa: E731
            self.k, self.v = pool(), pool()
            self.ks = torch.zeros((B * n + spare, Hkv, page // 16), device="cuda")
            self.vs = torch.zeros_like(self.ks)
        if fill is not None:
            for t in (self.k, self.v):
                t.view(torch.int8).fill_(fill)
        self.bind()
        self.lens = [0] * B
        self.val = {x: np.zeros((B, Hkv, max_len, D)) for x in "kv"}
        self.exp = {x: np.full((B, Hkv, max_len // 16), O8.E_MIN) for x in "kv"}
        self.raw_k = np.zeros((B, Hkv, max_len, D))

    def bind(self, layer=0):
        if self.page:
            self.ctx.bind_layer_kv8_paged(layer, self.k, self.v, self.ks, self.vs, self.table, self.kimp, self.w)
        else:
            self.ctx.bind_layer_kv8(layer, self.k, self.v, self.ks, self.vs, self.kimp, self.w)

    def track(self, k, v, counts):
        for b, n in enumerate(counts):
            for g in range(self.Hkv):
                for x, src in (("k", k), ("v", v)):
                    self.val[x][b, g], self.exp[x][b, g] = O8.append(self.val[x][b, g], self.exp[x][b, g], self.lens[b],
                                                                     src[b, g, :n], self.fmt)
                self.raw_k[b, g, self.lens[b]:self.lens[b] + n] = k[b, g, :n]
            self.lens[b] += n

    def append(self, counts, wide=False, layout="bhnd", k=None, v=None, stream=None):
        n = max(max(counts), 1)
        shape = (self.B, self.Hkv, n, self.D)
        k = dev(rng_rows(self.rng, shape, wide) if k is None else k, self.dtype)
        v = dev(rng_rows(self.rng, shape, wide) if v is None else v, self.dtype)
        hk, hv = host(k), host(v)
        if layout == "fused":  # views of one [B][n][2 Hkv + 1][D] tensor
            qkv = torch.empty((self.B, n, 2 * self.Hkv + 1, self.D), dtype=DT[self.dtype], device="cuda")
            qkv[:, :, 1:self.Hkv + 1] = k.transpose(1, 2)
            qkv[:, :, self.Hkv + 1:] = v.transpose(1, 2)
            k, v = qkv[:, :, 1:self.Hkv + 1].transpose(1, 2), qkv[:, :, self.Hkv + 1:].transpose(1, 2)
        self.ctx.append_kv_rows(0, k, v, counts, stream)
        self.track(hk, hv, counts)

    def step_rows(self):
        k, v = (dev(rng_rows(self.rng, (self.B, self.Hkv, self.D)), self.dtype) for _ in range(2))
        return k, v

    def cached(self):
        """(codes as values, scales) of both tensors as dense [B][Hkv][max_len][.] float64."""
        out = []
        for c, s in ((self.k, self.ks), (self.v, self.vs)):
            c, s = host(c), host(s)
            if self.page:
                t = self.table.cpu().numpy()
                c = np.moveaxis(c[t], 2, 1).reshape(self.B, self.Hkv, self.max_len, self.D)
                s = np.moveaxis(s[t], 2, 1).reshape(self.B, self.Hkv, self.max_len // 16)
            out.append((c, s))
        return out

    def check_cache(self):
        torch.cuda.synchronize()
        assert self.ctx.seq_lens(0) == self.lens
        kimp = kimp_rows(self.kimp)
        for x, (c, s) in zip("kv", self.cached()):
            for b, L in enumerate(self.lens):
                nb = (L + 15) // 16
                assert np.array_equal(s[b, :, :nb], 2.0 ** self.exp[x][b, :, :nb]), f"{x} scales b{b}"
                got = c[b, :, :L] * np.repeat(s[b, :, :nb], 16, axis=1)[:, :L, None]
                assert np.array_equal(got, self.val[x][b, :, :L]), f"{x} values b{b}"
        for b, L in enumerate(self.lens):
            ref = self.raw_k[b, :, :L] @ self.W
            tol = KIMP_REL * (np.abs(self.raw_k[b, :, :L]) @ np.abs(self.W)) + 1e-30
            if self.cfg.kimp_bf16:
                lo, hi = O.round_to_bf16(ref - tol), O.round_to_bf16(ref + tol)
                assert np.all((kimp[b, :, :L] >= lo) & (kimp[b, :, :L] <= hi))
            else:
                assert np.all(np.abs(kimp[b, :, :L] - ref) <= tol), f"K_imp b{b}"
            assert np.all(kimp[b, :, L:] == 7.0)

    def check_attention(self, q, sets, out, lse, what=""):
        """out within the rounding of its type, of the weights (fp16: half a
        step 2^-11 of each, bf16 outputs 2^-8) and of the logits, which are
        fp32 sums of D products: D 2^-24 sum |q k| / sqrt(D), twice for the
        ratio, plus a few ulp of exp2 and of the running sums."""
        q, out = host(q), host(out)
        for b in range(self.B):
            for h in range(self.Hq):
                g = h // self.gs
                o, z, weight, dot = O8.attend(q[b, h], self.val["k"][b, g], self.val["v"][b, g], sets[b, h])
                dl = (self.D + 8) * 2.0 ** -24 * dot / math.sqrt(self.D)
                half = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -24
                w = 2.0 ** -11 if self.dtype == "bf16" else 0.0
                tol = half * np.abs(o) + (w + 2 * dl + 1e-5) * weight + 1e-36
                assert np.all(np.abs(out[b, h] - o) <= tol), f"{what} b{b} h{h}"
                if lse is None:
                    continue
                got = float(lse[b, h])
                assert got == z if z == -math.inf else abs(got - z) <= dl + 2e-6 * (1 + abs(z)), f"{what} lse b{b} h{h}"

    def all_tokens(self):
        return {(b, h): np.arange(self.lens[b]) for b in range(self.B) for h in range(self.Hq)}


def random_sets(c, rows, share, empty=()):
    sets = {}
    for b, L in enumerate(c.lens):
        for r in range(rows):
            s = np.nonzero(c.rng.random(L) < share)[0]
            sets[b, r] = s[:0] if (b, r) in empty else s
    return sets


# ------------------------------------------------------------------ writing and reading
WRITES = [
    ((0, 0), (1, 16)), ((0, 0), (15, 17)), ((0, 0), (31, 500)), ((5, 16), (3, 1)), ((15, 31), (1, 2)), ((7, 200), (0, 312)),
    ((100, 1), (60, 0)), ((512, 0), (0, 0)),
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,D,dimp", [("bf16", 128, 32), ("bf16", 64, 16), ("f32", 64, 32), ("f32", 128, 16)])
@pytest.mark.parametrize("first,second", WRITES)
def test_append_rows_equals_the_oracle(fmt, dtype, D, dimp, first, second):
    c = Case(fmt, dtype, D=D, dimp=dimp, seed=len(WRITES) + sum(first) + D)
    c.append(first, wide=True)
    c.append(second, wide=True, layout="fused")
    c.check_cache()
    assert c.ctx.check_status() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_block_that_grows_re_rounds_its_older_rows(fmt):
    c = Case(fmt, Hq=2, Hkv=1, B=1, max_len=256)
    for t in range(40):   # every token louder than the last: the scale grows inside the blocks
        k = c.rng.normal(size=(1, 1, 1, c.D)) * 1.7 ** t
        c.append([1], k=k, v=k[..., ::-1] * 3.0)
        if t in (0, 7, 15, 16, 39):
            c.check_cache()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_edge_values(fmt):
    """Zero blocks, values at and beside the largest code, ties, the fp32 range's ends."""
    c = Case(fmt, "f32", Hq=1, Hkv=1, B=1, D=64, dimp=16, max_len=512)
    F = O8.LARGEST[fmt]
    x = np.zeros((1, 1, 160, 64))
    x[..., 16:32, 0] = F
    x[..., 32:48, 0] = np.nextafter(np.float32(F), np.float32(1e9))
    x[..., 48:64, :] = (np.arange(64) - 31.5) * 0.5     # halves: ties
    x[..., 48, 0] = F
    x[..., 64:80, 3] = 3.4e38
    x[..., 80:96, 5] = 1e-38
    x[..., 96:112, :] = np.exp2(-np.arange(64) / 2.0)
    x[..., 112:128, 1] = 2.0 ** -91
    x[..., 128:160, :] = c.rng.normal(size=(32, 64)) * np.exp2(c.rng.integers(-40, 40, size=(32, 64)))
    c.append([160], k=x, v=-x)
    torch.cuda.synchronize()
    for name, (codes, s) in zip("kv", c.cached()):
        assert np.array_equal(s[0, 0, :10], 2.0 ** c.exp[name][0, 0, :10])
        assert np.array_equal(codes[0, 0, :160] * np.repeat(s[0, 0, :10], 16)[:, None], c.val[name][0, 0, :160])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_the_top_of_the_range_stays_finite(fmt):
    """bf16 rows with the type's largest values, beside ordinary blocks."""
    c = Case(fmt, Hq=1, Hkv=1, B=1, max_len=256)
    top = float(torch.finfo(torch.bfloat16).max)
    k = c.rng.normal(size=(1, 1, 40, c.D))
    k[0, 0, 3, ::7], k[0, 0, 17, 5], k[0, 0, 18, 6] = top, -top, 2.9e38
    c.append([40], k=k, v=-k)
    out = torch.zeros((1, 1, 40, c.D), dtype=torch.bfloat16, device="cuda")
    c.ctx.read_kv(0, 0, 40, out)
    torch.cuda.synchronize()
    assert c.ctx.check_status() == 0
    assert np.array_equal(host(out)[0, 0], c.val["k"][0, 0, :40]) and bool(torch.isfinite(out).all())
    codes, s = c.cached()[1]
    assert np.array_equal(codes[0, 0, :40] * np.repeat(s[0, 0, :3], 16)[:40, None], c.val["v"][0, 0, :40])


def test_not_a_number_and_infinity_are_stored_finite_and_flagged():
    c = Case("e4m3", Hq=1, Hkv=1, B=1, max_len=256)
    k = c.rng.normal(size=(1, 1, 20, c.D))
    k[0, 0, 3, 5], k[0, 0, 4, 6], k[0, 0, 4, 7] = np.nan, np.inf, -np.inf
    v = c.rng.normal(size=k.shape)
    c.append([20], k=k, v=v)
    torch.cuda.synchronize()
    assert c.ctx.check_status() == 8
    codes, s = c.cached()[0]
    assert np.array_equal(s[0, 0, :2], 2.0 ** c.exp["k"][0, 0, :2])
    got = codes[0, 0, :20] * np.repeat(s[0, 0, :2], 16)[:20, None]
    assert np.array_equal(got, c.val["k"][0, 0, :20]) and got[3, 5] == 0
    assert got[4, 6] == 448 * s[0, 0, 0] == -got[4, 7]
    c.append([1])
    torch.cuda.synchronize()
    assert c.ctx.check_status() == 0


def test_rows_behind_the_end_keep_their_bytes():
    c = Case("int8", fill=77, seed=4)
    c.append((21, 40))
    c.append((2, 3), wide=True)
    torch.cuda.synchronize()
    for t in (c.k, c.v):
        for b, L in enumerate(c.lens):
            assert bool((t[b, :, L:] == 77).all())


def test_set_lengths_back_into_a_block_keeps_its_scale():
    c = Case("int8", B=1, Hq=2, Hkv=1, max_len=256)
    k = c.rng.normal(size=(1, 1, 24, c.D))
    k[0, 0, 22] *= 100.0
    c.append([24], k=k, v=k)
    c.ctx.set_seq_lens(0, [20])      # the loud row is dropped, its block's scale stays
    c.lens = [20]
    c.append([3])
    torch.cuda.synchronize()
    codes, s = c.cached()[0]
    assert s[0, 0, 1] == 2.0 ** c.exp["k"][0, 0, 1]
    assert np.array_equal(codes[0, 0, 16:23] * s[0, 0, 1], c.val["k"][0, 0, 16:23])


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("int8", "f32")])
def test_paged_rows_and_reading_back(page, fmt, dtype):
    c = Case(fmt, dtype, page=page, seed=page)
    c.append((37, 130), wide=True)
    c.append((100, 0), layout="fused")
    c.check_cache()
    start, n = 30, 120
    k, v = (torch.full((c.B, c.Hkv, n, c.D), 5.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    c.ctx.read_kv(0, start, n, k, v)
    only = torch.full_like(k, 5.0)
    c.ctx.read_kv(0, start, n, None, only)
    torch.cuda.synchronize()
    assert torch.equal(only, v)
    for x, t in (("k", host(k)), ("v", host(v))):
        for b, L in enumerate(c.lens):
            m = max(0, min(L - start, n))
            assert np.array_equal(t[b, :, :m], c.val[x][b, :, start:start + m])   # exact: 8 significant bits at most
            assert np.all(t[b, :, m:] == 5.0)
    assert c.ctx.check_status() == 0


@pytest.mark.parametrize("kimp_dtype", ["f32", "bf16"])
def test_single_token_append_and_step_write_like_the_oracle(kimp_dtype):
    c = Case("e4m3", B=3, dense=True, kimp_dtype=kimp_dtype, max_len=256)
    c.append((0, 15, 40))
    for i in range(18):
        k, v = c.step_rows()
        if i % 2:
            c.ctx.append_kv(0, k, v)
        else:
            q = dev(c.rng.normal(size=(c.B, c.Hq, c.D)), c.dtype)
            out = torch.empty((c.B, c.Hq, c.D), dtype=torch.bfloat16, device="cuda")
            c.ctx.decode_step(0, k, v, q, None, out)
        c.track(host(k)[:, :, None], host(v)[:, :, None], [1, 1, 1])
        if i % 2 == 0:
            torch.cuda.synchronize()
            c.check_attention(q, c.all_tokens(), out, None, f"step {i}")
    c.check_cache()


# ------------------------------------------------------------------ attention
MODES = {"head": TB.TB_MASK_PER_HEAD, "group": TB.TB_MASK_GROUP, "shared": TB.TB_MASK_SHARED, "dense": TB.TB_MASK_DENSE}


def run_attention(c, mode, share=0.4, empty=()):
    q = dev(c.rng.normal(size=(c.B, c.Hq, c.D)), c.dtype)
    rows = {"head": c.Hq, "group": c.Hkv, "shared": 1, "dense": 0}[mode]
    if rows:
        own = random_sets(c, rows, share, empty)
        mask = mask_from_sets(own, c.B, rows, c.max_len)
        sets = {(b, h): own[b, {"head": h, "group": h // c.gs, "shared": 0}[mode]] for b in range(c.B) for h in range(c.Hq)}
        for b, L in enumerate(c.lens):   # bits past the length are ignored
            mask[b, :, (L + 31) // 32:] = -1
            if L % 32:
                mask[b, :, L // 32] |= torch.tensor(np.uint32(0xFFFFFFFF << (L % 32) & 0xFFFFFFFF).astype(np.int32)).cuda()
    else:
        mask, sets = None, c.all_tokens()
    out = torch.full((c.B, c.Hq, c.D), 9.0, dtype=DT[c.dtype], device="cuda")
    lse = torch.full((c.B, c.Hq), 9.0, device="cuda")
    c.ctx.sparse_attn(0, q, mask, MODES[mode], out, lse)
    torch.cuda.synchronize()
    assert c.ctx.check_status() == 0
    return q, mask, sets, out, lse


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (128, 8, 1), (64, 2, 2), (64, 4, 2), (128, 3, 3)])
def test_attention_against_the_oracle(mode, fmt, D, Hq, Hkv):
    c = Case(fmt, B=4, Hq=Hq, Hkv=Hkv, D=D, max_len=512, seed=D + Hq)
    c.append((0, 1, 300, 512))
    q, _, sets, out, lse = run_attention(c, mode, empty={(2, 0), (3, Hkv - 1)} if mode != "dense" else ())
    c.check_attention(q, sets, out, lse, mode)


@pytest.mark.parametrize("mode", ["head", "dense"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attention_fp32(mode, fmt):
    c = Case(fmt, "f32", B=3, Hq=4, Hkv=2, D=64, max_len=512)
    c.append((1, 511, 40))
    q, _, sets, out, lse = run_attention(c, mode, empty={(1, 0)} if mode == "head" else ())
    c.check_attention(q, sets, out, lse, mode)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("L", [15, 16, 17, 31, 33, 2049, 5000])
def test_attention_lengths(fmt, L):
    c = Case(fmt, B=1, Hq=4, Hkv=1, max_len=(L + 255) // 256 * 256, seed=L)
    c.append((L,))
    for mode in ("head", "dense"):
        q, _, sets, out, lse = run_attention(c, mode, share=0.2)
        c.check_attention(q, sets, out, lse, f"{mode} L{L}")


@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("int8", "bf16"), ("e4m3", "f32")])
def test_large_batches(fmt, dtype):
    """More (sequence, KV head) pairs than CTAs of a wave: one split each, sequences
    without a token among them."""
    c = Case(fmt, dtype, B=80, Hq=16, Hkv=8, D=64, dimp=16, max_len=256, seed=80)
    c.append([int(x) for x in c.rng.choice([0, 1, 15, 33, 100, 250], size=80)])
    for mode in ("head", "shared", "dense"):
        q, mask, sets, out, lse = run_attention(c, mode, empty={(2, 0)} if mode != "dense" else ())
        c.check_attention(q, sets, out, lse, mode)
        part = torch.zeros(c.B * c.Hq * (c.D + 1), device="cuda")
        c.ctx.sparse_attn_partial(0, q, mask, MODES[mode], part)
        torch.cuda.synchronize()
        n = c.B * c.Hq * c.D
        assert torch.equal(part[:n].view_as(out).to(out.dtype), out) and torch.equal(part[n:].view_as(lse), lse)


@pytest.mark.parametrize("spread", [20, 60])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attention_over_blocks_of_very_different_scale(fmt, spread):
    """V blocks 2^-spread to 2^spread apart while the softmax prefers tokens of
    small blocks: every head's output keeps its own relative precision."""
    c = Case(fmt, B=1, Hq=4, Hkv=1, max_len=768, seed=spread)
    n = 700
    k = c.rng.normal(size=(1, 1, n, c.D)) * 3.0
    v = c.rng.normal(size=(1, 1, n, c.D)) * np.exp2(np.repeat(c.rng.integers(-spread, spread, size=44), 16)[:n])[:, None]
    c.append([n], k=k, v=v)
    for trial in range(4):
        share = (0.5, 0.02, 0.005, 1.0)[trial]
        q, _, sets, out, lse = run_attention(c, "head", share=share)
        c.check_attention(q, sets, out, lse, f"share {share}")


def test_attention_with_rising_and_falling_logits():
    """The running maximum moves at every tile, up and down, and one token holds nearly all weight."""
    c = Case("e4m3", B=1, Hq=2, Hkv=1, max_len=2304, seed=8)
    n = 2200
    u = c.rng.normal(size=c.D)
    amp = np.concatenate([np.linspace(-60, 60, n // 2), np.linspace(60, -60, n - n // 2)])
    k = (u[None] * amp[:, None] / np.linalg.norm(u) + 0.1 * c.rng.normal(size=(n, c.D)))[None, None]
    c.append([n], k=k, v=c.rng.normal(size=k.shape))
    q = dev(np.stack([u, -u])[None] * 3.0, "bf16")
    out, lse = torch.empty((1, 2, c.D), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 2), device="cuda")
    c.ctx.sparse_attn(0, q, None, TB.TB_MASK_DENSE, out, lse)
    torch.cuda.synchronize()
    c.check_attention(q, c.all_tokens(), out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", ["head", "dense"])
def test_a_query_that_is_not_a_number_shows_in_its_head_only(dtype, mode):
    c = Case("e4m3", dtype, B=2, max_len=512)
    c.append((300, 40))
    q = c.rng.normal(size=(c.B, c.Hq, c.D))
    q[1, 2, 7] = np.nan
    mask = None
    if mode == "head":
        mask = mask_from_sets(random_sets(c, c.Hq, 0.5), c.B, c.Hq, c.max_len)
    out = torch.zeros((c.B, c.Hq, c.D), dtype=DT[dtype], device="cuda")
    lse = torch.zeros((c.B, c.Hq), device="cuda")
    c.ctx.sparse_attn(0, dev(q, dtype), mask, MODES[mode], out, lse)
    votes = torch.zeros((c.B, c.max_len), device="cuda")
    if dtype == "bf16":
        c.ctx.softvote_scores(0, dev(q, dtype), votes)
    torch.cuda.synchronize()
    bad = torch.zeros((c.B, c.Hq), dtype=torch.bool, device="cuda")
    bad[1, 2] = True
    assert torch.equal(torch.isnan(out).all(-1), bad) and torch.equal(torch.isnan(out).any(-1), bad)
    assert torch.equal(torch.isnan(lse), bad)
    if dtype == "bf16":
        assert bool(torch.isnan(votes[1, :40]).all()) and not bool(torch.isnan(votes[0]).any())


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("mode", ["head", "group", "dense"])
def test_paged_attention_equals_dense(mode, page):
    got = []
    for p in (0, page):
        c = Case("int8", B=2, page=p, max_len=1024, seed=3)
        c.rng = np.random.default_rng(11)   # the same rows in both layouts
        c.append((1000, 333))
        q, _, sets, out, lse = run_attention(c, mode)
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_index_lists_and_partials_equal_the_mask():
    c = Case("e4m3", B=2, max_len=1024)
    c.append((1000, 65))
    q, mask, sets, out, lse = run_attention(c, "head", share=0.3, empty={(0, 3)})
    cap = max(len(s) for s in sets.values())
    idx = torch.zeros((c.B, c.Hq, cap), dtype=torch.int32, device="cuda")
    count = torch.zeros((c.B, c.Hq), dtype=torch.int32, device="cuda")
    for (b, h), s in sets.items():
        idx[b, h, :len(s)] = torch.from_numpy(c.rng.permutation(s).astype(np.int32)).cuda()
        count[b, h] = len(s)
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    c.ctx.sparse_attn_idx(0, q, idx, count, out2, lse2)
    part = torch.empty(c.B * c.Hq * (c.D + 1), device="cuda")
    c.ctx.sparse_attn_partial(0, q, mask, TB.TB_MASK_PER_HEAD, part)
    out3, lse3 = torch.empty_like(out), torch.empty_like(lse)
    c.ctx.merge_partials(part, 1, out3, lse3)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert torch.equal(part[: c.B * c.Hq * c.D].view_as(out).bfloat16(), out)
    c.check_attention(q, sets, out3, lse3)


def test_a_page_outside_the_pool_is_left_out_and_flagged():
    c = Case("e4m3", B=2, page=64, max_len=512, dense=True)
    c.append((300, 200))
    torch.cuda.synchronize()
    good = c.table.clone()
    for bad in (10 ** 6, -1, c.k.shape[0]):
        c.table.copy_(good)
        c.table[0, 2] = bad
        q = dev(c.rng.normal(size=(c.B, c.Hq, c.D)), c.dtype)
        out, lse = torch.empty((c.B, c.Hq, c.D), dtype=torch.bfloat16, device="cuda"), torch.empty((c.B, c.Hq), device="cuda")
        c.ctx.sparse_attn(0, q, None, TB.TB_MASK_DENSE, out, lse)
        torch.cuda.synchronize()
        assert c.ctx.check_status() == 1
        sets = c.all_tokens()
        for h in range(c.Hq):
            sets[0, h] = np.concatenate([np.arange(128), np.arange(192, 300)])
        c.check_attention(q, sets, out, lse, "without the page")
        k = torch.full((c.B, c.Hkv, 300, c.D), 5.0, dtype=torch.bfloat16, device="cuda")
        c.ctx.read_kv(0, 0, 300, k, None)
        votes = torch.zeros((c.B, c.max_len), device="cuda")
        c.ctx.softvote_scores(0, q, votes)
        torch.cuda.synchronize()
        assert c.ctx.check_status() == 1
        got = host(k)
        assert np.all(got[0, :, 128:192] == 5.0) and np.array_equal(got[0, :, 192:], c.val["k"][0, :, 192:300])
        assert float(votes[0, 128:192].abs().max()) == 0 and abs(float(votes[0].sum()) - c.Hq) < 1e-3
    # a write to it lands nowhere
    before = [t.clone() for t in (c.k.view(torch.int8), c.v.view(torch.int8), c.ks, c.vs)]
    c.table[0, 300 // 64], c.table[1, 200 // 64] = -5, 1 << 30
    k, v = c.step_rows()
    c.ctx.append_kv(0, k, v)
    torch.cuda.synchronize()
    assert c.ctx.check_status() == 1
    for a, b in zip(before, (c.k.view(torch.int8), c.v.view(torch.int8), c.ks, c.vs)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ votes, projection, steps
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D,Hq,Hkv,page", [(128, 8, 2, 0), (64, 8, 1, 16), (128, 2, 2, 64), (128, 4, 2, 0)])
def test_votes_against_the_oracle(fmt, D, Hq, Hkv, page):
    c = Case(fmt, B=4, Hq=Hq, Hkv=Hkv, D=D, page=page, max_len=1024, seed=D)
    c.append((1, 0, 259, 1000))
    q = dev(c.rng.normal(size=(c.B, Hq, D)), "bf16")
    votes = torch.full((c.B, c.max_len), 3.0, device="cuda")
    c.ctx.softvote_scores(0, q, votes)
    torch.cuda.synchronize()
    got, hq = host(votes), host(q)
    for b, L in enumerate(c.lens):
        ref, slack = np.zeros(L), 0.0
        for h in range(Hq):
            k = c.val["k"][b, h // c.gs, :L]
            if L:
                a = k @ hq[b, h] / math.sqrt(D)
                p = np.exp(a - a.max())
                ref += p / p.sum()
                slack = max(slack, (D + 8) * 2.0 ** -24 * float((np.abs(k) @ np.abs(hq[b, h])).max()) / math.sqrt(D))
        # logits off by `slack` move a probability by at most twice that, relatively; a few ulp of exp2 and sums
        assert np.all(np.abs(got[b, :L] - ref) <= (2 * slack + 4e-6) * ref + 1e-30)
        assert np.all(got[b, L:] == 3.0)


@pytest.mark.parametrize("fmt,dtype,page", [("e4m3", "bf16", 0), ("int8", "f32", 16)])
def test_projection_from_the_codes(fmt, dtype, page):
    c = Case(fmt, dtype, page=page)
    c.append((100, 333))
    c.ctx.project_kimp_layers(0, 1, 3, 90)
    torch.cuda.synchronize()
    got = kimp_rows(c.kimp)
    for b in range(c.B):
        n = min(93, c.lens[b]) - 3
        k = c.val["k"][b, :, 3:3 + n]
        assert np.all(np.abs(got[b, :, 3:3 + n] - k @ c.W) <= KIMP_REL * (np.abs(k) @ np.abs(c.W)) + 1e-30)


@pytest.mark.parametrize("variant", [TB.TB_BUTLER, TB.TB_BUTLER_GROUP, TB.TB_SOFTVOTE], ids=["butler", "group", "softvote"])
@pytest.mark.parametrize("page", [0, 64])
def test_steps_of_every_variant(variant, page):
    """Prompt, then decode steps: the attention runs over the step's own
    selection of the 8-bit cache; the selection has the budget's size."""
    c = Case("int8", B=2, variant=variant, page=page, max_len=1024, keep=30, seed=variant)
    c.append((900, 301), layout="fused")
    rows = {TB.TB_BUTLER: c.Hq, TB.TB_BUTLER_GROUP: c.Hkv, TB.TB_SOFTVOTE: 1}[variant]
    for step in range(3):
        k, v = c.step_rows()
        q = dev(c.rng.normal(size=(c.B, c.Hq, c.D)), "bf16")
        qi = dev(c.rng.normal(size=(c.B * c.Hq, 1, 1, c.dimp)), "bf16")
        out = torch.empty((c.B, c.Hq, c.D), dtype=torch.bfloat16, device="cuda")
        c.ctx.decode_step(0, k, v, q, qi, out)
        c.track(host(k)[:, :, None], host(v)[:, :, None], [1, 1])
        masks = c.ctx.step_masks(rows)
        torch.cuda.synchronize()
        assert c.ctx.check_status() == 0
        own = sets_from_mask(masks, c.lens)
        for b, L in enumerate(c.lens):
            for r in range(rows):
                assert len(own[b, r]) == min(L, 20 + min(30 * L // 100, L - 20))
        per = {c.Hq: lambda h: h, c.Hkv: lambda h: h // c.gs, 1: lambda h: 0}[rows]
        c.check_attention(q, {(b, h): own[b, per(h)] for b in range(c.B) for h in range(c.Hq)}, out, None, f"step {step}")
    c.check_cache()


def test_selection_does_not_depend_on_the_format():
    """K_imp comes from the unrounded keys: both formats select the same tokens."""
    masks = []
    for fmt in ("e4m3", "int8"):
        c = Case(fmt, B=2, max_len=1024, seed=21)
        c.append((900, 301))
        k, v = c.step_rows()
        qi = dev(c.rng.normal(size=(c.B * c.Hq, 1, 1, c.dimp)), "bf16")
        q = dev(c.rng.normal(size=(c.B, c.Hq, c.D)), "bf16")
        c.ctx.decode_step(0, k, v, q, qi, torch.empty_like(q))
        m = c.ctx.step_masks(c.Hq)
        torch.cuda.synchronize()
        masks.append(sets_from_mask(m, c.ctx.seq_lens(0)))
    assert all(np.array_equal(masks[0][k], masks[1][k]) for k in masks[0])


def test_sharded_step_over_8_bit_caches():
    """Two ranks' contexts in lock step: the merged output is the attention
    over the union of their masks."""
    world, L, cut = 2, 700, 304
    cs = [Case("e4m3", B=1, max_len=512, seed=31) for _ in range(world)]
    k = cs[0].rng.normal(size=(1, 2, L, 128))
    v = cs[0].rng.normal(size=k.shape)
    for r, (lo, hi) in enumerate(((0, cut), (cut, L - 1))):
        cs[r].append([hi - lo], k=k[:, :, lo:hi], v=v[:, :, lo:hi])
        cs[r].w.copy_(cs[0].w)
    q = dev(cs[0].rng.normal(size=(1, 8, 128)), "bf16")
    qi = dev(cs[0].rng.normal(size=(8, 1, 1, 32)), "bf16")
    kn, vn = dev(k[:, :, -1], "bf16"), dev(v[:, :, -1], "bf16")
    bufs = [ShardBuffers(c.cfg, world) for c in cs]
    outs = [torch.empty_like(q) for _ in cs]
    run_lockstep([shard_step(c.ctx, 0, r, world, (0, cut)[r], [L], q, qi, outs[r], bufs[r], *((kn, vn) if r else (None, None)))
                  for r, c in enumerate(cs)])
    torch.cuda.synchronize()
    cs[1].track(host(kn)[:, :, None], host(vn)[:, :, None], [1])
    whole = Case("e4m3", B=1, max_len=1024, seed=31)
    whole.lens = [L]
    for x in "kv":
        whole.val[x][:, :, :cut] = cs[0].val[x][:, :, :cut]
        whole.val[x][:, :, cut:L] = cs[1].val[x][:, :, :L - cut]
    parts = [sets_from_mask(bufs[r].mask, cs[r].lens) for r in range(world)]
    sets = {(0, h): np.concatenate([parts[0][0, h], parts[1][0, h] + cut]) for h in range(8)}
    assert all(len(s) == 20 + 210 for s in sets.values())
    for o in outs:
        whole.check_attention(q, sets, o, None)


def test_reused_selections_and_prefill_rows_on_8_bit_layers():
    """Amortised selection and the row selection of a prefill read K_imp only: an
    8-bit layer and a bf16 one with the same K_imp choose the same tokens."""
    c = Case("int8", B=2, max_len=512, layers=2, seed=12)
    c.append((400, 130))
    kb, vb = (torch.randn((2, 2, 512, 128), device="cuda").bfloat16() for _ in range(2))
    torch.cuda.synchronize()
    kimp = c.kimp.clone()
    c.ctx.bind_layer(1, kb, vb, kimp, c.w)
    c.ctx.set_seq_lens(1, c.lens)
    rows = dev(c.rng.normal(size=(c.B * c.Hq, 1, 20, c.dimp)), "bf16")
    masks = [torch.zeros((c.B, c.Hq, 20, 16), dtype=torch.int32, device="cuda") for _ in range(2)]
    for layer in (0, 1):
        c.ctx.select_prefill(layer, rows, 100, 20, masks[layer])
    torch.cuda.synchronize()
    assert torch.equal(masks[0], masks[1]) and int(masks[0].ne(0).sum()) > 0
    caches = [c.ctx.selection_cache(layer) for layer in (0, 1)]
    c.ctx.set_reuse(0.5, 3, 1)
    qi = dev(c.rng.normal(size=(c.B * c.Hq, 1, 1, c.dimp)), "bf16")
    q = dev(c.rng.normal(size=(c.B, c.Hq, c.D)), "bf16")
    for step in range(3):
        k, v = c.step_rows()
        got = []
        for layer in (0, 1):
            out = torch.empty_like(q)
            c.ctx.decode_step(layer, k, v, q, qi, out)
            got.append(sets_from_mask(c.ctx.step_masks(c.Hq), c.ctx.seq_lens(layer)))
        c.track(host(k)[:, :, None], host(v)[:, :, None], [1, 1])
        torch.cuda.synchronize()
        # the appended rows' K_imp differ by fp32 rounding (another order of the same sum)
        assert all(len(np.setxor1d(got[0][x], got[1][x])) <= 2 for x in got[0])
    assert c.ctx.check_status() == 0 and len(caches) == 2


def test_offsets_past_32_bits():
    """A cache whose codes pass 2^32 bytes: rows written, read and attended near its end."""
    n = 4194304 + 512
    c = Case("e4m3", B=1, Hq=8, Hkv=8, max_len=n, dense=True, seed=2)
    L0 = n - 300
    c.val = {x: np.zeros((1, 8, 512, 128)) for x in "kv"}   # the oracle's window: the last rows
    c.ctx.set_seq_lens(0, [L0])
    k, v = (dev(c.rng.normal(size=(1, 8, 200, 128)), "bf16") for _ in range(2))
    c.ctx.append_kv_rows(0, k, v)
    kn, vn = c.step_rows()
    q = dev(c.rng.normal(size=(1, 8, 128)), "bf16")
    c.ctx.append_kv(0, kn, vn)
    assert c.ctx.seq_lens(0) == [L0 + 201]
    base = L0 // 16 * 16
    assert base == L0 - 4   # the rows start inside a block whose older rows are zero
    for g in range(8):
        for x, a, b in (("k", k, kn), ("v", v, vn)):
            w, e = O8.append(np.zeros((512, 128)), np.full(32, O8.E_MIN), 4, host(a)[0, g], "e4m3")
            c.val[x][0, g], _ = O8.append(w, e, 204, host(b)[0, g][None], "e4m3")
    ko = torch.zeros((1, 8, 201, 128), dtype=torch.bfloat16, device="cuda")
    c.ctx.read_kv(0, L0, 201, ko)
    mask = torch.zeros((1, 8, n // 32), dtype=torch.int32, device="cuda")
    bits = np.zeros((8, 512), bool)
    for h in range(8):
        bits[h, 4:205] = c.rng.random(201) < 0.3
        for t in np.nonzero(bits[h])[0] + base:
            mask[0, h, t // 32] |= int(np.uint32(1 << (int(t) % 32)).astype(np.int32))
    out, lse = torch.empty_like(q), torch.empty((1, 8), device="cuda")
    c.ctx.sparse_attn(0, q, mask, TB.TB_MASK_PER_HEAD, out, lse)
    torch.cuda.synchronize()
    assert c.ctx.check_status() == 0
    assert np.array_equal(host(ko)[0], c.val["k"][0, :, 4:205])
    c.check_attention(q, {(0, h): np.nonzero(bits[h])[0] for h in range(8)}, out, lse)


# ------------------------------------------------------------------ use
def test_layers_of_both_kinds_in_one_context_and_rebinding():
    c = Case("e4m3", B=2, layers=2, dense=True, max_len=512)
    kb, vb = (torch.randn((2, 2, 512, 128), device="cuda").bfloat16() for _ in range(2))
    kimp = TB.kimp_cache(c.cfg)
    c.ctx.bind_layer(1, kb, vb, kimp, c.w)
    c.ctx.set_seq_lens(1, [200, 100])
    c.append((200, 100))
    q = dev(c.rng.normal(size=(2, 8, 128)), "bf16")
    out = torch.empty_like(q)
    c.ctx.sparse_attn(1, q, None, TB.TB_MASK_DENSE, out)
    alone = TB.Context(c.cfg)
    alone.bind_layer(1, kb, vb, kimp, c.w)
    alone.set_seq_lens(1, [200, 100])
    ref = torch.empty_like(q)
    alone.sparse_attn(1, q, None, TB.TB_MASK_DENSE, ref)
    # the 8-bit layer rebound as bf16, and back
    c.ctx.bind_layer(0, kb, vb, kimp, c.w)
    c.ctx.set_seq_lens(0, [200, 100])
    out0 = torch.empty_like(q)
    c.ctx.sparse_attn(0, q, None, TB.TB_MASK_DENSE, out0)
    c.bind()
    c.ctx.set_seq_lens(0, [200, 100])
    out8 = torch.empty_like(q)
    c.ctx.sparse_attn(0, q, None, TB.TB_MASK_DENSE, out8)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(out0, ref)
    c.check_attention(q, c.all_tokens(), out8, None)


def test_side_stream_and_captured_step():
    """A step's calls on a stream of their own, captured once (the graph holds
    the lengths of its capture) and replayed with other rows and queries."""
    c = Case("e4m3", B=2, dense=True, max_len=512)
    c.append((100, 37))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kn, vn = c.step_rows()
    q = dev(c.rng.normal(size=(2, 8, 128)), "bf16")
    rows_k, rows_v = (dev(rng_rows(c.rng, (2, 2, 20, 128)), "bf16") for _ in range(2))
    out, ko, vo = torch.empty_like(q), *(torch.zeros((2, 2, 512, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def calls():
        c.ctx.set_seq_lens(0, [100, 37])
        c.ctx.append_kv_rows(0, rows_k, rows_v, [20, 5], s)
        c.ctx.decode_step(0, kn, vn, q, None, out, s)
        c.ctx.read_kv(0, 0, 512, ko, vo, s)
    with torch.cuda.stream(s):
        calls()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        calls()
    for _ in range(2):
        for t in (rows_k, rows_v, kn, vn, q):
            t.copy_(dev(c.rng.normal(size=tuple(t.shape)), "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        d = Case("e4m3", B=2, dense=True, max_len=512, seed=0)
        d.append((100, 37))              # the same seed: the same first rows
        d.track(host(rows_k), host(rows_v), [20, 5])
        d.track(host(kn)[:, :, None], host(vn)[:, :, None], [1, 1])
        # the block the rows started in may keep a larger scale from an earlier run: compare from the next one on
        for x, got in (("k", host(ko)), ("v", host(vo))):
            assert np.array_equal(got[0, :, 112:121], d.val[x][0, :, 112:121])
    assert c.ctx.check_status() == 0


def test_refusals():
    c = Case("e4m3", B=2, max_len=512, layers=2)
    L = TB.lib()
    h = c.ctx._h
    import ctypes
    ptr = [ctypes.c_void_p(t.data_ptr()) for t in (c.k, c.v, c.ks, c.vs, c.kimp, c.w)]
    assert L.tb_bind_layer_kv8(h, 0, 0, *ptr) == 1 and L.tb_bind_layer_kv8(h, 0, 3, *ptr) == 1
    assert L.tb_bind_layer_kv8(h, 2, 1, *ptr) == 1 and L.tb_bind_layer_kv8(h, -1, 1, *ptr) == 1
    for i in range(6):
        bad = list(ptr)
        bad[i] = None
        assert L.tb_bind_layer_kv8(h, 0, 1, *bad) == 1
        bad[i] = ctypes.c_void_p(ptr[i].value + 4)
        assert L.tb_bind_layer_kv8(h, 0, 1, *bad) == 2
    table = ctypes.c_void_p(c.kimp.data_ptr())
    for pages, size, most, want in ((8, 8, 64, 2), (8, 24, 64, 2), (8, 64, 7, 2), (0, 64, 8, 2), (1 << 25, 64, 8, 2)):
        assert L.tb_bind_layer_kv8_paged(h, 0, 1, *ptr[:4], pages, table, size, most, *ptr[4:]) == want
    assert L.tb_bind_layer_kv8_paged(h, 0, 1, *ptr[:4], 8, None, 64, 8, *ptr[4:]) == 1
    k = torch.zeros((2, 2, 300, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TB.TBError) as e:
        c.ctx.append_kv_rows(1, k, k)              # not bound
    assert e.value.status == 8
    c.append((300, 0))
    with pytest.raises(TB.TBError) as e:
        c.ctx.append_kv_rows(0, k, k, [300, 10])   # one sequence would not fit
    assert e.value.status == 3 and c.ctx.seq_lens(0) == [300, 0]
    for counts in ([301, 0], [-1, 0], [1], [1, 2, 3]):
        with pytest.raises(ValueError):
            c.ctx.append_kv_rows(0, k, k, counts)
    with pytest.raises(ValueError):
        c.ctx.append_kv_rows(0, k.transpose(2, 3).contiguous().transpose(2, 3), k)   # rows not contiguous
    with pytest.raises(TypeError):
        c.ctx.append_kv_rows(0, k.float(), k.float())
    with pytest.raises(ValueError):
        c.ctx.append_kv_rows(0, k[:1], k[:1])
    odd = torch.zeros(2 * 2 * 300 * 132 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TB.TBError) as e:           # row stride not a multiple of 16 bytes
        c.ctx.append_kv_rows(0, odd[: 2 * 2 * 300 * 132].view(2, 2, 300, 132)[..., :128], k, [10, 10])
    assert e.value.status == 2
    with pytest.raises(TB.TBError) as e:           # rows not 16-byte aligned
        c.ctx.append_kv_rows(0, odd[4:4 + 2 * 2 * 300 * 128].view(2, 2, 300, 128), k, [10, 10])
    assert e.value.status == 2
    with pytest.raises(TB.TBError) as e:
        c.ctx.append_kv(0, odd[4:4 + 512].view(2, 2, 128), k[:, :, 0].contiguous())
    assert e.value.status == 2 and c.ctx.seq_lens(0) == [300, 0]
    assert L.tb_bind_layer_kv8_paged(h, 1, 1, *ptr[:4], 8, ctypes.c_void_p(c.kimp.data_ptr() + 2), 64, 8, *ptr[4:]) == 2
    out = torch.zeros((2, 2, 10, 128), dtype=torch.bfloat16, device="cuda")
    for start, n, want in ((-1, 10, 1), (508, 10, 3)):
        with pytest.raises(TB.TBError) as e:
            c.ctx.read_kv(0, start, n, out)
        assert e.value.status == want
    with pytest.raises(TB.TBError):
        c.ctx.read_kv(0, 0, 10)
    with pytest.raises(ValueError):
        c.ctx.read_kv(0, 0, 11, out)
    with pytest.raises(TypeError):
        c.ctx.read_kv(0, 0, 10, out.float())
    with pytest.raises(TypeError):
        c.ctx.bind_layer_kv8(1, c.k.view(torch.uint8), c.v, c.ks, c.vs, c.kimp, c.w)
    with pytest.raises(TypeError):
        c.ctx.bind_layer_kv8(1, c.k, c.v.view(torch.int8), c.ks, c.vs, c.kimp, c.w)
    with pytest.raises(ValueError):
        c.ctx.bind_layer_kv8(1, c.k, c.v, c.ks[..., :8], c.vs, c.kimp, c.w)
    with pytest.raises(ValueError):
        c.ctx.bind_layer_kv8(1, c.k, c.v, c.ks, c.vs, c.kimp[:1], c.w)
    kb = torch.zeros((2, 2, 512, 128), dtype=torch.bfloat16, device="cuda")
    c.ctx.bind_layer(1, kb, kb.clone(), c.kimp, c.w)
    for call in (lambda: c.ctx.append_kv_rows(1, k, k, [1, 1]), lambda: c.ctx.read_kv(1, 0, 10, out)):
        with pytest.raises(TB.TBError) as e:       # not an 8-bit layer
            call()
        assert e.value.status == 7
    c.ctx.append_kv_rows(0, k[:, :, :0], k[:, :, :0])
    c.ctx.append_kv_rows(0, k, k, [0, 0])
    torch.cuda.synchronize()
    assert c.ctx.seq_lens(0) == [300, 0] and c.ctx.check_status() == 0
