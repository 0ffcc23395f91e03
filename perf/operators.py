"""Workloads of the 8-bit K/V cache operators, with their plain forms.

A cache layer holds K and V as one byte an element, with one fp32 scale (a
power of two) for every block of 16 tokens of a (sequence, KV head): codes
[B][Hkv][max_len][D], scales [B][Hkv][max_len/16], or the same in pages.

  write   rows of every sequence are quantised behind its cached rows, their
          importance keys K W_K are formed from the unrounded rows, and the
          touched range is read back as values;
  attend  single-token attention over the 8-bit cache: every token, or the
          tokens of a bit mask for each query head, KV group or sequence;
  step    one decode step of a dense layer: append, then attention;
  votes   soft votes: softmax of q . K for each head, summed over the heads.

`own` chooses between the plain form and the framework's calls.
"""
import math

import torch

own = False

BLOCK = 16       # tokens that share a scale
TILE = 256       # tokens of a K_imp tile
E_MIN = -100     # the smallest scale is 2**E_MIN
LARGEST = {"e4m3": 448.0, "int8": 127.0}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a prompt of 32768 tokens written in one call
        {"name": "write prompt", "op": "write", "fmt": "e4m3", "type": "bf16", "heads": 32, "kv": 8, "dim": 128, "imp": 32,
         "had": "0", "new": "32768"},
        # chunks of a continued prefill: ragged, one sequence idle, starts inside a block
        {"name": "write ragged", "op": "write", "fmt": "int8", "type": "bf16", "heads": 32, "kv": 8, "dim": 128, "imp": 32,
         "had": "5,777,0,4095,2000", "new": "512,1,0,513,1000"},
        # fp32 rows of a small model
        {"name": "write small", "op": "write", "fmt": "e4m3", "type": "f32", "heads": 4, "kv": 2, "dim": 64, "imp": 16,
         "had": "0,33", "new": "100,20"},
        # the long-context decode: 30 % of 131072 tokens for each head, plus sink and window
        {"name": "attend long", "op": "attend", "fmt": "e4m3", "type": "bf16", "heads": 32, "kv": 8, "dim": 128, "imp": 32,
         "lens": "131072,131072,131072,131072", "mask": "head", "keep": 30, "page": 0},
        # one sequence, every token
        {"name": "attend one", "op": "attend", "fmt": "e4m3", "type": "bf16", "heads": 32, "kv": 8, "dim": 128, "imp": 32,
         "lens": "4096", "mask": "dense", "keep": 100, "page": 0},
        # a serving batch in pages of 64 tokens, one set for each KV group
        {"name": "attend paged", "op": "attend", "fmt": "int8", "type": "bf16", "heads": 32, "kv": 8, "dim": 128, "imp": 32,
         "lens": "32768,1000,17,9999,20001,32000,1,512", "mask": "group", "keep": 50, "page": 64},
        # small heads, groups of eight, a shared set, and a sequence without a token
        {"name": "attend odd", "op": "attend", "fmt": "int8", "type": "bf16", "heads": 16, "kv": 2, "dim": 64, "imp": 16,
         "lens": "777,0,5001", "mask": "shared", "keep": 10, "page": 0},
        # fp32 queries
        {"name": "attend f32", "op": "attend", "fmt": "e4m3", "type": "f32", "heads": 4, "kv": 2, "dim": 64, "imp": 16,
         "lens": "512,100", "mask": "head", "keep": 50, "page": 0},
        # a dense layer's step for a batch of chats
        {"name": "step batch", "op": "step", "fmt": "e4m3", "type": "bf16", "heads": 32, "kv": 8, "dim": 128, "imp": 32,
         "batch": 16, "len": 8191},
        # the smallest step: latency
        {"name": "step one", "op": "step", "fmt": "int8", "type": "bf16", "heads": 32, "kv": 8, "dim": 128, "imp": 32,
         "batch": 1, "len": 1000},
        # soft votes of the long-context sweep
        {"name": "votes long", "op": "votes", "fmt": "e4m3", "type": "bf16", "heads": 32, "kv": 8, "dim": 128, "imp": 32,
         "lens": "131072"},
        # soft votes of a ragged batch
        {"name": "votes ragged", "op": "votes", "fmt": "int8", "type": "bf16", "heads": 32, "kv": 8, "dim": 128, "imp": 32,
         "lens": "16383,1,1000,4097"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "attend", "attend", "step", "votes"))
    kv = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 4, 8))
    c = {"op": op, "fmt": rng.choice(("e4m3", "int8")), "type": "bf16", "heads": kv * group, "kv": kv,
         "dim": rng.choice((64, 128, 128)), "imp": rng.choice((16, 32))}
    batch = rng.randint(1, 8)
    room = (4 * 8 * 131072) // (batch * kv)     # tokens a sequence, inside the largest listed case
    if op == "write":
        c["type"] = rng.choice(("bf16", "bf16", "f32"))
        room = min(16384, (8 * 32768) // (batch * kv))
        c["had"] = ",".join(str(rng.choice((0, _log_uniform(rng, 1, 4096)))) for _ in range(batch))
        c["new"] = ",".join(str(_log_uniform(rng, 1, room)) for _ in range(batch))
    elif op == "step":
        c.update(batch=batch, len=_log_uniform(rng, 1, min(65536, room // 2)))
    else:
        c["lens"] = ",".join(str(_log_uniform(rng, 1, min(131072, room // 2))) for _ in range(batch))
        if op == "attend":
            c["mask"] = rng.choice(("dense", "head", "group", "shared"))
            c["keep"] = 100 if c["mask"] == "dense" else rng.randint(1, 90)
            c["page"] = rng.choice((0, 0, 16, 64, 256))
            c["type"] = "f32" if rng.random() < 0.1 else "bf16"
            if c["type"] == "f32":
                c["lens"] = ",".join(str(min(int(x), 8192)) for x in c["lens"].split(","))
    return c


def _ints(text):
    return [int(x) for x in text.split(",")]


def _up(n, m):
    return -(-n // m) * m


def work(case):
    c = case
    size = 2 if c["type"] == "bf16" else 4
    kv, d, heads, imp = c["kv"], c["dim"], c["heads"], c["imp"]
    group = heads // kv
    if c["op"] == "write":
        rows = sum(_ints(c["new"])) * kv
        kept = sum(h % BLOCK for h in _ints(c["had"])) * kv
        # read k and v, write codes, scales and K_imp; then read the range's codes back into values
        first = min(_ints(c["had"])) // TILE * TILE
        back = sum(max(0, h + n - first) for h, n in zip(_ints(c["had"]), _ints(c["new"]))) * kv
        nbytes = rows * (2 * d * (size + 1) + 4 * imp + 8 / BLOCK) + kept * 2 * d + d * imp * size
        return {"bytes": nbytes + back * (2 * d * (size + 1) + 8 / BLOCK), "flops": 2 * rows * d * imp}
    if c["op"] == "step":
        b, n = c["batch"], c["len"] + 1
        nbytes = b * kv * (n * (2 * d + 8 / BLOCK) + d * 2 * (size + 1) + 4 * imp) + 2 * b * heads * d * size + d * imp * size
        return {"bytes": nbytes, "flops": 4 * b * heads * n * d}
    lens = _ints(c["lens"])
    if c["op"] == "votes":
        return {"bytes": sum(lens) * (kv * (d + 4 / BLOCK) + 4) + len(lens) * heads * d * size,
                "flops": sum(lens) * heads * 2 * d}
    share = c["keep"] / 100
    rows = 1 - (1 - share) ** group if c["mask"] == "head" else share
    words = {"dense": 0, "head": heads, "group": kv, "shared": 1}[c["mask"]]
    blocks = 1 - (1 - rows) ** BLOCK
    nbytes = sum(lens) * (kv * (rows * 2 * d + blocks * 8 / BLOCK) + words / 8) + len(lens) * heads * (2 * d * size + 4)
    return {"bytes": nbytes, "flops": 4 * d * heads * share * sum(lens)}


# ------------------------------------------------------------------ the inputs
def _pow2(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scale_exp(amax, fmt):
    """The smallest e with amax <= LARGEST * 2**e, not under E_MIN."""
    lm, le = math.frexp(LARGEST[fmt])
    m, e = torch.frexp(amax)
    e = e.to(torch.int32) - le + (m > lm).to(torch.int32)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(min=E_MIN)


def _random_cache(g, batch, kv, max_len, d, fmt, loud):
    """Codes and scales of normal rows; `loud` channels of the heads stand out, as those of keys do."""
    codes = torch.empty((batch, kv, max_len, d), dtype=CODES[fmt], device="cuda")
    scale = torch.empty((batch, kv, max_len // BLOCK), dtype=torch.float32, device="cuda")
    gain = torch.ones(d, device="cuda")
    gain[torch.arange(loud, device="cuda") * (d // max(loud, 1))] = 4.0
    for b in range(batch):
        x = torch.randn((kv, max_len // BLOCK, BLOCK, d), device="cuda", generator=g) * gain
        e = _scale_exp(x.abs().amax((2, 3)), fmt)
        y = x * _pow2(-e)[..., None, None]
        codes[b] = (y.round() if fmt == "int8" else y).reshape(kv, max_len, d).to(CODES[fmt])
        scale[b] = _pow2(e)
    return codes, scale


def _pages(g, codes, scale, page):
    """The same rows in pages, in an order of their own, with spare pages: pools, scale pools and the table."""
    batch, kv, max_len, d = codes.shape
    n = max_len // page
    table = torch.randperm(batch * n + 3, device="cuda", generator=g)[: batch * n].reshape(batch, n)
    pool = torch.zeros((batch * n + 3, kv, page, d), dtype=torch.uint8, device="cuda")
    pool[table.reshape(-1)] = codes.view(torch.uint8).reshape(batch, kv, n, page, d).transpose(1, 2).reshape(-1, kv, page, d)
    pscale = torch.ones((batch * n + 3, kv, page // BLOCK), device="cuda")
    pscale[table.reshape(-1)] = scale.reshape(batch, kv, n, page // BLOCK).transpose(1, 2).reshape(-1, kv, page // BLOCK)
    return pool.view(codes.dtype), pscale, table


def _random_mask(g, rows_of, words, lens, share):
    """Bit masks [B][rows][words]: a sink of 4 tokens and `share` of the others; one row of each batch is left empty."""
    bits = torch.rand((len(lens), rows_of, words, 32), device="cuda", generator=g) < share
    bits[:, :, 0, :4] = True
    if rows_of > 1:
        bits[len(lens) - 1, rows_of - 1] = False
    weight = torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
    return (bits * weight).sum(-1).to(torch.int32)


def _context(case, s, batch, max_len):
    from query_aware_sparse_decode_b200 import tb as TB
    cfg = TB.make_config(n_layers=1, batch=batch, n_q_heads=case["heads"], n_kv_heads=case["kv"], head_dim=case["dim"],
                         d_imp=case["imp"], producer_freq=1, max_len=max_len, kv_dtype=case["type"], keep_pct=100, sink=4,
                         window=16)
    ctx = TB.Context(cfg)
    s["ctx"], s["mode"] = ctx, {"head": TB.TB_MASK_PER_HEAD, "group": TB.TB_MASK_GROUP, "shared": TB.TB_MASK_SHARED,
                                "dense": TB.TB_MASK_DENSE}[case.get("mask", "dense")]
    if case.get("page"):
        ctx.bind_layer_kv8_paged(0, s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"].to(torch.int32), s["kimp"], s["w"])
    else:
        ctx.bind_layer_kv8(0, s["k"], s["v"], s["k_scale"], s["v_scale"], s["kimp"], s["w"])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, kv, d, heads, imp = TYPES[c["type"]], c["kv"], c["dim"], c["heads"], c["imp"]
    lens = _ints(c["had"]) if c["op"] == "write" else [c["len"]] * c["batch"] if c["op"] == "step" else _ints(c["lens"])
    new = _ints(c["new"]) if c["op"] == "write" else [1 if c["op"] == "step" else 0] * len(lens)
    batch, max_len = len(lens), _up(max(max(h + n for h, n in zip(lens, new)), 1), TILE)
    s = {"op": c["op"], "fmt": c["fmt"], "lens": lens, "new": new, "len_t": torch.tensor(lens, device="cuda"),
         "new_t": torch.tensor(new, device="cuda"), "page": c.get("page", 0), "mask_of": c.get("mask", "dense")}
    s["k"], s["k_scale"] = _random_cache(g, batch, kv, max_len, d, c["fmt"], 4)
    s["v"], s["v_scale"] = _random_cache(g, batch, kv, max_len, d, c["fmt"], 0)
    if s["page"]:
        order = torch.Generator(device="cuda")
        order.manual_seed(seed + 1)
        k, ks, s["table"] = _pages(order, s["k"], s["k_scale"], s["page"])
        order.manual_seed(seed + 1)
        v, vs, _ = _pages(order, s["v"], s["v_scale"], s["page"])
        s.update(k=k, k_scale=ks, v=v, v_scale=vs)
    s["kimp"] = torch.zeros((batch, kv, max_len // TILE, imp, TILE), device="cuda")
    s["w"] = (torch.randn((d, imp), device="cuda", generator=g) / math.sqrt(d)).to(dt)
    s["q"] = torch.randn((batch, heads, d), device="cuda", generator=g).to(dt)
    s["out"] = torch.zeros((batch, heads, d), dtype=dt, device="cuda")
    s["lse"] = torch.zeros((batch, heads), device="cuda")
    if c["op"] == "write":
        s["first"] = min(lens) // TILE * TILE
        n = _up(max(h + m for h, m in zip(lens, new)), TILE) - s["first"]
        # rows as a fused projection leaves them: [B][tokens][K heads, V heads][D]
        qkv = torch.randn((batch, max(new), 2 * kv, d), device="cuda", generator=g) * 1.5
        qkv[:, :, :kv, :: d // 4] *= 4.0
        qkv = qkv.to(dt)
        s["k_new"], s["v_new"] = qkv[:, :, :kv].transpose(1, 2), qkv[:, :, kv:].transpose(1, 2)
    else:
        s["first"], n = c.get("len", 0) // BLOCK * BLOCK, BLOCK
        s["k_new"] = torch.randn((batch, kv, 1, d), device="cuda", generator=g).to(dt)
        s["v_new"] = torch.randn((batch, kv, 1, d), device="cuda", generator=g).to(dt)
    s["k_out"] = torch.zeros((batch, kv, n, d), dtype=dt, device="cuda")
    s["v_out"] = torch.zeros_like(s["k_out"])
    if c["op"] == "votes":
        s["votes"] = torch.zeros((batch, max_len), device="cuda")
    s["mask"] = None
    if c["op"] == "attend" and c["mask"] != "dense":
        rows = {"head": heads, "group": kv, "shared": 1}[c["mask"]]
        s["mask"] = _random_mask(g, rows, max_len // 32, lens, c["keep"] / 100)
    if own:
        _context(c, s, batch, max_len)
        s["k_row"], s["v_row"] = s["k_new"][:, :, 0].contiguous(), s["v_new"][:, :, 0].contiguous()
    return s


# ------------------------------------------------------------------ the plain forms
def _dense(s, which):
    codes, scale = s[which], s[which + "_scale"]
    if not s["page"]:
        return codes, scale
    t = s["table"]
    batch, n = t.shape
    kv, page, d = codes.shape[1:]
    codes = codes.view(torch.uint8)[t].transpose(1, 2).reshape(batch, kv, n * page, d).view(s[which].dtype)
    return codes, scale[t].transpose(1, 2).reshape(batch, kv, n * page // BLOCK)


def _values(codes, scale):
    batch, kv, n, d = codes.shape
    x = codes.to(torch.float32).reshape(batch, kv, n // BLOCK, BLOCK, d) * scale[..., None, None]
    return x.reshape(batch, kv, n, d)


def _round(y, fmt):
    if fmt == "int8":
        return y.round().clamp(-127.0, 127.0)
    _, e = torch.frexp(y)
    e = (e - 4).clamp(min=-9)      # three bits behind the leading one; steps of 2**-9 at the smallest
    return ((y * _pow2(-e)).round() * _pow2(e)).clamp(-448.0, 448.0)


def _keys_values(s, which, first, n):
    """Rows [first, first + n) with the new ones written: what the cache holds, as values, and the unrounded new rows."""
    codes, scale = _dense(s, which)
    fmt = s["fmt"]
    batch, kv, _, d = codes.shape
    old = codes[:, :, first:first + n].to(torch.float32)
    e_old = torch.frexp(scale[:, :, first // BLOCK:(first + n) // BLOCK])[1].to(torch.int32) - 1
    t = torch.arange(first, first + n, device="cuda")[None]
    at = t - s["len_t"][:, None]
    fresh, kept = (at >= 0) & (at < s["new_t"][:, None]), at < 0
    src = s[which + "_new"].to(torch.float32)
    x = src.gather(2, at.clamp(0, src.shape[2] - 1)[:, None, :, None].expand(batch, kv, n, d))
    x = torch.where(fresh[:, None, :, None], x, torch.zeros_like(x))
    per = lambda a: a.reshape(batch, a.shape[1], n // BLOCK, BLOCK, -1)  # noqa: E731
    need = _scale_exp(per(x).abs().amax((3, 4)), fmt)
    any_kept = kept.reshape(batch, 1, n // BLOCK, BLOCK).any(-1)
    any_new = fresh.reshape(batch, 1, n // BLOCK, BLOCK).any(-1)
    e = torch.where(any_kept, torch.where(any_new, torch.maximum(need, e_old), e_old), need)
    back = lambda a: a[..., None].expand(batch, kv, n // BLOCK, BLOCK).reshape(batch, kv, n, 1)  # noqa: E731
    new_v = _round(x * _pow2(back(-e)), fmt) * _pow2(back(e))
    old_v = _round(old * _pow2(back(e_old - e).clamp(min=-126)), fmt) * _pow2(back(e))
    zero = torch.zeros_like(x)
    val = torch.where(fresh[:, None, :, None], new_v, torch.where(kept[:, None, :, None], old_v, zero))
    return val, x, fresh


def _attention(q, k, v, keep):
    batch, kv, n, d = k.shape
    q = q.to(torch.float32).reshape(batch, kv, -1, d)
    a = (q @ k.transpose(2, 3)) / math.sqrt(d)
    a = torch.where(keep, a, torch.full_like(a, -math.inf))
    top = a.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(a - top)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return out.reshape(batch, -1, d), (torch.log(total) + top).reshape(batch, -1)


def _keep(s, n, kv, group):
    t = torch.arange(n, device="cuda")
    inside = (t[None] < s["len_t"][:, None])[:, None, None]
    if s["mask"] is None:
        return inside
    m = s["mask"]
    bits = ((m[..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1).bool().reshape(m.shape[0], m.shape[1], n)
    bits = bits[:, :, None] if s["mask_of"] != "head" else bits.reshape(m.shape[0], kv, group, n)
    return inside & bits


def _plain(s):
    dt = s["q"].dtype
    if s["op"] == "write":
        n = s["k_out"].shape[2]
        k, x, fresh = _keys_values(s, "k", s["first"], n)
        v, _, _ = _keys_values(s, "v", s["first"], n)
        imp = (x @ s["w"].to(torch.float32)) * fresh[:, None, :, None]
        batch, kv = k.shape[:2]
        imp = imp.reshape(batch, kv, n // TILE, TILE, -1).transpose(3, 4)
        return {"k": k.to(dt), "v": v.to(dt), "kimp": imp.contiguous()}
    if s["op"] == "step":
        n, size = s["lens"][0] + 1, s["k"].shape[2]
        k, x, _ = _keys_values(s, "k", 0, size)
        v, _, _ = _keys_values(s, "v", 0, size)
        out, _ = _attention(s["q"], k[:, :, :n], v[:, :, :n], torch.ones((), dtype=torch.bool, device="cuda"))
        imp = x[:, :, n - 1] @ s["w"].to(torch.float32)
        f = s["first"]
        return {"out": out.to(dt), "k": k[:, :, f:f + BLOCK].to(dt), "v": v[:, :, f:f + BLOCK].to(dt), "kimp": imp}
    k = _values(*_dense(s, "k"))
    batch, kv, n, d = k.shape
    group = s["q"].shape[1] // kv
    keep = _keep(s, n, kv, group)
    if s["op"] == "attend":
        out, lse = _attention(s["q"], k, _values(*_dense(s, "v")), keep)
        return {"out": out.to(dt), "lse": lse}
    a = (s["q"].to(torch.float32).reshape(batch, kv, group, d) @ k.transpose(2, 3)) / math.sqrt(d)
    a = torch.where(keep, a, torch.full_like(a, -math.inf))
    p = torch.exp(a - a.amax(-1, keepdim=True))
    return {"votes": (p / p.sum(-1, keepdim=True)).sum((1, 2))}


# ------------------------------------------------------------------ the framework's calls
def _framework(s):
    ctx = s["ctx"]
    ctx.set_seq_lens(0, s["lens"])
    n = s["k_out"].shape[2]
    if s["op"] == "write":
        ctx.append_kv_rows(0, s["k_new"], s["v_new"], s["new"])
        ctx.read_kv(0, s["first"], n, s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"], "kimp": s["kimp"][:, :, s["first"] // TILE:]}
    if s["op"] == "step":
        ctx.decode_step(0, s["k_row"], s["v_row"], s["q"], None, s["out"])
        ctx.read_kv(0, s["first"], n, s["k_out"], s["v_out"])
        at = s["lens"][0]
        return {"out": s["out"], "k": s["k_out"], "v": s["v_out"], "kimp": s["kimp"][:, :, at // TILE, :, at % TILE]}
    if s["op"] == "attend":
        ctx.sparse_attn(0, s["q"], s["mask"], s["mode"], s["out"], s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    ctx.softvote_scores(0, s["q"], s["votes"])
    return {"votes": s["votes"]}


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------ 64 bits
def _exact_block(old, e_old, x, fmt):
    """One block's values: `old` codes (or None) at 2**e_old, and new rows x, on the definition."""
    big = LARGEST[fmt]
    top = float(x.abs().max()) if x.numel() else 0.0
    e = E_MIN
    if top > 0:
        e = math.ceil(math.log2(top / big))
        while big * 2.0 ** (e - 1) >= top:
            e -= 1
        while big * 2.0 ** e < top:
            e += 1
        e = max(e, E_MIN)
    if old is not None:
        e = max(e, e_old)
        x = torch.cat([old * 2.0 ** e_old, x])
    y = x / 2.0 ** e
    y = torch.round(y) if fmt == "int8" else y.to(torch.float32).to(torch.float8_e4m3fn).to(torch.float64)
    return y * 2.0 ** e


def _exact_rows(s, which, b, h, lo, hi):
    """The values of rows [lo, hi) of one head, lo a block's start, those of the call's new rows among them."""
    codes, scale = _dense(s, which)
    codes, scale = codes[b, h].to(torch.float64).cpu(), scale[b, h].to(torch.float64).cpu()
    new = s[which + "_new"][b, h].to(torch.float64).cpu()
    had, count = s["lens"][b], s["new"][b]
    got = torch.zeros((hi - lo, codes.shape[1]), dtype=torch.float64)
    for t in range(lo, min(hi, _up(had + count, BLOCK)), BLOCK):
        last = min(t + BLOCK, had + count)
        e_old = int(round(math.log2(float(scale[t // BLOCK]))))
        if t >= had + count:
            break
        if last <= had:
            rows = codes[t:last] * 2.0 ** e_old
        else:
            mine = new[max(0, t - had):last - had]
            rows = _exact_block(codes[t:had] if t < had else None, e_old, mine, s["fmt"])
        got[t - lo:last - lo] = rows
    return got


def _exact_head(q, k, v):
    """Attention of one head's query over the rows given (double): output and log of the sum."""
    if not len(k):
        return torch.zeros_like(q), -math.inf
    a = (k * q).sum(1) / math.sqrt(len(q))
    z = torch.logsumexp(a, 0)
    return (torch.exp(a - z)[:, None] * v).sum(0), float(z)


def exact(case, seed):
    c = case
    if c["op"] == "write" and sum(_ints(c["had"]) + _ints(c["new"])) * c["kv"] > 60000:
        return None
    if c["op"] != "write":
        tokens = c["batch"] * c["len"] if c["op"] == "step" else sum(_ints(c["lens"]))
        if tokens * c["heads"] * c["dim"] > 1 << 31:
            return None
    s = prepare(case, seed)
    f64 = torch.float64
    batch, kv, d = len(s["lens"]), c["kv"], c["dim"]
    group = c["heads"] // kv
    w = s["w"].to(f64).cpu()
    if c["op"] == "write":
        first, n = s["first"], s["k_out"].shape[2]
        k, v = (torch.stack([torch.stack([_exact_rows(s, x, b, h, first, first + n) for h in range(kv)]) for b in range(batch)])
                for x in ("k", "v"))
        imp = torch.zeros((batch, kv, n, c["imp"]), dtype=f64)
        for b in range(batch):
            at = s["lens"][b] - first
            imp[b, :, at:at + s["new"][b]] = s["k_new"][b, :, :s["new"][b]].to(f64).cpu() @ w
        return {"k": k, "v": v, "kimp": imp.reshape(batch, kv, n // TILE, TILE, -1).permute(0, 1, 2, 4, 3).contiguous()}
    q = s["q"].to(f64)
    if c["op"] == "step":
        n, f = c["len"] + 1, s["first"]
        out = torch.empty((batch, c["heads"], d), dtype=f64)
        last = {}
        for x in ("k", "v"):
            last[x] = torch.stack([torch.stack([_exact_rows(s, x, b, h, f, f + BLOCK) for h in range(kv)]) for b in range(batch)])
        for b in range(batch):
            for h in range(kv):
                rows = {}
                for x in ("k", "v"):
                    sc = s[x + "_scale"][b, h].to(f64).repeat_interleave(BLOCK)[:f, None]
                    rows[x] = torch.cat([s[x][b, h, :f].to(f64) * sc, last[x][b, h, :n - f].cuda()])
                for i in range(h * group, (h + 1) * group):
                    out[b, i] = _exact_head(q[b, i], rows["k"], rows["v"])[0].cpu()
        return {"out": out, "k": last["k"], "v": last["v"], "kimp": s["k_new"][:, :, 0].to(f64).cpu() @ w}
    out = torch.zeros((batch, c["heads"], d), dtype=f64)
    lse = torch.full((batch, c["heads"]), -math.inf, dtype=f64)
    (kc, ks), (vc, vs) = _dense(s, "k"), _dense(s, "v")
    votes = torch.zeros((batch, kc.shape[2]), dtype=f64, device="cuda")
    for b in range(batch):
        n = s["lens"][b]
        for h in range(kv):
            k = kc[b, h, :n].to(f64) * ks[b, h].to(f64).repeat_interleave(BLOCK)[:n, None]
            v = vc[b, h, :n].to(f64) * vs[b, h].to(f64).repeat_interleave(BLOCK)[:n, None]
            for i in range(h * group, (h + 1) * group):
                if c["op"] == "votes":
                    if n:
                        votes[b, :n] += torch.softmax((k * q[b, i]).sum(1) / math.sqrt(d), 0)
                    continue
                kept = torch.ones(n, dtype=torch.bool, device="cuda")
                if s["mask"] is not None:
                    row = s["mask"][b, {"head": i, "group": h, "shared": 0}[c["mask"]]]
                    at = torch.arange(n, device="cuda")
                    kept = ((row[at // 32] >> (at % 32).to(torch.int32)) & 1) == 1
                o, z = _exact_head(q[b, i], k[kept], v[kept])
                out[b, i], lse[b, i] = o.cpu(), z
    return {"votes": votes} if c["op"] == "votes" else {"out": out, "lse": lse}
