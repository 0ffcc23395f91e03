"""Page ids outside the pool of an 8-bit layer: sequences with no other pages, and pages that a call does not need."""
import math

import numpy as np
import pytest
import torch

from query_aware_sparse_decode_b200 import tb as TB

from harness import KIMP_REL, kimp_rows, mask_from_sets, sets_from_mask
from test_gpu_kv8 import DT, MODES, Case, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("L", [40, 900])
def test_a_sequence_without_a_page_of_the_pool(fmt, L):
    """All its tokens are left out: no votes, no attention; the other sequence has its own."""
    c = Case(fmt, B=2, page=32, max_len=1024, seed=L)
    c.append((L, 333))
    q = dev(c.rng.normal(size=(c.B, c.Hq, c.D)), "bf16")
    whole = torch.full((c.B, c.max_len), 3.0, device="cuda")
    c.ctx.softvote_scores(0, q, whole)
    torch.cuda.synchronize()
    c.table[0] = -1
    votes = torch.full((c.B, c.max_len), 3.0, device="cuda")
    c.ctx.softvote_scores(0, q, votes)
    torch.cuda.synchronize()
    assert c.ctx.check_status() == 1
    assert bool((votes[0, :L] == 0).all()) and bool((votes[0, L:] == 3.0).all()) and torch.equal(votes[1], whole[1])
    out = torch.full((c.B, c.Hq, c.D), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.B, c.Hq), 9.0, device="cuda")
    c.ctx.sparse_attn(0, q, None, TB.TB_MASK_DENSE, out, lse)
    torch.cuda.synchronize()
    assert c.ctx.check_status() == 1
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    sets = c.all_tokens()
    sets.update({(0, h): np.arange(0) for h in range(c.Hq)})
    c.check_attention(q, sets, out, lse)


def test_a_votes_step_over_a_sequence_without_pages_selects_in_order():
    """Votes that are all zero tie: sink, window and the lowest 30 % of the indices; the attention over them is empty."""
    c = Case("int8", B=1, page=32, max_len=1024, variant=TB.TB_SOFTVOTE, keep=30)
    c.append((900,))
    c.table[0] = 1 << 20
    k, v = c.step_rows()
    q = dev(c.rng.normal(size=(1, c.Hq, c.D)), "bf16")
    out = torch.full_like(q, 9.0)
    c.ctx.decode_step(0, k, v, q, None, out)
    mask = c.ctx.step_masks(1)
    torch.cuda.synchronize()
    assert c.ctx.check_status() == 1 and bool((out == 0).all())
    # 901 tokens: a sink of 4, a window of 16, 30 % of 901 = 270 of those between
    assert np.array_equal(sets_from_mask(mask, [901])[0, 0], np.concatenate([np.arange(274), np.arange(885, 901)]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_that_hold_no_listed_token_are_not_missed(dtype):
    """One page after another leaves the pool; the mask lists tokens of the others only."""
    c = Case("e4m3", dtype, B=1, D=64, page=16, max_len=256)
    c.append((100,))
    torch.cuda.synchronize()
    for bad in range(4):
        good = c.table.clone()
        c.table[0, bad] = -1
        sets = {(0, h): np.setdiff1d(np.arange(3, 90, 5), np.arange(16 * bad, 16 * bad + 16)) for h in range(c.Hq)}
        mask = mask_from_sets(sets, 1, c.Hq, c.max_len)
        q = dev(c.rng.normal(size=(1, c.Hq, c.D)), dtype)
        out, lse = torch.zeros((1, c.Hq, c.D), dtype=DT[dtype], device="cuda"), torch.zeros((1, c.Hq), device="cuda")
        c.ctx.sparse_attn(0, q, mask, MODES["head"], out, lse)
        torch.cuda.synchronize()
        assert c.ctx.check_status() == 0
        c.check_attention(q, sets, out, lse, f"page {bad}")
        c.table.copy_(good)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_projection_does_not_miss_pages_past_the_length(dtype):
    """A ragged batch in a table whose unused entries are no pages; a page that holds tokens is missed."""
    c = Case("int8", dtype, B=2, page=16, max_len=512, D=64, dimp=16)
    c.append((300, 37))
    torch.cuda.synchronize()
    c.table[0, 19:] = -1      # 300 tokens lie on 19 pages, 37 on 3
    c.table[1, 3:] = 1 << 30
    c.kimp.fill_(7.0)
    c.ctx.project_kimp(0, 0, 300)
    torch.cuda.synchronize()
    assert c.ctx.check_status() == 0
    got = kimp_rows(c.kimp)
    for b, L in enumerate(c.lens):
        k = c.val["k"][b, :, :L]
        assert np.all(np.abs(got[b, :, :L] - k @ c.W) <= KIMP_REL * (np.abs(k) @ np.abs(c.W)) + 1e-30)
    assert np.all(got[1, :, 48:300] == 0) and np.all(got[:, :, 300:] == 7.0)
    c.table[1, 1] = -1
    c.ctx.project_kimp(0, 0, 300)
    torch.cuda.synchronize()
    assert c.ctx.check_status() == 1
    assert np.all(kimp_rows(c.kimp)[1, :, 16:32] == 0)
