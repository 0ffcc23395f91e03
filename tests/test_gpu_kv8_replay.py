"""A captured sequence of 8-bit calls (prompt, chunk, step, lists, votes, read-back), replayed with other inputs: every
output and the whole cache against the oracle."""
import math

import numpy as np
import pytest
import torch

from oracle import kv8 as O8
from query_aware_sparse_decode_b200 import tb as TB

from harness import mask_from_sets
from test_gpu_kv8 import Case, dev, host, random_sets, rng_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dtype,page", [("e4m3", "bf16", 0), ("int8", "bf16", 64), ("e4m3", "f32", 16)])
def test_replays_equal_the_oracle(fmt, dtype, page):
    c = Case(fmt, dtype, B=2, D=64, page=page, dense=True, max_len=512, seed=page)
    prompt, chunk, end = [100, 37], [20, 5], [121, 43]  # a step follows the chunk
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pk, pv, ck, cv = (dev(rng_rows(c.rng, (2, c.Hkv, n, 64)), dtype) for n in (100, 100, 20, 20))
    kn, vn = c.step_rows()
    q = dev(c.rng.normal(size=(2, c.Hq, 64)), dtype)
    c.lens = list(end)
    mask = mask_from_sets(random_sets(c, c.Hq, 0.3), 2, c.Hq, c.max_len)
    dense, sparse = torch.empty_like(q), torch.empty_like(q)
    lse, votes = torch.empty((2, c.Hq), device="cuda"), torch.zeros((2, c.max_len), device="cuda")
    ko, vo = (torch.zeros((2, c.Hkv, 512, 64), dtype=q.dtype, device="cuda") for _ in range(2))

    def calls():
        c.ctx.set_seq_lens(0, [0, 0])      # blocks are written from their start: no older scale stays
        c.ctx.append_kv_rows(0, pk, pv, prompt, s)
        c.ctx.append_kv_rows(0, ck, cv, chunk, s)
        c.ctx.decode_step(0, kn, vn, q, None, dense, s)
        c.ctx.sparse_attn(0, q, mask, TB.TB_MASK_PER_HEAD, sparse, lse, s)
        if dtype == "bf16":
            c.ctx.softvote_scores(0, q, votes, s)
        c.ctx.read_kv(0, 0, 512, ko, vo, s)
    with torch.cuda.stream(s):
        calls()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        calls()
    for size in (1.0, 64.0, 0.01):
        for t in (pk, pv, ck, cv, kn, vn):
            t.copy_(dev(c.rng.normal(size=tuple(t.shape)) * size, dtype))
        q.copy_(dev(c.rng.normal(size=tuple(q.shape)) / size, dtype))
        sets = random_sets(c, c.Hq, 0.4, empty={(1, 3)})
        mask.copy_(mask_from_sets(sets, 2, c.Hq, c.max_len))
        for t in (dense, sparse, lse, votes, ko, vo):
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        c.lens = [0, 0]
        for x in "kv":
            c.val[x][:], c.exp[x][:] = 0.0, O8.E_MIN
        c.track(host(pk), host(pv), prompt)
        c.track(host(ck), host(cv), chunk)
        c.track(host(kn)[:, :, None], host(vn)[:, :, None], [1, 1])
        assert c.lens == end and c.ctx.check_status() == 0
        c.check_cache()
        c.check_attention(q, c.all_tokens(), dense, None, "step")
        c.check_attention(q, sets, sparse, lse, "lists")
        for b, L in enumerate(end):
            for x, t in (("k", ko), ("v", vo)):
                assert np.array_equal(host(t)[b, :, :L], c.val[x][b, :, :L]) and np.all(host(t)[b, :, L:] == 9.0)
            if dtype != "bf16":
                continue
            ref, slack = np.zeros(L), 0.0
            for h in range(c.Hq):
                k = c.val["k"][b, h // c.gs, :L]
                a = k @ host(q)[b, h] / math.sqrt(64)
                p = np.exp(a - a.max())
                ref += p / p.sum()
                slack = max(slack, 72 * 2.0 ** -24 * float((np.abs(k) @ np.abs(host(q)[b, h])).max()) / math.sqrt(64))
            assert np.all(np.abs(host(votes)[b, :L] - ref) <= (2 * slack + 4e-6) * ref + 1e-30)
