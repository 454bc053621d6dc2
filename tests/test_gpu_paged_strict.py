"""Attention over shared prefixes, the tokens' attention weight and their eviction on the GPU: the order of their launches,
their rounding, workspaces, graphs and refusals, held more tightly than tests/test_gpu_paged_more.py does."""
import numpy as np
import pytest

from oracle import serving
from tests.test_gpu_paged_more import shared_cache
from tests.test_gpu_serving import Dev, dev, starts

pytestmark = pytest.mark.gpu


def _t():
    import torch

    return torch


# --------------------------------------------------------------------------------------------- order
@pytest.mark.parametrize("legacy", [False, True])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("S,n,H,Hkv,hs", [(4, 1, 2, 2, 64), (70, 1, 2, 1, 128), (3, 80, 2, 2, 64)])
def test_shared_sees_what_was_launched_before_and_keeps_it_from_what_follows(S, n, H, Hkv, hs, q8, legacy):
    """Steps queued without a pause, each over rows, lengths, prefixes, a table and tokens that the launches right before it
    write and the next step's overwrite: the bits of the same steps one at a time. On the legacy stream and another, and
    captured (the graph holds all steps)."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(4000 + S)
    c, ns, gs, prefix = shared_cache(rng, [(2300, [(n + 40, n)] * S), (700, [(n + 3, n)] * 3)], Hkv, hs, 64, q8)
    rows, w, B, steps = sum(ns), H * hs, len(ns), 6
    d, qs, dgs, dpl = Dev(c, poison=False), dev(starts(ns)), dev(gs), dev(prefix)
    most = int(max(starts(ns)[gs[1:]] - starts(ns)[gs[:-1]]))
    q = [dev(serving.bf16(rng.standard_normal((rows, w)) * 2), t.bfloat16) for _ in range(steps)]
    kv = [dev(serving.bf16(rng.standard_normal((rows, 2 * Hkv * hs))), t.bfloat16) for _ in range(steps)]
    cut = [0, 30, 0, 25, 7, 1]  # own tokens fewer by so many
    lens = [dev((c.kv_len - x).astype(np.int32)) for x in cut]
    plens = [dev((prefix - 64 * (i % 3)).astype(np.int32)) for i in range(steps)]
    # every other step the first prefix's pages the other way round (in all rows that share them)
    turned = c.table.copy()
    turned[:S, :35] = turned[:S, 34::-1]
    tables = [dev(c.table), dev(turned)]
    s_q, s_kv, s_len, s_plen, s_table = (x.clone() for x in (q[0], kv[0], lens[0], plens[0], tables[0]))
    h = gk.PagedKv(d.k, d.v, d.ks, d.vs, s_table, s_len)
    blank = [x.clone() for x in (d.k, d.v, d.ks, d.vs) if x is not None]
    y = t.zeros(steps, rows, w, dtype=t.bfloat16, device="cuda")
    lse = t.zeros(steps, rows, H, device="cuda")

    def run(ctx, pause):
        for a, b in zip([x for x in (d.k, d.v, d.ks, d.vs) if x is not None], blank):
            a.copy_(b)
        for i in range(steps):
            for a, b in ((s_q, q[i]), (s_kv, kv[i]), (s_plen, plens[i]), (s_table, tables[i % 2]), (s_len, lens[i])):
                a.copy_(b)
                pause()
            gk.gk_paged_write(ctx, h, gk.GK_BF16, s_kv, 2 * Hkv * hs, s_kv[:, Hkv * hs :], 2 * Hkv * hs, qs, B, rows)
            pause()
            gk.gk_paged_attn_shared(ctx, h, gk.GK_BF16, s_q, w, y[i], w, lse[i], qs, B, dgs, s_plen, 2, H, rows, n, most, 0.125)
            pause()

    def taken():
        got = y.clone(), lse.clone()
        y.zero_()
        lse.zero_()
        return got

    stream = t.cuda.default_stream() if legacy else t.cuda.Stream()
    ctx = gk.Ctx(stream.cuda_stream, workspace_bytes=64 << 20)
    t.cuda.synchronize()
    with t.cuda.stream(stream):
        run(ctx, t.cuda.synchronize)
        want = taken()
        assert all(not t.equal(want[0][i], want[0][i + 1]) for i in range(steps - 1)) and want[0].isfinite().all()
        for _ in range(3):
            t.cuda._sleep(2_000_000)  # the host is ahead: all launches are queued
            run(ctx, lambda: None)
            assert all(t.equal(a, b) for a, b in zip(taken(), want))
    gk.gk_sync(ctx)
    if not legacy:
        t.cuda.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=stream):
            run(ctx, lambda: None)
        for _ in range(2):
            g.replay()
            t.cuda.synchronize()
            assert all(t.equal(a, b) for a, b in zip(taken(), want))
        gk.gk_sync(ctx)
    ctx.close()
