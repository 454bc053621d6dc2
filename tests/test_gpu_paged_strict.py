"""Attention over shared prefixes, the tokens' attention weight and their eviction on the GPU: the order of their launches,
their rounding, workspaces, graphs and refusals, held more tightly than tests/test_gpu_paged_more.py does."""
import numpy as np
import pytest

from oracle import serving
from tests.test_gpu_paged_more import attend_shared, check_evict, evict, shared_cache, shared_ref, to_pages, weigh
from tests.test_gpu_serving import Dev, check_attention, dev, refused, starts
from tests.test_oracle_serving import cache

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
        with t.cuda.stream(stream):  # and not captured again, by the context that was
            run(ctx, lambda: None)
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip(taken(), want))
        gk.gk_sync(ctx)
    ctx.close()


# ----------------------------------------------------------------------------------------- rounding
def few_heavy_keys(rng, S, n, H, Hkv, hs, page, q8, prefix=2100, tail=6):
    """Sequences behind one prefix in which three keys of it and one own one share all of the weight, their values near 1 and
    -1: sums cancel, and what a weight was rounded to shows. (cache, rows, new tokens, group_start, prefix_len)"""
    c, ns, gs, pl = shared_cache(rng, [(prefix, [(tail + n, n)] * S)], Hkv, hs, page, False)
    k = rng.standard_normal(c.k.shape).astype(np.float32) * np.float32(0.3)
    k[..., 0] = -24
    v = rng.standard_normal(c.v.shape).astype(np.float32)
    at = [c.place(0, j) for j in (17, 1200, prefix - 130)] + [c.place(b, prefix + 3) for b in range(S)]
    pg, rw = (np.array(x) for x in zip(*at))
    k[pg, :, rw] = rng.standard_normal((len(at), Hkv, hs))
    k[pg, :, rw, 0] = 4
    v[pg, :, rw] = rng.choice([-1, 1], (len(at), Hkv, hs)) * rng.uniform(0.9, 1.1, (len(at), Hkv, hs))
    if q8:
        (kc, ks), (vc, vs) = serving.quantise(k), serving.quantise(v)
        c = serving.Pages(kc, vc, ks, vs, c.table, c.kv_len)
    else:
        c = serving.Pages(serving.bf16(k), serving.bf16(v), None, None, c.table, c.kv_len)
    # (a page in which the prefix ends is each sequence's own: the same tokens)
    if prefix % page:
        for x in (c.k, c.v, c.k_scale, c.v_scale):
            if x is not None:
                x[c.table[:, prefix // page], :, : prefix % page] = x[c.table[0, prefix // page], :, : prefix % page]
    q = rng.standard_normal((sum(ns), H, hs)) * 0.5
    q[..., 0] = 16
    return c, serving.bf16(q), ns, gs, pl


# Beside y's own rounding (half a step of bf16: 2^-8 |y|) a weight of 16 bits may be off by 2^-17 relative, and by what its
# float32 score is: a sum of hs products, each addition cut by a step of 2^-23 of a running sum of at most scale sum |q||k| <
# 9.5 here, 128 2^-23 9.5 = 2^-12.7; the same again in the sum of weights that divides. Together below 2^-11.5 of the spread
# sum w |v|. (Weights rounded to bf16 are off by up to 2^-8 each.)
FINE = 2.0 ** -11.5


@pytest.mark.parametrize("S,n,H,Hkv,hs,page,q8,ws", [
    (64, 1, 8, 2, 128, 64, True, 64),  # 256 rows, codes laid out as bf16 first
    (64, 1, 8, 2, 128, 64, True, 2),  # no room for that: unpacked on the way
    (40, 1, 4, 2, 64, 16, True, 64),
    (130, 1, 4, 1, 64, 32, True, 64),  # more than 512 rows
    (40, 1, 2, 2, 64, 64, False, 64),
    (36, 3, 4, 2, 128, 128, False, 64),
    (9, 8, 4, 1, 96, 256, False, 64),
    (10, 16, 4, 1, 80, 16, True, 64),
    (5, 1, 4, 1, 64, 64, True, 64),  # few rows in all
])
def test_shared_weights_of_few_rows_have_16_bits(S, n, H, Hkv, hs, page, q8, ws):
    """As many rows as a sequence may have (64 a key / value head over 8-bit pages, 32 over bf16), in groups of many more."""
    from gpt_decoder_gb300 import gk

    assert n * H // Hkv <= (64 if q8 else 32)
    rng = np.random.default_rng(4100 + S + hs)
    c, q, ns, gs, pl = few_heavy_keys(rng, S, n, H, Hkv, hs, page, q8)
    scale = hs ** -0.5
    y_ref, lse_ref, spread = shared_ref(c, q, ns, gs, pl, scale)
    ctx = gk.Ctx(_t().cuda.current_stream().cuda_stream, workspace_bytes=ws << 20)
    y, lse = attend_shared(ctx, c, q, ns, gs, pl, scale)
    ctx.close()
    off = np.abs(y - y_ref) - 2.0 ** -8 * np.abs(y_ref)
    assert off.max() <= FINE * spread.max() and (off <= FINE * spread).all(), (off / spread).max()
    assert np.abs(lse - lse_ref).max() < 2.0 ** -11.5


# ----------------------------------------------------------------------------------------- workspace
@pytest.mark.parametrize("width,mib", [(16384, 64), (16000, 64), (15008, 64), (14000, 64), (65536, 256), (16384, 96), (2048, 3)])
def test_shared_8_bit_prefixes_leave_room_for_the_parts(width, mib):
    """One group of 64 samples, 32 heads over 8 of 128, behind 8-bit pages, in workspaces that the prefix's codes as bf16 would
    take whole (64 MiB: 16384 positions), nearly, or that hold two parts of every row and no codes: the shared way is taken, as an
    impossible group shows, which gk_paged_attn would not look at."""
    from gpt_decoder_gb300 import gk

    rng = np.random.default_rng(4200)
    H, Hkv, hs, page = 32, 8, 128, 16
    c, ns, gs, pl = shared_cache(rng, [(190, [(9, 1)] * 64)], Hkv, hs, page, True)
    c.table = np.pad(c.table[:, : 2048 // page], ((0, 0), (0, width // page - 2048 // page)), constant_values=-1)
    assert (64 * H * (hs * 4 + 8)) * 2 + 64 * 8 <= mib << 20
    q = serving.bf16(rng.standard_normal((64, H, hs)) * 2)
    ctx = gk.Ctx(_t().cuda.current_stream().cuda_stream, workspace_bytes=mib << 20)
    check_attention(*attend_shared(ctx, c, q, ns, gs, pl, 0.088), shared_ref(c, q, ns, gs, pl, 0.088))
    y, lse = attend_shared(ctx, c, q, ns, gs, pl, 0.088, max_group=63, fails=True)
    assert (y == 3).all() and (lse == 3).all()
    ctx.close()


# ---------------------------------------------------------------------------------------------- mass
# With scores near zero a weight is 2^(-l) alone, l the row's log sum in powers of two, and what is lost on the way from lse to
# the weight shows. In tiles it goes through a product, of 1 / f and -l in three bf16 parts each (a part rounds by 2^-9, so
# three leave 2^-27): its one step may cut the sum twice by a step of float32 (2 2^-23 |l|), and lse log2(e), 1 / f, the products of
# parts that are left out and the result times f each round by at most 2^-24 |l|: |l| 2^-21 in all, as the exponential's argument, so
# times ln 2 relative to the weight. The exponential itself: 2^-22. Scores: sums of hs products with scale sum |q||k| < 2^-4.9 (asserted),
# hs + 16 cuts of 2^-23 of that: below 2^-20.7. A key's sum over its N rows and heads: at most min(N, 48) additions in a chain (a
# thread has four sums of a tile's 128 rows, then joins them, and there are three pairs of tiles at most): 2^-24 each.
# A log sum of two parts would be off by up to 2^-18 |l|; one whose step comes first in the product is cut hs / 16 times more, always to the
# same side: by |l| 2^-24 in the mean each time, which the sum over all keys shows (there the chains' roundings average out).
def mass_and_bounds(c, q, lse, n, scale):
    """{place: (mass, bound)} in 64 bits, and the sums over all keys of both without the chains' roundings."""
    qs, G, out, total = starts(n), q.shape[1] // c.Hkv, {}, np.zeros(2)
    for b in range(len(n)):
        kv = int(c.kv_len[b])
        pos = np.arange(kv)
        pg, rw = (np.array(x) for x in zip(*(c.place(b, j) for j in range(kv))))
        k = np.stack([c.vector("k", p, r) for p, r in zip(pg, rw)])  # [kv, Hkv, hs]
        rows = slice(qs[b], qs[b + 1])
        seen = pos[None] <= (kv - n[b] + np.arange(n[b]))[:, None]
        for hk in range(c.Hkv):
            heads = slice(hk * G, hk * G + G)
            z = scale * np.einsum("ihd,jd->ihj", q[rows, heads].astype(np.float64), k[:, hk])
            l = lse[rows, heads].astype(np.float64)[..., None]
            size = scale * np.einsum("ihd,jd->ihj", np.abs(q[rows, heads]).astype(np.float64), np.abs(k[:, hk]))
            assert size.max() < 2.0 ** -4.9
            w = np.exp(z - l) * seen[:, None]
            bound = w * (np.abs(l) * 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -20.7)  # (|l| log2(e) ln(2) = |lse|)
            m, e = w.sum((0, 1)), bound.sum((0, 1))
            total += m.sum(), (w * (np.abs(l) * 2.0 ** -22 + 2.0 ** -22 + 2.0 ** -20.7)).sum()
            chain = np.minimum(seen.sum(0) * G, 48) * 2.0 ** -24
            for j in range(kv):
                out[pg[j], hk, rw[j]] = m[j], e[j] + chain[j] * m[j]
    return out, total


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kv_len,n,H,Hkv,hs,page", [
    ([300, 700, 90, 1500], [70, 90, 66, 80], 4, 4, 64, 16),
    ([2000, 400, 130], [128, 100, 129], 3, 3, 128, 64),
    ([600, 1800], [33, 40], 8, 4, 96, 32),
    ([900, 128], [30, 20], 4, 1, 128, 128),
    ([500, 90, 1700], [1, 3, 2], 8, 4, 64, 32),  # few rows: scores in registers
    ([500, 90, 1700], [16, 9, 12], 8, 2, 128, 64),
])
def test_mass_keeps_float32_of_the_log_sums(gkctx, kv_len, n, H, Hkv, hs, page, q8):
    rng = np.random.default_rng(4300 + hs + len(n))
    c = cache(rng, kv_len, Hkv, hs, page, q8)
    q = serving.bf16(rng.standard_normal((sum(n), H, hs)) * 2.0 ** -9)
    scale = hs ** -0.5
    # log sums as attention leaves them, and others that spread over more sizes
    lse = serving.paged_attn(c, q, starts(n), scale)[1]
    for ls in (lse, lse + rng.uniform(-1, 6, lse.shape)):
        ls = ls.astype(np.float32)
        got = weigh(gkctx, c, q, ls, n, scale)
        want, total = mass_and_bounds(c, q, ls, n, scale)
        at = tuple(np.array(x) for x in zip(*want))
        m, e = (np.array(x) for x in zip(*want.values()))
        off = np.abs(got[at] - m)
        assert (off <= e).all(), (float((off / e).max()), int((off > e).sum()), len(e))
        assert abs(got[at].astype(np.float64).sum() - total[0]) <= total[1], (got[at].astype(np.float64).sum() - total[0]) / total[1]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kv_len,n,H,Hkv,hs,first", [([300, 130], [1, 4], 4, 2, 64, [7, 0]), ([700, 260], [100, 65], 2, 2, 128, [0, 129]),
                                                     ([400], [70], 3, 1, 80, None)])
def test_mass_in_place_gives_the_bits_of_another_array(gkctx, kv_len, n, H, Hkv, hs, first, q8):
    """At every weighed key, and nothing else is touched."""
    rng = np.random.default_rng(4400 + hs)
    c = cache(rng, kv_len, Hkv, hs, 16, q8)
    q = serving.bf16(rng.standard_normal((sum(n), H, hs)) * 2)
    scale = hs ** -0.5
    lse = serving.paged_attn(c, q, starts(n), scale)[1].astype(np.float32)
    first = None if first is None else np.array(first, np.int32)
    weighed = np.zeros(c.k.shape[:3], bool)
    for at in serving.paged_mass(c, q, lse, starts(n), scale, first=first):
        weighed[at] = True
    assert weighed.any() and not weighed.all()
    old = rng.uniform(0, 2, weighed.shape).astype(np.float32)
    apart = weigh(gkctx, c, q, lse, n, scale, old=dev(old), decay=0.75, first=first, mass=dev(np.full(old.shape, 5, np.float32)))
    mass = dev(old)
    in_place = weigh(gkctx, c, q, lse, n, scale, old=mass, decay=0.75, first=first, mass=mass)
    assert np.array_equal(in_place[weighed], apart[weighed]) and (in_place[weighed] != old[weighed]).all()
    assert np.array_equal(in_place[~weighed], old[~weighed]) and (apart[~weighed] == 5).all()


@pytest.mark.parametrize("n,H,Hkv,hs,q8", [(1, 4, 2, 64, True), (1, 8, 2, 128, False), (90, 4, 2, 128, True), (200, 2, 2, 64, False)])
def test_mass_and_evict_replayed_on_other_lengths(n, H, Hkv, hs, q8):
    """A captured call against an eager one, all outputs (scales among them) after each replay: lengths, page tables, `first` and
    inputs change between them, and the last of them is not what was captured either."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(4500 + n + hs)
    c = cache(rng, [1500, 900], Hkv, hs, 64, q8)
    to = to_pages(rng, c, [300, 300], False)
    w, qs = H * hs, dev(starts([n, n]))
    d, td = Dev(c, poison=False), Dev(to, poison=False)
    q = dev(serving.bf16(rng.standard_normal((2 * n, w))), t.bfloat16)
    lse, first = t.zeros(2 * n, H, device="cuda"), dev(np.array([20, 0], np.int32))

    class Out:
        def __init__(self):
            self.mass, self.to_mass = t.zeros(c.k.shape[:3], device="cuda"), t.zeros(to.k.shape[:3], device="cuda")
            self.k, self.v = (t.zeros_like(x) for x in (td.k, td.v))
            self.ks, self.vs = (None if x is None else t.zeros_like(x) for x in (td.ks, td.vs))
            self.new, self.kept = t.zeros(2, dtype=t.int32, device="cuda"), t.zeros(2, Hkv, 280, dtype=t.int32, device="cuda")
            self.h = gk.PagedKv(self.k, self.v, self.ks, self.vs, td.table, self.new)

        def all(self):
            return [x for x in (self.mass, self.to_mass, self.k, self.v, self.ks, self.vs, self.new, self.kept) if x is not None]

    def call(ctx, o):
        y = spare
        gk.gk_paged_attn(ctx, d.h, gk.GK_BF16, q, w, y, w, lse, qs, 2, H, 2 * n, n, 0.125)
        gk.gk_paged_mass(ctx, d.h, gk.GK_BF16, q, w, lse, None, 1.0, o.mass, first, qs, 2, H, 2 * n, n, 0.125)
        gk.gk_paged_evict(ctx, d.h, o.mass, o.h, o.to_mass, first, 280, 30, o.new, o.kept, 2)

    spare = t.zeros(2 * n, w, dtype=t.bfloat16, device="cuda")
    side = t.cuda.Stream()
    ctx, o = gk.Ctx(side, workspace_bytes=16 << 20), Out()
    eager = gk.Ctx(t.cuda.current_stream().cuda_stream, workspace_bytes=16 << 20)
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=side):
        call(ctx, o)
    turned = c.table[:, ::-1].copy()
    turned[1, :] = np.where(c.table[1] < 0, -1, c.table[1])
    for lens, firsts, table in (([n, n + 3], [0, 1], c.table), ([700, 900], [20, 0], c.table), ([n + 1300, 280], [9, 130], turned), ([1499, 281], [3, 7], c.table)):
        d.kv_len.copy_(dev(np.array(lens, np.int32)))
        first.copy_(dev(np.array(firsts, np.int32)))
        d.table.copy_(dev(table))
        q.copy_(dev(serving.bf16(rng.standard_normal((2 * n, w))), t.bfloat16))
        for x in o.all():
            x.zero_()
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        want = Out()
        call(eager, want)
        gk.gk_sync(eager)
        assert all(t.equal(a, b) for a, b in zip(o.all(), want.all())) and o.mass.abs().sum() > 0
        # and those against the oracle: the lengths that the call saw are these
        now = serving.Pages(c.k, c.v, c.k_scale, c.v_scale, table, np.array(lens, np.int32))
        blank = serving.Pages(*(None if x is None else np.zeros_like(x) for x in (to.k, to.v, to.k_scale, to.v_scale)), to.table, to.kv_len)
        mass = o.mass.cpu().numpy()
        new_len, kept = serving.paged_evict(now, mass, blank, np.zeros(to.k.shape[:3], np.float32), np.array(firsts, np.int32), 280, 30)
        assert np.array_equal(o.new.cpu().numpy(), new_len) and np.array_equal(o.kept.cpu().numpy(), kept)
        assert np.array_equal(o.k.float().cpu().numpy(), blank.k.astype(np.float32))
    gk.gk_sync(ctx)
    ctx.close()
    eager.close()


# ---------------------------------------------------------------------------------------------- eviction
@pytest.mark.parametrize("one_pool", [False, True])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kv_len,first,budget,recent,Hkv,hs,page", [([9000, 300], [8500, 64], 16, 4, 2, 64, 64), ([4100] * 20, [4000] * 20, 1, 0, 4, 16, 16),
                                                                    ([20000], [19999], 64, 32, 1, 32, 256)])
def test_evict_of_first_tokens_far_above_the_budget(gkctx, kv_len, first, budget, recent, Hkv, hs, page, q8, one_pool):
    """Every one of the first tokens moves, whatever the number of blocks that the budget gives."""
    rng = np.random.default_rng(4600 + budget)
    c = cache(rng, kv_len, Hkv, hs, page, q8)
    first = np.array(first, np.int32)
    to = to_pages(rng, c, np.minimum(kv_len, first + budget), one_pool)
    mass = np.exp(rng.standard_normal(c.k.shape[:3]) * 3).astype(np.float32)
    to_mass = mass if one_pool else np.full(to.k.shape[:3], 3, np.float32)
    got = evict(gkctx, c, mass, to, to_mass, first, budget, recent)
    check_evict(got, c, mass, to, to_mass, first, budget, recent)


@pytest.mark.parametrize("B,Hkv,width", [(1, 2, 390000), (160, 4, 48896), (2, 3, 16400)])
def test_evict_of_tables_as_wide_as_the_blocks_hold(gkctx, B, Hkv, width):
    """Close under what a block's shared memory has room for, in clusters of eight and alone."""
    rng = np.random.default_rng(4700 + B)
    page = 16
    lens = [int(x) for x in rng.integers(100, 900, B)]
    lens[0] = 9000
    c = cache(rng, lens, Hkv, 16, page, False)
    c.table = np.pad(c.table, ((0, 0), (0, width // page - c.table.shape[1])), constant_values=-1)
    to = to_pages(rng, c, np.minimum(lens, 90), False)
    mass = np.exp(rng.standard_normal(c.k.shape[:3]) * 3).astype(np.float32)
    to_mass = np.full(to.k.shape[:3], 3, np.float32)
    got = evict(gkctx, c, mass, to, to_mass, None, 90, 20)
    check_evict(got, c, mass, to, to_mass, None, 90, 20)


# ------------------------------------------------------------------------------------------ refusals
def test_evict_refuses_pools_that_share_some_arrays():
    """Two pools with one array of values, of steps or of masses would be read and written at unlike places; new_len over first
    would change what the call reads."""
    from gpt_decoder_gb300 import gk

    t = _t()
    ctx = gk.Ctx(t.cuda.current_stream().cuda_stream, workspace_bytes=0)
    for q8 in (False, True):
        c, to = (cache(np.random.default_rng(i), [20], 2, 32, 16, q8) for i in (1, 2))
        a, b = Dev(c, poison=False), Dev(to, poison=False)
        assert a.k.shape == b.k.shape
        ma, mb = (t.full(a.k.shape[:3], 4.0, device="cuda") for _ in range(2))
        new, kept = t.zeros(1, dtype=t.int32, device="cuda"), t.zeros(1, 2, 8, dtype=t.int32, device="cuda")
        before = [x.clone() for x in (b.k, b.v, ma, mb)]

        def call(k=b.k, v=b.v, ks=b.ks, vs=b.vs, m=mb, table=b.table, first=None):
            gk.gk_paged_evict(ctx, a.h, ma, gk.PagedKv(k, v, ks, vs, table, new), m, first, 8, 2, new, kept, 1)

        bad = [dict(m=ma), dict(v=a.v), dict(k=a.k), dict(k=a.k, v=a.v, ks=a.ks, vs=a.vs), dict(v=a.v, m=ma), dict(first=new)]
        for args in bad + ([dict(ks=a.ks), dict(vs=a.vs), dict(k=a.k, v=a.v, m=ma)] if q8 else []):
            refused(gk.GK_ERR_ARG, lambda: call(**args))
        gk.gk_sync(ctx)
        assert all(t.equal(x, y) for x, y in zip((b.k, b.v, ma, mb), before)) and (new == 0).all()
        call()
        gk.gk_sync(ctx)
        assert new.tolist() == [8]
    ctx.close()
