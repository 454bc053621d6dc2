"""Attention over shared prefixes, the tokens' attention weight and their eviction on the GPU against the float64
oracle, a run of them together, and what they refuse.

Tolerances, fixed from the arithmetic:
* attention over shared prefixes: as gk_paged_attn (tests/test_gpu_serving.py): U (|y| + spread) + 2^-10 spread, where a
  row's parts add one more float32 rounding each, far below them; lse within 2^-10.
* mass: a weight 2^(s - l) has an argument of float32 operations: the product's sum (hs 2^-23 of |q||k| scale at most, as
  above below 2^-11 for scores up to 64), s and l in powers of two with a rounding each (3 2^-24 of |s| + |l|), so the
  weight is off by 2^-11 + (|s| + |l|) 2^-22 relative, the exponential's own 2^-22 among it; sums of N terms add at
  most N 2^-24 relative, N <= 2^13 here (2^-11). Together 2^-10 of the size sum w (1 + |s| + |l|) that the oracle gives; and
  decay old has two roundings. Most masses are far nearer; a wrong mask, head or row is off by whole weights.
* eviction: exact.
"""
import math

import numpy as np
import pytest

from oracle import serving
from tests.test_gpu_serving import Dev, check_attention, dev, refused, starts
from tests.test_oracle_serving import cache

pytestmark = pytest.mark.gpu


def _t():
    import torch

    return torch


# ----------------------------------------------------------------------------------- shared prefixes
def shared_cache(rng, groups, Hkv, hs, page, q8):
    """groups: [(prefix, [(tail, n)])]. A cache whose sequences hold their group's prefix (whole pages shared, the page in
    which it ends copied), and (kv_len, n, group_start, prefix_len)."""
    tails = [(p, tail, n) for p, seqs in groups for tail, n in seqs]
    kv = [p + tail if tail >= 0 else 0 for p, tail, _ in tails]
    c = cache(rng, kv, Hkv, hs, page, q8)
    b = 0
    for p, seqs in groups:
        full = p // page
        lead = next(i for i in range(b, b + len(seqs)) if kv[i] >= p)
        if lead > b:  # a padding row first: it names the prefix's pages all the same
            c.table[b, : -(-p // page)] = c.table[lead, : -(-p // page)]
        for i in range(lead + 1, b + len(seqs)):
            if kv[i] < p:
                continue
            c.table[i, :full] = c.table[lead, :full]
            if p % page:
                for x in (c.k, c.v, c.k_scale, c.v_scale):
                    if x is not None:
                        x[c.table[i, full], :, : p % page] = x[c.table[lead, full], :, : p % page]
        b += len(seqs)
    group_start = starts([len(s) for _, s in groups])
    # room for 2048 positions: with less a call does not look at the groups
    c.table = np.pad(c.table, ((0, 0), (0, max(0, 2048 // page - c.table.shape[1]))), constant_values=-1)
    return c, [n for _, _, n in tails], group_start, np.array([p for p, _ in groups], np.int32)


def attend_shared(ctx, c, q, n, group_start, prefix, scale, extra_rows=0, pad=0, d=None, max_q=None, max_group=None, fails=False):
    from gpt_decoder_gb300 import gk

    t = _t()
    rows, H, hs = q.shape
    d = d or Dev(c)
    w, ld, B, G = H * hs, H * hs + pad, len(n), len(prefix)
    buf = t.full((rows + extra_rows, ld), float("nan"), dtype=t.bfloat16, device="cuda")
    buf[:rows, :w] = dev(q.reshape(rows, w), t.bfloat16)
    y = t.full((rows + extra_rows, ld), 3.0, dtype=t.bfloat16, device="cuda")
    lse = t.full((rows + extra_rows, H), 3.0, device="cuda")
    qs = starts(n)
    most = max_group or max(1, *(int(qs[min(B, group_start[g + 1])] - qs[group_start[g]]) for g in range(G)))
    gk.gk_paged_attn_shared(ctx, d.h, gk.GK_BF16, buf, ld, y, ld, lse, dev(qs), B, dev(group_start), dev(prefix), G, H, rows + extra_rows,
                            max_q or max(max(n), 1), most, scale)
    if fails:
        with pytest.raises(gk.GkError) as e:
            gk.gk_sync(ctx)
        assert e.value.status == gk.GK_ERR_INDEX
    else:
        gk.gk_sync(ctx)
    y, lse = y.float().cpu().numpy(), lse.cpu().numpy()
    assert (y[rows:] == 3).all() and (y[:, w:] == 3).all() and (lse[rows:] == 3).all()
    return y[:rows, :w].reshape(rows, H, hs).astype(np.float64), lse[:rows].astype(np.float64)


def shared_ref(c, q, n, group_start, prefix, scale):
    groups = [(int(group_start[g]), int(group_start[g + 1]), int(prefix[g])) for g in range(len(prefix))]
    return serving.paged_attn(serving.SharedPages(c, groups, starts(n)), q, starts(n), scale)


SHARED = [  # groups (prefix, [(own tokens or -1: a padding row, new rows)]), H, Hkv, hs, page
    ([(40, [(1, 1), (5, 1), (17, 1)])], 2, 2, 16, 16),
    ([(777, [(40, 1), (3, 1), (1, 1), (16, 1)])], 12, 12, 64, 16),
    ([(64, [(10, 1)] * 9), (1, [(2, 1), (3, 2)]), (0, [(90, 3)]), (130, [(4, 4), (-1, 1)])], 4, 2, 64, 32),
    ([(1000, [(300, 1)] * 20), (3000, [(129, 1)] * 5)], 8, 2, 128, 64),
    ([(2000, [(20, 1)] * 33)], 2, 2, 80, 128),  # 33 rows of a key / value head
    ([(2500, [(1, 1)] * 70), (100, [(200, 1)] * 65)], 1, 1, 64, 16),
    ([(513, [(70, 64), (65, 65), (300, 1)]), (128, [(128, 128)])], 2, 1, 64, 64),
    ([(300, [(40, 40), (60, 33), (200, 129)])], 6, 3, 96, 32),
    ([(1500, [(260, 200), (333, 257)]), (2, [(700, 600), (4, 3)])], 2, 2, 128, 256),
    ([(5000, [(37, 5)] * 12), (6000, [(-1, 2), (9, 9)])], 4, 4, 32, 16),
    ([(90 + i, [(3, 1), (5, 2)]) for i in range(40)] + [(2048, [(1, 1)] * 3)], 2, 1, 32, 32),  # more groups than a lookup's round
    ([(200, [(3, 3), (500, 40)]), (9000, [(1, 1), (2, 2)] * 4)], 16, 2, 48, 128),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_shared_prefixes(gkctx, case, q8):
    """Each also with no more room in the table than there are tokens, where short prefixes are not shared."""
    groups, H, Hkv, hs, page = SHARED[case]
    rng = np.random.default_rng(2000 + case)
    c, n, gs, prefix = shared_cache(rng, groups, Hkv, hs, page, q8)
    q = serving.bf16(rng.standard_normal((sum(n), H, hs)) * 2)
    scale = 1 / math.sqrt(hs)
    ref = shared_ref(c, q, n, gs, prefix, scale)
    assert 2 * len(prefix) <= len(n)
    check_attention(*attend_shared(gkctx, c, q, n, gs, prefix, scale, extra_rows=case % 3, pad=8 * (case % 2)), ref)
    c.table = np.ascontiguousarray(c.table[:, : -(-int(c.kv_len.max()) // page)])
    check_attention(*attend_shared(gkctx, c, q, n, gs, prefix, scale), ref)


# ---------------------------------------------------------------------------------------------- mass
def weigh(ctx, c, q, lse, n, scale, old=None, decay=1.0, first=None, mass=None, d=None, pad=0, extra_rows=0, max_q=None, fails=False):
    """The pool's masses (device order) after the call; what the call leaves alone holds 5."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rows, H, hs = q.shape
    d = d or Dev(c)
    ld = H * hs + pad
    buf = t.full((rows + extra_rows, ld), float("nan"), dtype=t.bfloat16, device="cuda")
    buf[:rows, : H * hs] = dev(q.reshape(rows, H * hs), t.bfloat16)
    ls = t.full((rows + extra_rows, H), float("nan"), device="cuda")
    ls[:rows] = dev(lse.astype(np.float32))
    mass = t.full(c.k.shape[:3], 5.0, device="cuda") if mass is None else mass
    gk.gk_paged_mass(ctx, d.h, gk.GK_BF16, buf, ld, ls, old, decay, mass, dev(first), dev(starts(n)), len(n), H, rows + extra_rows,
                     max_q or max(max(n), 1), scale)
    if fails:
        with pytest.raises(gk.GkError) as e:
            gk.gk_sync(ctx)
        assert e.value.status == gk.GK_ERR_INDEX
    else:
        gk.gk_sync(ctx)
    return mass.cpu().numpy()


def check_mass(got, ref, untouched=5.0):
    want, tol = np.full(got.shape, untouched, np.float64), np.zeros(got.shape)
    for at, (m, size) in ref.items():
        want[at], tol[at] = m, 2.0 ** -10 * size + 2.0 ** -100
    odd = np.isnan(want)
    assert np.array_equal(odd, np.isnan(got)), np.argwhere(odd != np.isnan(got))[:5].tolist()
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= tol) & ~odd & (got != want)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


MASS = [  # kv_len, n, H, Hkv, hs, page, first
    ([1], [1], 1, 1, 16, 16, None),
    ([777], [1], 12, 12, 64, 16, [4]),
    ([0, 130, 1, 128, 129, 15, 16, 17], [1] * 8, 8, 2, 128, 16, [0, 130, 0, 5, 200, -3, 15, 16]),
    ([64, 65, 700, 33], [1, 3, 0, 2], 4, 4, 80, 32, None),
    ([3, 1500], [5, 4], 8, 2, 32, 128, [2, 1400]),  # more rows than tokens
    ([200, 300], [17, 16], 4, 2, 64, 16, [190, 7]),
    ([333, 65, 400], [65, 65, 1], 1, 1, 128, 64, None),
    ([300, 300, 128, 129], [129, 128, 127, 1], 2, 1, 64, 16, [1, 299, 0, 128]),
    ([513, 77], [200, 77], 6, 3, 96, 32, None),
    ([700], [300], 8, 1, 128, 64, [150]),
    ([1100, 20], [260, 20], 3, 3, 48, 256, None),
    ([140] * 40, [2] * 40, 5, 5, 112, 16, [16] * 40),
    ([2600, 0, 900], [513, 3, 600], 2, 2, 64, 128, [129, 0, 0]),
    ([3000], [2], 16, 2, 128, 64, None),
    ([400, 130], [70, 33], 6, 2, 64, 16, [3, 128]),  # three heads a key head: 42 queries of a tile of 128 rows, 126 rows
    ([300], [50], 10, 2, 96, 32, None),  # five
    ([150], [3], 200, 1, 32, 16, None),  # 200: a query's heads fill two tiles, the second in part
    ([290, 40], [90, 1], 24, 2, 128, 128, [256, 0]),  # twelve
    ([64], [64], 8, 1, 64, 16, None),
    ([2000], [2000], 1, 1, 16, 256, [1999]),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("case", range(len(MASS)))
def test_mass(gkctx, case, q8):
    kv_len, n, H, Hkv, hs, page, first = MASS[case]
    rng = np.random.default_rng(2100 + case)
    c = cache(rng, kv_len, Hkv, hs, page, q8)
    q = serving.bf16(rng.standard_normal((sum(n), H, hs)) * 2)
    scale = 1 / math.sqrt(hs)
    lse = serving.paged_attn(c, q, starts(n), scale)[1].astype(np.float32)
    first = None if first is None else np.array(first, np.int32)
    got = weigh(gkctx, c, q, lse, n, scale, first=first, pad=8 * (case % 2), extra_rows=case % 3)
    check_mass(got, serving.paged_mass(c, q, lse, starts(n), scale, first=first))
    if first is None:  # every row gives a weight of one for each head
        alone = [b for b in range(len(n)) if n[b] and kv_len[b] >= n[b]]
        total = sum(float(got[at[0], :, at[1]].astype(np.float64).sum()) for b in alone for at in (c.place(b, j) for j in range(kv_len[b])))
        assert abs(total - H * sum(n[b] for b in alone)) < 2.0 ** -9 * H * max(1, sum(n))
    # added to masses before, forgetting some: into another array and in place, the same bits
    old = rng.uniform(0, 2, c.k.shape[:3]).astype(np.float32)
    mass = dev(old)
    more = weigh(gkctx, c, q, lse, n, scale, old=dev(old), decay=0.75, first=first)
    check_mass(more, serving.paged_mass(c, q, lse, starts(n), scale, old=old, decay=0.75, first=first))
    same = weigh(gkctx, c, q, lse, n, scale, old=mass, decay=0.75, first=first, mass=mass)
    assert np.array_equal(np.where(same == old, 5.0, same), np.where((more == 5) | (same == old), 5.0, more))


# ------------------------------------------------------------------------------------------ eviction
def to_pages(rng, c, new_len, one_pool, spare=1):
    """Pages for sequences of these lengths: others of c's arrays, or a pool of their own (filled with a mark)."""
    page = c.page
    need = [-(-int(x) // page) for x in new_len]
    table = np.full((len(need), max(1, max(need))), -1, np.int32)
    base = c.n_pages if one_pool else 0
    ids = base + rng.permutation(sum(need) + spare)[: sum(need)]
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at : at + k]
        at += k
    new = lambda x: None if x is None else np.full((sum(need) + spare, *x.shape[1:]), 3, x.dtype)  # noqa: E731
    if not one_pool:
        return serving.Pages(new(c.k), new(c.v), new(c.k_scale), new(c.v_scale), table, np.zeros(len(need), np.int32))
    c.k, c.v, c.k_scale, c.v_scale = (None if x is None else np.concatenate([x, new(x)]) for x in (c.k, c.v, c.k_scale, c.v_scale))
    c.n_pages = c.k.shape[0]
    return other_table(c, table)


def other_table(c, table):
    """The same arrays under another table."""
    to = serving.SharedPages.__new__(serving.SharedPages)
    to.__dict__.update(c.__dict__, table=table, lead={})
    return to


def evict(ctx, c, mass, to, to_mass, first, budget, recent, fails=False):
    """The call on the GPU: (k, v, k_scale, v_scale, mass) of `to`, new_len, kept."""
    from gpt_decoder_gb300 import gk

    t = _t()
    one = to.k is c.k
    src = Dev(c, poison=False)
    dst = src if one else Dev(to, poison=False)
    m = dev(mass)
    tm = m if one else dev(to_mass)
    B = len(c.kv_len)
    new_len = t.full((B,), -9, dtype=t.int32, device="cuda")
    kept = t.full((B, c.Hkv, budget), -9, dtype=t.int32, device="cuda")
    h = gk.PagedKv(dst.k, dst.v, dst.ks, dst.vs, dev(to.table), new_len)
    gk.gk_paged_evict(ctx, src.h, m, h, tm, dev(first), budget, recent, new_len, kept, B)
    if fails:
        with pytest.raises(gk.GkError) as e:
            gk.gk_sync(ctx)
        assert e.value.status == gk.GK_ERR_INDEX
    else:
        gk.gk_sync(ctx)
    out = [None if x is None else x.float().cpu().numpy() for x in (dst.k, dst.v, dst.ks, dst.vs, tm)]
    return out, new_len.cpu().numpy(), kept.cpu().numpy()


def check_evict(got, c, mass, to, to_mass, first, budget, recent):
    out, new_len, kept = got
    nr, kr = serving.paged_evict(c, mass, to, to_mass, first, budget, recent)
    assert np.array_equal(new_len, nr) and np.array_equal(kept, kr)
    for x, y in zip(out, (to.k, to.v, to.k_scale, to.v_scale, to_mass)):
        if y is not None:
            assert np.array_equal(x, y.astype(np.float32), equal_nan=True)


EVICT = [  # kv_len, first, budget, recent, Hkv, hs, page
    ([20], None, 8, 2, 1, 16, 16),
    ([1], None, 1, 0, 2, 32, 16),
    ([100, 0, 17, 16, 300], [4, 0, 4, 4, 30], 16, 5, 3, 80, 16),
    ([700, 3, 130], [16, 5, 2], 64, 64, 2, 128, 64),  # the last ones alone
    ([700, 3, 130], None, 64, 0, 2, 64, 32),  # the heaviest alone
    ([1100], [4], 512, 64, 12, 64, 16),
    ([5000, 2100, 2049], [1, 0, 2000], 2048, 100, 2, 48, 256),
    ([3000] * 5, [129, 0, 3000, 9000, -4], 1000, 999, 4, 112, 128),
    ([40] * 70, [3] * 70, 11, 4, 2, 16, 16),
    ([40000, 20], None, 300, 7, 2, 32, 128),
]


@pytest.mark.parametrize("one_pool", [False, True])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("case", range(len(EVICT)))
def test_evict(gkctx, case, q8, one_pool):
    kv_len, first, budget, recent, Hkv, hs, page = EVICT[case]
    rng = np.random.default_rng(2200 + case)
    c = cache(rng, kv_len, Hkv, hs, page, q8)
    first = None if first is None else np.array(first, np.int32)
    f = np.zeros(len(kv_len), int) if first is None else np.clip(first, 0, kv_len)
    to = to_pages(rng, c, np.minimum(kv_len, f + budget), one_pool)
    mass = np.exp(rng.standard_normal(c.k.shape[:3]) * 3).astype(np.float32)
    mass *= rng.random(mass.shape) > 0.2  # zeros: ties
    to_mass = mass if one_pool else np.full(to.k.shape[:3], 3, np.float32)
    got = evict(gkctx, c, mass, to, to_mass, first, budget, recent)
    check_evict(got, c, mass, to, to_mass, first, budget, recent)


@pytest.mark.parametrize("values", ["equal", "few", "odd", "near"])
def test_evict_ties_and_odd_masses(gkctx, values):
    rng = np.random.default_rng(2300)
    c = cache(rng, [3000, 500], 4, 32, 32, False)
    shape = c.k.shape[:3]
    mass = {"equal": lambda: np.full(shape, 0.25), "few": lambda: rng.integers(-2, 3, shape) * 1.0,
            "odd": lambda: rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, 3e38, -3e38], shape),
            "near": lambda: 1 + rng.integers(0, 400, shape) * 2.0 ** -23}[values]().astype(np.float32)
    for budget, recent in ((100, 10), (1, 0), (499, 1), (2999, 0)):
        to = to_pages(rng, c, np.minimum([3000, 500], budget), False)
        to_mass = np.full(to.k.shape[:3], 3, np.float32)
        got = evict(gkctx, c, mass, to, to_mass, None, budget, recent)
        check_evict(got, c, mass, to, to_mass, None, budget, recent)


# ------------------------------------------------------------------- what is not finite, bad pages and lengths
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("S,n,H,Hkv,hs", [(4, 1, 2, 2, 64), (40, 1, 2, 1, 128), (3, 70, 2, 1, 64), (5, 50, 1, 1, 128)])
def test_shared_infinities_and_nan(gkctx, S, n, H, Hkv, hs, q8):
    """Values of the prefix, of its last page, of a sequence's own tokens and of the last new one that are not finite, and a
    NaN key: in the rows that see them and no others."""
    rng = np.random.default_rng(2400 + S)
    groups = [(333, [(n + 20, n)] * S), (300, [(n + 1, n)] * S), (200, [(n, n), (n + 3, n)])]
    c, ns, gs, prefix = shared_cache(rng, groups, Hkv, hs, 16, q8)

    def spoil(which, b, pos):
        p, r = c.place(b, pos)
        if q8:
            (c.v_scale if which == "v" else c.k_scale)[p, 0, r] = np.nan
        elif which == "v":
            c.v[p, 0, r, 5], c.v[p, -1, r, 9] = np.inf, np.nan
        else:
            c.k[p, 0, r, 3] = np.nan

    spoil("v", 0, 333 + n + 19)  # the first sequence's last token
    spoil("v", 1, 333)  # an own token, in the page in which the prefix ends
    spoil("k", 2, 340)
    spoil("v", S, 7)  # a prefix: the whole second group
    spoil("v", 2 * S + 1, 200)  # the first own token of the last sequence, at the start of a page's half
    q = serving.bf16(rng.standard_normal((sum(ns), H, hs)))
    ref = shared_ref(c, q, ns, gs, prefix, 0.125)
    y, lse = attend_shared(gkctx, c, q, ns, gs, prefix, 0.125)
    odd = ~np.isfinite(ref[0])
    assert odd.any() and not odd.all() and np.array_equal(odd, ~np.isfinite(y)), np.argwhere(odd != ~np.isfinite(y))[:5].tolist()
    tol = 2.0 ** -8 * (np.abs(ref[0]) + ref[2]) + 2.0 ** -10 * ref[2]
    assert (np.abs(y[~odd] - ref[0][~odd]) <= tol[~odd]).all()
    assert np.array_equal(np.isnan(lse), np.isnan(ref[1]))


@pytest.mark.parametrize("n", [1, 3, 90])
def test_shared_bad_pages_and_groups(gkctx, n):
    from gpt_decoder_gb300 import gk

    rng = np.random.default_rng(2500 + n)
    c, ns, gs, prefix = shared_cache(rng, [(160, [(n + 9, n)] * 3), (96, [(n, n)] * 2)], 2, 64, 16, True)
    q = serving.bf16(rng.standard_normal((sum(ns), 2, 64)))
    want = shared_ref(c, q, ns, gs, prefix, 0.125)
    # a table page of the first prefix that does not exist, in every row
    good = c.table.copy()
    c.table[:3, 2] = c.n_pages
    y, lse = attend_shared(gkctx, c, q, ns, gs, prefix, 0.125, fails=True, d=Dev(c, poison=False))
    check_attention(y, lse, shared_ref(c, q, ns, gs, prefix, 0.125))
    c.table[:] = good
    # sequences in no group, a group that shares nothing
    for groups, lens in (([0, 2], [160]), ([0, 3, 5], [0, 96]), ([0, 3, 5], [-7, 5000]), ([0, 0, 3], [96, 160])):
        gs2, p2 = np.array(groups, np.int32), np.array(lens, np.int32)
        past = 5000 in lens
        y, lse = attend_shared(gkctx, c, q, ns, gs2, p2, 0.125, fails=past)
        check_attention(y, lse, want)
    # groups that cannot be: their rows are left as they were; the others are right
    for groups, lens, left, most in (([0, 3, 7], [160, 96], range(3, 5), 3 * n), ([0, 3, 5], [160, 96], range(0, 3), 3 * n - 1),
                                     ([0, 3, 5], [160, 96], range(0), 3 * n)):
        y, lse = attend_shared(gkctx, c, q, ns, np.array(groups, np.int32), np.array(lens, np.int32), 0.125, fails=bool(left), max_group=most)
        for b in range(5):
            rows = slice(b * n, b * n + n)
            if b in left:
                assert (y[rows] == 3).all() and (lse[rows] == 3).all()
            else:
                check_attention(y[rows], lse[rows], [w[rows] for w in want])
    gk.gk_sync(gkctx)


def test_mass_infinities_nan_and_refused_pages(gkctx):
    rng = np.random.default_rng(2600)
    for n, H, Hkv, hs in ((1, 4, 2, 64), (5, 2, 2, 128), (40, 2, 1, 64), (150, 2, 2, 64), (200, 1, 1, 128)):
        for q8 in (False, True):
            c = cache(rng, [n + 200, 100 + n, 0], Hkv, hs, 16, q8)
            q = serving.bf16(rng.standard_normal((2 * n + 1, H, hs)))
            ns = [n, n, 1]
            lse = serving.paged_attn(c, q, starts(ns), 0.125)[1].astype(np.float32)
            lse[n // 2] = -np.inf
            lse[n + n // 2, 0] = np.inf
            if n > 1:
                lse[0, H - 1] = np.nan
            p, r = c.place(0, 77)
            if q8:
                c.k_scale[p, 0, r] = np.nan
            else:
                c.k[p, 0, r, 1], c.k[c.place(0, n + 190)[0], 0, c.place(0, n + 190)[1], 2] = np.nan, -np.inf
            d = Dev(c)
            check_mass(weigh(gkctx, c, q, lse, ns, 0.125, d=d), serving.paged_mass(c, q, lse, starts(ns), 0.125))
            good = c.table.copy()
            c.table[0, 3], c.table[1, 0] = -1, c.n_pages
            d.table.copy_(dev(c.table))
            check_mass(weigh(gkctx, c, q, lse, ns, 0.125, d=d, fails=True), serving.paged_mass(c, q, lse, starts(ns), 0.125))
            c.table[:] = good
            # more rows than max_q: left as they were; lengths past the table
            d.table.copy_(dev(c.table))
            if n > 1:
                got = weigh(gkctx, c, q, lse, ns, 0.125, d=d, max_q=n - 1, fails=True)
                assert (got == 5).all()
            c.kv_len[0] = c.table.shape[1] * 16 + 3
            d = Dev(c, poison=False)
            ref = serving.paged_mass(c, q, lse, starts(ns), 0.125)
            check_mass(weigh(gkctx, c, q, lse, ns, 0.125, d=d, fails=True), ref)


def test_evict_bad_pages_and_lengths(gkctx):
    rng = np.random.default_rng(2700)
    for q8 in (False, True):
        c = cache(rng, [300, 100, 40], 2, 32, 16, q8)
        mass = rng.random(c.k.shape[:3]).astype(np.float32)
        c.table[0, 2], c.table[0, 18], c.table[1, 0] = -1, c.n_pages, 1 << 30  # 18: the last tokens, which stay
        to = to_pages(rng, c, [64, 64, 40], False)
        to.table[2, 1] = to.n_pages
        to_mass = np.full(to.k.shape[:3], 3, np.float32)
        got = evict(gkctx, c, mass, to, to_mass, None, 64, 20, fails=True)
        check_evict(got, c, mass, to, to_mass, None, 64, 20)
        # a length past the table, one below zero, and a table of `to` that is too short
        c = cache(rng, [300, 100, 40], 2, 32, 16, q8)
        mass = rng.random(c.k.shape[:3]).astype(np.float32)
        c.kv_len[:] = 5000, -3, 40
        to = to_pages(rng, c, [48, 16, 40], False)
        to_mass = np.full(to.k.shape[:3], 3, np.float32)
        got = evict(gkctx, c, mass, to, to_mass, None, 64, 20, fails=True)
        check_evict(got, c, mass, to, to_mass, None, 64, 20)


def test_evict_keeps_shared_pages_where_they_are(gkctx):
    """Both tables name a prefix's pages, which two sequences hold; and every page of a sequence that is not cut."""
    rng = np.random.default_rng(2800)
    c = cache(rng, [700, 500, 90], 3, 64, 16, True)
    c.table[1, :4] = c.table[0, :4]
    first = np.array([64, 64, 5], np.int32)
    to = to_pages(rng, c, [264, 264, 90], True)
    to.table[:2, :4] = c.table[:2, :4]
    to.table[2, :6] = c.table[2, :6]
    mass = rng.random(c.k.shape[:3]).astype(np.float32)
    before = c.k[c.table[0, :4]].copy()
    got = evict(gkctx, c, mass, to, mass, first, 200, 50)
    check_evict(got, c, mass, to, mass, first, 200, 50)
    assert np.array_equal(got[0][0][c.table[0, :4]], before)


# ------------------------------------------------------------------ workspaces, graphs, streams, far offsets
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("S,n,H,Hkv,hs", [(6, 1, 4, 2, 64), (70, 1, 4, 2, 128), (5, 40, 2, 2, 64), (4, 200, 4, 2, 128)])
def test_shared_small_workspace_graph_and_streams(gkctx, S, n, H, Hkv, hs, q8):
    """Any workspace will do; a captured call replays on changed lengths; two contexts at once give the bits of one."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(3000 + S)
    groups = [(2300, [(n + 40, n)] * S), (700, [(n, n)] * 3)]
    c, ns, gs, prefix = shared_cache(rng, groups, Hkv, hs, 64, q8)
    q = serving.bf16(rng.standard_normal((sum(ns), H, hs)))
    ref = shared_ref(c, q, ns, gs, prefix, 0.125)
    rows, w, B = sum(ns), H * hs, len(ns)
    part = rows * H * (hs * 4 + 8)
    for ws in (0, part, 2 * part + 8 * rows + 64, 3 << 20, 64 << 20):
        ctx = gk.Ctx(t.cuda.current_stream().cuda_stream, workspace_bytes=ws)
        check_attention(*attend_shared(ctx, c, q, ns, gs, prefix, 0.125), ref, ws)
        ctx.close()
    d, qd, qs, dgs, dpl = Dev(c, poison=False), dev(q.reshape(rows, w), t.bfloat16), dev(starts(ns)), dev(gs), dev(prefix)
    most = int(max(starts(ns)[gs[1:]] - starts(ns)[gs[:-1]]))

    def call(ctx, y, lse):
        gk.gk_paged_attn_shared(ctx, d.h, gk.GK_BF16, qd, w, y, w, lse, qs, B, dgs, dpl, 2, H, rows, n, most, 0.125)

    out = lambda: (t.zeros(rows, w, dtype=t.bfloat16, device="cuda"), t.zeros(rows, H, device="cuda"))  # noqa: E731
    side = t.cuda.Stream()
    ctx = gk.Ctx(side, workspace_bytes=64 << 20)
    y, lse = out()
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=side):
        call(ctx, y, lse)
    want = out()
    for cut in (0, 900, 0):  # prefixes shorter by so much, and with them the sequences
        p2, kv2 = np.maximum(prefix - cut, 0).astype(np.int32), c.kv_len.copy()
        kv2[:S] -= min(cut, 2300)
        kv2[S:] -= min(cut, 700)
        old, c.kv_len = c.kv_len, kv2
        d.kv_len.copy_(dev(kv2))
        dpl.copy_(dev(p2))
        y.fill_(7)
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        # the own keys now begin inside what was the prefix: the first sequence's pages and each one's own agree there
        r2 = shared_ref(c, q, ns, gs, p2, 0.125)
        check_attention(y.float().cpu().numpy().reshape(q.shape).astype(np.float64), lse.cpu().numpy().astype(np.float64), r2, cut)
        if cut == 0:
            want[0].copy_(y)
            want[1].copy_(lse)
        c.kv_len = old
    gk.gk_sync(ctx)
    ctx.close()
    ctxs = [gk.Ctx(t.cuda.Stream(), workspace_bytes=64 << 20) for _ in range(2)]
    got = [[out() for _ in range(8)] for _ in ctxs]
    t.cuda.synchronize()
    for i in range(8):
        for ctx, o in zip(ctxs, got):
            call(ctx, *o[i])
    for ctx, o in zip(ctxs, got):
        gk.gk_sync(ctx)
        assert all(t.equal(a, b) for each in o for a, b in zip(each, want))
        ctx.close()


def test_shared_8_bit_prefixes_a_few_heads_at_a_time(gkctx):
    """A workspace with room for the codes of three of five heads' prefixes as bf16: two turns, the second of two."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(3100)
    Hkv, G, hs, n, S, cap = 5, 8, 128, 40, 10, 65536
    c, ns, gs, prefix = shared_cache(rng, [(1900, [(n + 5, n)] * S), (100, [(n, n)] * 2)], Hkv, hs, 64, True)
    c.table = np.pad(c.table, ((0, 0), (0, cap // 64 - c.table.shape[1])), constant_values=-1)
    q = serving.bf16(rng.standard_normal((sum(ns), Hkv * G, hs)))
    ref = shared_ref(c, q, ns, gs, prefix, 0.1)
    a_head, part = 2 * cap * hs * 2, sum(ns) * Hkv * G * (hs * 4 + 8)  # two groups' keys; a part of every row
    ws = 9 * a_head
    assert ws // 2 < Hkv * a_head and 3 <= ws // 8 * 3 // a_head < 4 and 2 * 3 * 2 * -(-S * n * G // 256) >= 152 and 3 * a_head > 2 * part + 8 * sum(ns)
    ctx = gk.Ctx(t.cuda.current_stream().cuda_stream, workspace_bytes=ws)
    check_attention(*attend_shared(ctx, c, q, ns, gs, prefix, 0.1), ref)
    ctx.close()


def test_mass_and_evict_graph_and_streams(gkctx):
    """Captured and replayed on changed lengths, beside another context's calls: the bits of one alone."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(3200)
    for n, H, Hkv, hs, q8 in ((1, 4, 2, 64, True), (1, 8, 2, 128, False), (90, 4, 2, 128, True), (200, 2, 2, 64, False)):
        c = cache(rng, [1500, 900], Hkv, hs, 64, q8)
        q, w, qs = serving.bf16(rng.standard_normal((2 * n, H, hs))), H * hs, dev(starts([n, n]))
        lse = serving.paged_attn(c, q, starts([n, n]), 0.125)[1].astype(np.float32)
        to = to_pages(rng, c, [300, 300], False)
        d, td, qd, ld = Dev(c, poison=False), Dev(to, poison=False), dev(q.reshape(2 * n, w), t.bfloat16), dev(lse)
        first = dev(np.array([20, 0], np.int32))

        class Out:
            def __init__(self):
                self.mass, self.to_mass = t.zeros(c.k.shape[:3], device="cuda"), t.zeros(to.k.shape[:3], device="cuda")
                self.k, self.v = (t.zeros_like(x) for x in (td.k, td.v))
                self.ks, self.vs = (None if x is None else t.zeros_like(x) for x in (td.ks, td.vs))
                self.new, self.kept = t.zeros(2, dtype=t.int32, device="cuda"), t.zeros(2, Hkv, 280, dtype=t.int32, device="cuda")
                self.h = gk.PagedKv(self.k, self.v, self.ks, self.vs, td.table, self.new)

            def all(self):
                return [x for x in (self.mass, self.to_mass, self.k, self.v, self.new, self.kept) if x is not None]

        def call(ctx, o):
            gk.gk_paged_mass(ctx, d.h, gk.GK_BF16, qd, w, ld, None, 1.0, o.mass, None, qs, 2, H, 2 * n, n, 0.125)
            gk.gk_paged_evict(ctx, d.h, o.mass, o.h, o.to_mass, first, 280, 30, o.new, o.kept, 2)

        want = Out()
        call(gkctx, want)
        gk.gk_sync(gkctx)
        side = t.cuda.Stream()
        ctx, o = gk.Ctx(side, workspace_bytes=0), Out()
        t.cuda.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            call(ctx, o)
        for lens in ([n, n + 3], [700, 900], [1500, 900]):
            d.kv_len.copy_(dev(np.array(lens, np.int32)))
            for x in o.all():
                x.zero_()
            t.cuda.synchronize()
            g.replay()
            t.cuda.synchronize()
            assert o.new.tolist() == [min(lens[0], 300), min(lens[1], 280)]
        assert all(t.equal(a, b) for a, b in zip(o.all(), want.all()))
        gk.gk_sync(ctx)
        ctx.close()
        ctxs, outs = [gk.Ctx(t.cuda.Stream(), workspace_bytes=0) for _ in range(2)], [[Out() for _ in range(5)] for _ in range(2)]
        t.cuda.synchronize()
        for i in range(5):
            for ctx, each in zip(ctxs, outs):
                call(ctx, each[i])
        for ctx, each in zip(ctxs, outs):
            gk.gk_sync(ctx)
            assert all(t.equal(a, b) for o in each for a, b in zip(o.all(), want.all()))
            ctx.close()


@pytest.mark.parametrize("q8", [False, True])
def test_shared_mass_and_evict_offsets_past_32_bits(gkctx, q8):
    """Pages whose first element lies past 2^32 elements of the cache: the bits of a small one."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(3300)
    Hkv, hs, page, n_pages = 8, 128, 128, 33000
    c, ns, gs, prefix = shared_cache(rng, [(2100, [(40, 1)] * 4), (1000, [(300, 200)] * 2)], Hkv, hs, page, q8)
    to = to_pages(rng, c, [400] * 6, True)
    assert (n_pages - c.n_pages) * Hkv * hs * page > 1 << 32
    d, rows, w, B = Dev(c, poison=False), sum(ns), Hkv * hs, len(ns)
    at = n_pages - c.n_pages
    q, qs = dev(rng.standard_normal((rows, w)).astype(np.float32), t.bfloat16), dev(starts(ns))
    results = []
    for base in (0, at):

        def big(x):  # the last pages are the small cache's
            if x is None or not base:
                return None if x is None else x.clone()
            y = t.empty(n_pages, *x.shape[1:], dtype=x.dtype, device="cuda")
            y[base:].copy_(x)
            return y

        k, v, ks, vs = (big(x) for x in (d.k, d.v, d.ks, d.vs))
        h = gk.PagedKv(k, v, ks, vs, d.table + base, d.kv_len)
        y, lse = t.zeros(rows, w, dtype=t.bfloat16, device="cuda"), t.zeros(rows, Hkv, device="cuda")
        gk.gk_paged_attn_shared(gkctx, h, gk.GK_BF16, q, w, y, w, lse, qs, B, dev(gs), dev(prefix), 2, Hkv, rows, 200, 400, 0.088)
        mass = t.zeros((n_pages if base else c.n_pages), Hkv, page, device="cuda")
        new, kept = t.zeros(B, dtype=t.int32, device="cuda"), t.zeros(B, Hkv, 400, dtype=t.int32, device="cuda")
        first = dev(np.array([0] * 6, np.int32))
        for b in range(4):  # (the group's sequences hold the prefix's pages together: one at a time)
            one = gk.PagedKv(k, v, ks, vs, (d.table + base)[b : b + 1], d.kv_len[b : b + 1])
            gk.gk_paged_mass(gkctx, one, gk.GK_BF16, q[b:], w, lse[b:], mass, 1.0, mass, None, dev(starts([1])), 1, Hkv, 1, 1, 0.088)
        for b in (4, 5):
            one = gk.PagedKv(k, v, ks, vs, (d.table + base)[b : b + 1], d.kv_len[b : b + 1])
            r = 4 + 200 * (b - 4)
            gk.gk_paged_mass(gkctx, one, gk.GK_BF16, q[r:], w, lse[r:], mass, 1.0, mass, None, dev(starts([200])), 1, Hkv, 200, 200, 0.088)
        gk.gk_paged_evict(gkctx, h, mass, gk.PagedKv(k, v, ks, vs, dev(to.table) + base, new), mass, first, 400, 100, new, kept, B)
        gk.gk_sync(gkctx)
        results.append([y, lse, mass[-c.n_pages :], k[-c.n_pages :], v[-c.n_pages :], new, kept])
    assert results[0][0].abs().sum() > 0 and results[0][2].sum() > 0
    for a, b in zip(*results):
        assert t.equal(a, b)


def test_evict_of_tables_wider_than_the_blocks_hold(gkctx):
    """More positions than a cluster's shared memory has room for: masses are read again for each digit."""
    rng = np.random.default_rng(3400)
    for kv, page in (([500000], 256), ([1000, 30], 64)):
        c = cache(rng, kv, 1, 16, page, False, spare=0)
        if len(kv) > 1:
            c.table = np.pad(c.table, ((0, 0), (0, 400000 // page)), constant_values=-1)
        mass = np.exp(rng.standard_normal(c.k.shape[:3]) * 3).astype(np.float32)
        to = to_pages(rng, c, [107] * len(kv), False)
        to_mass = np.full(to.k.shape[:3], 3, np.float32)
        got = evict(gkctx, c, mass, to, to_mass, None, 107, 9)
        check_evict(got, c, mass, to, to_mass, None, 107, 9)


# --------------------------------------------------------------------------------------- together
@pytest.mark.parametrize("q8", [False, True])
def test_sampling_from_a_prompt_under_a_budget(gkctx, q8):
    """Six continuations of two prompts: each step writes a token, attends over prompt and own tokens, adds the weights,
    and sequences past their budget are cut and go on in other pages. Against the oracle step by step."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(2900)
    H, Hkv, hs, page, B, budget, recent = 4, 2, 64, 16, 6, 24, 8
    first = np.array([37, 37, 37, 80, 80, 80], np.int32)
    groups = [(37, [(20, 1)] * 3), (80, [(20, 1)] * 3)]
    c, _, gs, prefix = shared_cache(rng, groups, Hkv, hs, page, q8)
    # room for all that is to come: every sequence has two sets of pages behind its prefix's whole ones
    width, spare, room = 8, 60, c.table.shape[1]
    grow = lambda x: None if x is None else np.concatenate([x, np.zeros((spare, *x.shape[1:]), x.dtype)])  # noqa: E731
    free = list(range(c.n_pages, c.n_pages + spare))
    c.k, c.v, c.k_scale, c.v_scale = (grow(x) for x in (c.k, c.v, c.k_scale, c.v_scale))
    c.n_pages = c.k.shape[0]
    full = [int(p) // page for p in first]
    table = c.table.copy()
    assert table.shape == (B, room) and room * page >= 2048
    for b in range(B):
        for j in range(-(-int(c.kv_len[b]) // page), width):
            table[b, j] = free.pop()
    c.table = table
    other = table.copy()
    for b in range(B):
        for j in range(full[b], width):
            other[b, j] = free.pop()
    mass = np.zeros(c.k.shape[:3], np.float32)
    d = Dev(c, poison=False)
    tables, now = [dev(table), dev(other)], 0
    hosts = [table, other]
    kv = [d.kv_len, t.zeros(B, dtype=t.int32, device="cuda")]
    dm = dev(mass)
    n, qs, w = [1] * B, starts([1] * B), H * hs
    dqs, dgs, dpl, dfirst = dev(qs), dev(gs), dev(prefix), dev(first)
    y = t.zeros(B, w, dtype=t.bfloat16, device="cuda")
    lse = t.zeros(B, H, device="cuda")
    cuts = 0
    for step in range(14):
        c.kv_len = c.kv_len + 1
        kv[now].add_(1)
        h = gk.PagedKv(d.k, d.v, d.ks, d.vs, tables[now], kv[now])
        new = serving.bf16(rng.standard_normal((B, (H + 2 * Hkv) * hs)) * 1.5)
        x = dev(new, t.bfloat16)
        gk.gk_paged_write(gkctx, h, gk.GK_BF16, x[:, w:], x.shape[1], x[:, w + Hkv * hs :], x.shape[1], dqs, B, B)
        gk.gk_paged_attn_shared(gkctx, h, gk.GK_BF16, x, x.shape[1], y, w, lse, dqs, B, dgs, dpl, 2, H, B, 1, 3, 0.125)
        gk.gk_paged_mass(gkctx, h, gk.GK_BF16, x, x.shape[1], lse, dm, 1.0, dm, dfirst, dqs, B, H, B, 1, 0.125)
        gk.gk_sync(gkctx)
        c.table = hosts[now]
        serving.paged_write(c, new[:, w : w + Hkv * hs].reshape(B, Hkv, hs), new[:, w + Hkv * hs :].reshape(B, Hkv, hs), qs)
        q = new[:, :w].reshape(B, H, hs)
        ref = shared_ref(c, q, n, gs, prefix, 0.125)
        ls = lse.cpu().numpy()
        check_attention(y.float().cpu().numpy().reshape(B, H, hs).astype(np.float64), ls.astype(np.float64), ref, step)
        want = mass.astype(np.float64)
        tol = np.zeros(want.shape)
        for at, (m, size) in serving.paged_mass(c, q, ls, qs, 0.125, old=mass, first=first).items():
            want[at], tol[at] = m, 2.0 ** -10 * size
        mass = dm.cpu().numpy()
        assert (np.abs(mass - want) <= tol).all()
        if int(c.kv_len[0]) - 37 > budget + 3:
            cuts += 1
            kept = t.zeros(B, Hkv, budget, dtype=t.int32, device="cuda")
            gk.gk_paged_evict(gkctx, h, dm, gk.PagedKv(d.k, d.v, d.ks, d.vs, tables[1 - now], kv[1 - now]), dm, dfirst, budget, recent,
                              kv[1 - now], kept, B)
            gk.gk_sync(gkctx)
            lens, kr = serving.paged_evict(c, mass, other_table(c, hosts[1 - now]), mass, first, budget, recent)
            assert np.array_equal(kept.cpu().numpy(), kr) and np.array_equal(kv[1 - now].cpu().numpy(), lens)
            assert np.array_equal(dm.cpu().numpy(), mass)
            assert np.array_equal(d.k.float().cpu().numpy(), c.k.astype(np.float32))
            now, c.kv_len = 1 - now, lens
    assert cuts >= 2


# --------------------------------------------------------------------------------- the measured cases
@pytest.mark.parametrize("name", ["shared_few", "shared_groups", "mass_one_token", "mass_chunk", "evict_one", "evict_step"])
def test_measured_cases_under_a_side_stream(monkeypatch, name):
    """The calls that they make, beside their plain forms, and again on a stream that is not the default one."""
    import torch

    from perf import more_operators

    case = next(c for c in more_operators.listed() if c["name"] == name)

    def outputs(own):
        monkeypatch.setattr(more_operators, "own", own)
        out = more_operators.run(more_operators.prepare(case, 3))
        return [x.clone() for x in (out if isinstance(out, tuple) else (out,))]

    plain, want = outputs(False), outputs(True)
    for a, b in zip(want, plain):
        if a.dtype == torch.int32 or name == "evict_one":
            assert torch.equal(a, b)
        else:  # both within a rounding or two of the same numbers (bf16; masses in 32 bits)
            assert ((a.float() - b.float()).abs() <= 2.0 ** (-6 if a.dtype == torch.bfloat16 else -14) * (b.float().abs() + 0.05)).all()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # the stream is about 10 ms behind the host: nothing is there yet by chance
        got = outputs(True)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------------------------------- refusals
def test_shared_mass_and_evict_refuse(gkctx):
    from gpt_decoder_gb300 import gk

    t = _t()
    A, L, UN = gk.GK_ERR_ARG, gk.GK_ERR_ALIGN, gk.GK_ERR_UNSUPPORTED
    c = cache(np.random.default_rng(1), [20], 2, 32, 16, True)
    d = Dev(c)
    y, qs, gs, pl = t.zeros(4, 64, dtype=t.bfloat16, device="cuda"), dev(starts([4])), dev(starts([1])), dev(np.array([16], np.int32))
    sh = lambda dt=gk.GK_BF16, q=y, ldq=64, o=y, gs=gs, pl=pl, G=1, H=2, rows=4, mq=4, mg=4, s=1.0: (  # noqa: E731
        gkctx, d.h, dt, q, ldq, o, 64, None, qs, 1, gs, pl, G, H, rows, mq, mg, s)
    for bad, status in ((dict(dt=gk.GK_F32), UN), (dict(q=None), A), (dict(H=3), A), (dict(H=4), A), (dict(mq=0), A), (dict(mg=0), A),
                        (dict(s=0.0), A), (dict(s=float("nan")), A), (dict(s=3e38), A), (dict(ldq=68), L), (dict(o=y.data_ptr() + 2), L),
                        (dict(gs=None), A), (dict(pl=None), A), (dict(G=0), A), (dict(G=65536), A), (dict(rows=-1), A),
                        (dict(rows=1 << 30, mq=1, mg=1 << 30), UN)):
        refused(status, gk.gk_paged_attn_shared, *sh(**bad))
    gk.gk_paged_attn_shared(*sh(rows=0))
    m, lse = t.full((c.n_pages, 2, 16), 4.0, device="cuda"), t.zeros(4, 2, device="cuda")
    ma = lambda dt=gk.GK_BF16, q=y, ldq=64, lse=lse, old=None, decay=1.0, m=m, H=2, rows=4, mq=4, s=1.0: (  # noqa: E731
        gkctx, d.h, dt, q, ldq, lse, old, decay, m, None, qs, 1, H, rows, mq, s)
    for bad, status in ((dict(dt=gk.GK_F32), UN), (dict(q=None), A), (dict(lse=None), A), (dict(m=None), A), (dict(H=3), A), (dict(mq=0), A),
                        (dict(decay=-1.0), A), (dict(decay=float("inf")), A), (dict(decay=float("nan")), A), (dict(s=-1.0), A),
                        (dict(ldq=56), A), (dict(ldq=68), L), (dict(m=m.data_ptr() + 4), L), (dict(old=m.data_ptr() + 8), L),
                        (dict(rows=1 << 31), A), (dict(rows=1 << 30, mq=1 << 30), UN)):
        refused(status, gk.gk_paged_mass, *ma(**bad))
    gk.gk_paged_mass(*ma(rows=0))
    to = cache(np.random.default_rng(2), [20], 2, 32, 16, True)
    dt_ = Dev(to)
    new, kept, tm = t.zeros(1, dtype=t.int32, device="cuda"), t.zeros(1, 2, 8, dtype=t.int32, device="cuda"), t.zeros(to.n_pages, 2, 16, device="cuda")
    ev = lambda m=m, to=dt_.h, tm=tm, budget=8, recent=2, new=new, kept=kept, B=1: (  # noqa: E731
        gkctx, d.h, m, to, tm, None, budget, recent, new, kept, B)
    for bad, status in ((dict(m=None), A), (dict(tm=None), A), (dict(new=None), A), (dict(kept=None), A), (dict(budget=0), A), (dict(recent=9), A),
                        (dict(recent=-1), A), (dict(budget=(1 << 30) + 1), A), (dict(B=0), A), (dict(new=d.kv_len), A),
                        (dict(m=m.data_ptr() + 4), L), (dict(tm=tm.data_ptr() + 4), L)):
        refused(status, gk.gk_paged_evict, *ev(**bad))
    for Hkv, hs, page, q8 in ((1, 32, 16, True), (2, 48, 16, True), (2, 32, 32, True), (2, 32, 16, False)):
        refused(A, gk.gk_paged_evict, *ev(to=Dev(cache(np.random.default_rng(3), [20], Hkv, hs, page, q8)).h))
    same = gk.PagedKv(d.k, d.v, d.ks, d.vs, d.table, new)
    refused(A, gk.gk_paged_evict, *ev(to=same))  # one pool, two arrays of masses
    s = dt_.h.struct
    for name, bad, status in (("page_size", 24, UN), ("hs", 24, UN), ("dtype", gk.GK_F32, A), ("k_scale", None, A), ("n_pages", 0, A),
                              ("ld_table", 1, A), ("v", s.v + 2, L), ("page_table", None, A)):
        old = getattr(s, name)
        setattr(s, name, bad)
        refused(status, gk.gk_paged_evict, *ev())
        setattr(s, name, old)
    with pytest.raises(ValueError):
        gk.gk_paged_evict(*ev(B=2))
    gk.gk_sync(gkctx)
    assert (m == 4).all() and (new == 0).all() and (kept == 0).all()
