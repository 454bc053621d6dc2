"""The serving operators on the GPU against the float64 oracle: the paged cache's write and read, attention of
new tokens over it, products with 4-bit weights, filtered sampling, a run of them together, and what they refuse.

Tolerances, fixed from the arithmetic (u = 2^-8 is bf16's rounding, half a step relative to the value):
* the cache: exact. Codes, scales and the values read back follow float32 operations step by step.
* attention: the result is rounded to bf16 (u |y|), each weight may be rounded to bf16 before the product with
  v (u times spread = sum p |v|), and scores carry float32 errors: a score is a sum of hs products whose running
  sum may be cut by one float32 step each (hs 2^-23 |q||k| scale, below 2^-11 for the inputs here) and the
  exponential's argument and result are good to 2^-20, together taken as 2^-10 of spread.
* lse: float32 scores of size up to S: absolute (hs + 8) 2^-23 S, with S <= 64 here below 2^-10.
* 4-bit products: K float32 additions of exact products, at most K 2^-24 of sum |x w| (the oracle's own sum of
  magnitudes), then one rounding.
* sampling: indices exact unless the decision lies within 1e-9 of the kept weight of going another way (none of
  these inputs does, which is asserted); probabilities to 2^-22.
"""
import math

import numpy as np
import pytest

from oracle import serving
from tests.test_oracle_serving import cache

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


def _t():
    import torch

    return torch


def dev(a, dtype=None):
    if a is None:
        return None
    t = _t().as_tensor(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


class Dev:
    """An oracle cache's arrays on the GPU, and the binding's handle."""

    def __init__(self, c, poison=True):
        from gpt_decoder_gb300 import gk

        t = _t()
        q8 = c.k_scale is not None
        self.k, self.v = (dev(a, t.int8 if q8 else t.bfloat16) for a in (c.k, c.v))
        self.ks, self.vs = dev(c.k_scale), dev(c.v_scale)
        self.table, self.kv_len = dev(c.table), dev(c.kv_len)
        if poison:  # what no position names holds NaN
            named = np.zeros((c.n_pages, c.page), bool)
            for b, n in enumerate(c.kv_len):
                for j in range(int(n)):
                    at = c.place(b, j)
                    if at is not None:
                        named[at] = True
            hole = dev(~named)
            for x, s in ((self.k, self.ks), (self.v, self.vs)):
                if q8:
                    s.masked_fill_(hole[:, None, :], float("nan"))
                else:
                    x.masked_fill_(hole[:, None, :, None], float("nan"))
        self.h = gk.PagedKv(self.k, self.v, self.ks, self.vs, self.table, self.kv_len)


def starts(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


# ------------------------------------------------------------------------------ cache write, read
CACHE = [  # kv_len, n, Hkv, hs, page
    ([1], [1], 1, 16, 16),
    ([5, 0, 17, 64], [5, 1, 3, 64], 12, 64, 16),
    ([100, 3, 31, 200, 0], [37, 0, 31, 130, 2], 3, 80, 32),
    ([2, 300], [5, 300], 8, 128, 64),  # more rows than tokens: the first three are padding
    ([260, 1, 256], [259, 1, 1], 5, 112, 256),
    ([40] * 70, [1] * 70, 2, 48, 16),  # more sequences than one round of the row lookup
    ([9000], [9000], 2, 32, 128),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("src", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(CACHE)))
def test_write_and_read_exact(gkctx, case, src, q8):
    from gpt_decoder_gb300 import gk

    t = _t()
    kv_len, n, Hkv, hs, page = CACHE[case]
    rng = np.random.default_rng(100 + case)
    c = cache(rng, kv_len, Hkv, hs, page, q8)
    q_start, rows, w = starts(n), int(sum(n)), Hkv * hs
    new = (rng.standard_normal((rows, 2 * w + 8)) * np.exp(rng.uniform(-8, 8, (rows, 1)))).astype(np.float32)
    if rows > 3:
        new[1, :hs] = 0  # a head of zeros
        new[2, w : w + hs] *= np.float32(2.0 ** -120)  # below the quantiser's smallest
        new[3, 2 * hs - 1 if Hkv > 1 else 0] = np.inf
        new[3, w] = np.nan
    new = new if src == "f32" else serving.bf16(new)
    d = Dev(c, poison=False)
    x = dev(new, None if src == "f32" else t.bfloat16)
    dt = gk.GK_F32 if src == "f32" else gk.GK_BF16
    gk.gk_paged_write(gkctx, d.h, dt, x, 2 * w + 8, x[:, w:], 2 * w + 8, dev(q_start), len(n), rows)
    gk.gk_sync(gkctx)
    serving.paged_write(c, new[:, :w].reshape(rows, Hkv, hs), new[:, w : 2 * w].reshape(rows, Hkv, hs), q_start)
    for a, b in ((d.k, c.k), (d.v, c.v), (d.ks, c.k_scale), (d.vs, c.v_scale)):  # the whole pool: nothing else changed
        if b is not None:
            assert np.array_equal(a.float().cpu().numpy(), b.astype(np.float32), equal_nan=True)
    # read whole sequences, with two rows of no sequence behind them and a wider row stride
    every = starts(np.maximum(kv_len, 1))
    for od, tdt in ((gk.GK_F32, t.float32), (gk.GK_BF16, t.bfloat16)):
        ko, vo = (t.full((every[-1] + 2, w + 16), 7.0, dtype=tdt, device="cuda") for _ in range(2))
        gk.gk_paged_read(gkctx, d.h, od, ko, w + 16, vo, w + 16, dev(every), len(n), every[-1] + 2)
        gk.gk_sync(gkctx)
        ref = serving.paged_read(c, every, every[-1])
        for o, r in zip((ko, vo), ref):
            o = o.float().cpu().numpy()
            r = r.reshape(every[-1], w)
            assert np.array_equal(o[:-2, :w], r if od == gk.GK_F32 else serving.bf16(r), equal_nan=True)
            assert (o[-2:] == 7).all() and (o[:, w:] == 7).all()


def test_write_and_read_refuse_bad_pages_on_the_device(gkctx):
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(7)
    c = cache(rng, [40, 16], 2, 32, 16, True)
    c.table[0, 1], c.table[1, 0] = c.n_pages, -1
    d = Dev(c, poison=False)
    before = d.k.clone()
    q_start, x = starts([10, 1]), dev(rng.standard_normal((11, 64)).astype(np.float32))
    gk.gk_paged_write(gkctx, d.h, gk.GK_F32, x, 64, x, 64, dev(q_start), 2, 11)
    with pytest.raises(gk.GkError) as e:
        gk.gk_sync(gkctx)
    assert e.value.status == gk.GK_ERR_INDEX
    changed = (d.k != before).flatten(2).any(2).any(1).cpu().numpy()
    assert set(np.flatnonzero(changed)) == {int(c.table[0, 2])}  # positions 32..39 only
    out = [t.full((11, 64), 5.0, device="cuda") for _ in range(2)]
    gk.gk_paged_read(gkctx, d.h, gk.GK_F32, out[0], 64, out[1], 64, dev(q_start), 2, 11)
    with pytest.raises(gk.GkError):
        gk.gk_sync(gkctx)
    assert (out[0][[0, 1, 10]] == 0).all() and (out[0][2:10] != 0).any()
    # a length past the table: the row is refused, the others are not
    d.kv_len.copy_(t.tensor([49, 0], dtype=t.int32))
    gk.gk_paged_read(gkctx, d.h, gk.GK_F32, out[0], 64, out[1], 64, dev(q_start), 2, 11)
    with pytest.raises(gk.GkError):
        gk.gk_sync(gkctx)
    assert (out[0][9] == 0).all() and (out[0][8] != 0).any()


# ------------------------------------------------------------------------------------- attention
def attend(gkctx, c, q, n, scale, q8=None, extra_rows=0, pad=0, max_q=None, d=None):
    from gpt_decoder_gb300 import gk

    t = _t()
    rows, H, hs = q.shape
    d = d or Dev(c)
    w, ld = H * hs, H * hs + pad
    buf = t.full((rows + extra_rows, ld), float("nan"), dtype=t.bfloat16, device="cuda")
    buf[:rows, :w] = dev(q.reshape(rows, w), t.bfloat16)
    y = t.full((rows + extra_rows, ld), 3.0, dtype=t.bfloat16, device="cuda")
    lse = t.full((rows + extra_rows, H), 3.0, device="cuda")
    gk.gk_paged_attn(gkctx, d.h, gk.GK_BF16, buf, ld, y, ld, lse, dev(starts(n)), len(n), H, rows + extra_rows,
                     max_q or max(max(n), 1), scale)
    gk.gk_sync(gkctx)
    y, lse = y.float().cpu().numpy(), lse.cpu().numpy()
    assert (y[rows:] == 3).all() and (y[:, w:] == 3).all() and (lse[rows:] == 3).all()
    return y[:rows, :w].reshape(rows, H, hs).astype(np.float64), lse[:rows].astype(np.float64)


def check_attention(y, lse, ref, what=""):
    yr, lr, spread = ref
    tol = U * (np.abs(yr) + spread) + 2.0 ** -10 * spread
    bad = ~(np.abs(y - yr) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), y[bad][:4], yr[bad][:4])
    assert np.array_equal(np.isneginf(lse), np.isneginf(lr)), what
    f = np.isfinite(lr)
    assert np.abs(lse[f] - lr[f]).max(initial=0) < 2.0 ** -10, what


ATTN = [  # kv_len, n, H, Hkv, hs, page
    ([1], [1], 1, 1, 16, 16),
    ([777], [1], 12, 12, 64, 16),
    ([0, 130, 1, 128, 129, 15, 16, 17], [1] * 8, 8, 2, 128, 16),
    ([64, 65, 700, 33], [1, 3, 0, 2], 4, 4, 80, 32),
    ([5000], [1], 3, 1, 64, 64),  # split over the GPU
    ([3, 1500], [5, 4], 8, 2, 32, 128),  # more rows than tokens
    ([200, 300], [16, 15], 2, 2, 64, 16),
    ([200, 300], [17, 16], 4, 2, 64, 16),
    ([333, 64, 400], [64, 64, 1], 1, 1, 128, 64),
    ([333, 65, 400], [65, 65, 1], 1, 1, 128, 64),
    ([300, 300, 128, 129], [129, 128, 127, 1], 2, 1, 64, 16),
    ([513, 77], [200, 77], 6, 3, 96, 32),
    ([1100, 20], [260, 20], 3, 3, 48, 256),
    ([700], [300], 8, 1, 128, 64),
    ([2600, 0, 900], [513, 3, 600], 2, 2, 64, 128),
    ([140] * 40, [2] * 40, 5, 5, 112, 16),
    ([20000, 4000], [2, 1], 16, 2, 128, 64),
    ([6000, 3000], [300, 70], 2, 1, 64, 32),
    ([5000, 700], [260, 600], 1, 1, 128, 16),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention(gkctx, case, q8):
    kv_len, n, H, Hkv, hs, page = ATTN[case]
    rng = np.random.default_rng(200 + case)
    c = cache(rng, kv_len, Hkv, hs, page, q8)
    q = serving.bf16(rng.standard_normal((sum(n), H, hs)) * 2)
    scale = 1 / math.sqrt(hs)
    y, lse = attend(gkctx, c, q, n, scale, extra_rows=case % 3, pad=8 * (case % 2))
    check_attention(y, lse, serving.paged_attn(c, q, starts(n), scale))


@pytest.mark.parametrize("n", [1, 5, 40, 150])
def test_attention_peaks_and_large_scores(gkctx, n):
    """Scores of up to about 60, so that the running maximum moves by much along the keys."""
    rng = np.random.default_rng(300 + n)
    c = cache(rng, [600, 300], 2, 64, 16, False)
    c.k *= np.exp2(rng.integers(-2, 2, c.k.shape[:1] + (1, 1, 1))).astype(np.float32)
    q = serving.bf16(rng.standard_normal((2 * n, 4, 64)) * 3)
    y, lse = attend(gkctx, c, q, [n, n], 0.125)
    check_attention(y, lse, serving.paged_attn(c, q, starts([n, n]), 0.125))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("n,H,Hkv", [(6, 2, 2), (40, 1, 1), (100, 2, 1), (200, 1, 1)])
def test_attention_unseen_infinities_and_nan(gkctx, n, H, Hkv, q8):
    """Later tokens of the chunk hold infinities and NaN: the rows before them are as without them, the rows
    that see them carry them exactly where the oracle does (a NaN or infinity there, not which of the two)."""
    rng = np.random.default_rng(400 + n)
    kv = n + 30
    c = cache(rng, [kv, 50], Hkv, 64, 16, q8)
    q = serving.bf16(rng.standard_normal((n + 1, H, 64)))
    hot = kv - n // 2  # a position of the chunk
    p, r = c.place(0, hot)
    if q8:
        c.v_scale[p, 0, r] = np.nan
    else:
        c.v[p, 0, r, 5], c.v[p, 0, r, 9] = np.inf, np.nan
    p2, r2 = c.place(0, kv - 1)
    if q8:
        c.k_scale[p2, 0, r2] = np.nan
    else:
        c.k[p2, 0, r2, 3] = np.nan
    y, lse = attend(gkctx, c, q, [n, 1], 0.125)
    yr, lr, spread = serving.paged_attn(c, q, starts([n, 1]), 0.125)
    odd = ~np.isfinite(yr)
    assert np.array_equal(odd, ~np.isfinite(y))
    assert odd.any() and not odd[: n // 2].any()
    fine = ~odd
    tol = U * (np.abs(yr) + spread) + 2.0 ** -10 * spread
    assert (np.abs(y - yr)[fine] <= tol[fine]).all()
    assert np.array_equal(np.isnan(lse), np.isnan(lr))


@pytest.mark.parametrize("n", [1, 3, 90])
def test_attention_bad_pages_and_lengths(gkctx, n):
    from gpt_decoder_gb300 import gk

    rng = np.random.default_rng(500 + n)
    c = cache(rng, [200, 100], 2, 64, 16, True)
    d = Dev(c)
    c.table[0, 3], c.table[0, 5], c.table[1, 0] = c.n_pages, -7, 1 << 30
    d.table.copy_(dev(c.table))
    q = serving.bf16(rng.standard_normal((2 * n, 2, 64)))
    with pytest.raises(gk.GkError) as e:
        attend(gkctx, c, q, [n, n], 0.125, d=d)
    assert e.value.status == gk.GK_ERR_INDEX
    t = _t()
    y = t.empty(2 * n, 128, dtype=t.bfloat16, device="cuda")
    args = (gk.GK_BF16, dev(q.reshape(2 * n, 128), t.bfloat16), 128, y, 128, None, dev(starts([n, n])), 2, 2, 2 * n)
    gk.gk_paged_attn(gkctx, d.h, *args, n, 0.125)
    t.cuda.synchronize()
    ref = serving.paged_attn(c, q, starts([n, n]), 0.125)
    tol = U * (np.abs(ref[0]) + ref[2]) + 2.0 ** -10 * ref[2]
    assert (np.abs(y.float().cpu().numpy().reshape(ref[0].shape) - ref[0]) <= tol).all()
    with pytest.raises(gk.GkError):
        gk.gk_sync(gkctx)
    if n > 1:  # more rows than max_q: refused on the device, rows left
        y.fill_(9)
        gk.gk_paged_attn(gkctx, d.h, *args, n - 1, 0.125)
        with pytest.raises(gk.GkError):
            gk.gk_sync(gkctx)
        assert (y == 9).all()
    # a length past the table: the tokens that are there are attended
    d.table.copy_(dev(np.maximum(c.table, 0) % c.n_pages))
    d.kv_len.copy_(t.tensor([1 << 29, 100], dtype=t.int32))
    gk.gk_paged_attn(gkctx, d.h, *args, n, 0.125)
    with pytest.raises(gk.GkError):
        gk.gk_sync(gkctx)


def test_attention_small_workspace_and_graph(gkctx):
    """Any workspace will do, and a captured call replays on changed inputs (the split runs either way)."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(600)
    for n, hs, q8 in ((1, 64, True), (70, 64, True), (70, 64, False), (300, 128, True), (300, 128, False)):
        c = cache(rng, [6000, 2500], 2, hs, 64, q8)
        q = serving.bf16(rng.standard_normal((2 * n, 4, hs)))
        ref = serving.paged_attn(c, q, starts([n, n]), 0.125)
        w = 4 * hs
        for ws in (0, 1 << 16, 64 << 20):
            ctx = gk.Ctx(t.cuda.current_stream().cuda_stream, workspace_bytes=ws)
            check_attention(*attend(ctx, c, q, [n, n], 0.125), ref, ws)
            ctx.close()
        s = t.cuda.Stream()
        ctx = gk.Ctx(s, workspace_bytes=64 << 20)
        d, y = Dev(c), t.zeros(2 * n, w, dtype=t.bfloat16, device="cuda")
        qd, qs = t.zeros(2 * n, w, dtype=t.bfloat16, device="cuda"), dev(starts([n, n]))
        t.cuda.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=s):
            gk.gk_paged_attn(ctx, d.h, gk.GK_BF16, qd, w, y, w, None, qs, 2, 4, 2 * n, n, 0.125)
        qd.copy_(dev(q.reshape(2 * n, w), t.bfloat16))
        for _ in range(2):
            y.zero_()
            g.replay()
            t.cuda.synchronize()
            check_attention(y.float().cpu().numpy().reshape(ref[0].shape), ref[1], ref)
        gk.gk_sync(ctx)
        ctx.close()


# --------------------------------------------------------------------------------- 4-bit products
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("transW", [0, 1])
def test_quant_w4_exact(gkctx, group, transW):
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(group + transW)
    M, K = 77, 384
    w = rng.standard_normal((M, K)).astype(np.float32)
    w[3, :group], w[4, 1], w[5, K - 1] = 0, np.inf, np.nan
    W = w if transW else np.ascontiguousarray(w.T)
    Wd = t.zeros(W.shape[0], W.shape[1] + 3, device="cuda")
    Wd[:, : W.shape[1]] = dev(W)
    q, s = t.zeros(M, K // 2, dtype=t.uint8, device="cuda"), t.zeros(M, K // group, dtype=t.bfloat16, device="cuda")
    gk.gk_quant_w4(gkctx, Wd, W.shape[1] + 3, transW, q, s, group, K, M)
    gk.gk_sync(gkctx)
    qr, sr = serving.quant_w4(w, group)
    assert np.array_equal(q.cpu().numpy(), qr) and np.array_equal(s.float().cpu().numpy(), sr, equal_nan=True)


W4 = [  # N, K, M, group
    (1, 32, 1, 32), (1, 768, 2304, 64), (3, 128, 17, 128), (8, 1600, 50, 64), (9, 4096, 1000, 128), (16, 96, 333, 32),
    (17, 768, 64, 128), (32, 2048, 255, 32), (1, 16384, 130, 128), (5, 11008, 48, 128), (2, 544, 16, 32), (31, 64, 5, 64),
    (1, 768, 50257, 64),
]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("N,K,M,group", W4)
def test_matvec_w4(gkctx, N, K, M, group, f32):
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(N * 7 + K + M)
    packed = rng.integers(0, 256, (M, K // 2), dtype=np.uint8)
    scales = serving.bf16(rng.uniform(0.5, 1.5, (M, K // group)) / math.sqrt(K))
    x = serving.bf16(rng.standard_normal((N, K)))
    bias, res = rng.standard_normal(M).astype(np.float32), rng.standard_normal((N, M)).astype(np.float32)
    extra = (N + M) % 2 == 0
    ldx, ldy, ldr = K + 8, M + 3, M + 1
    xd = t.full((N, ldx), float("nan"), dtype=t.bfloat16, device="cuda")
    xd[:, :K] = dev(x, t.bfloat16)
    rd = t.zeros(N, ldr, device="cuda")
    rd[:, :M] = dev(res)
    y = t.full((N, ldy), 3.0, dtype=t.float32 if f32 else t.bfloat16, device="cuda")
    call = lambda: gk.gk_matvec_w4(gkctx, gk.GK_BF16, xd, ldx, dev(packed), dev(scales, t.bfloat16), group,  # noqa: E731
                                   dev(bias) if extra else None, rd if extra else None, ldr, y, ldy,
                                   gk.GK_F32 if f32 else gk.GK_BF16, N, K, M)
    call()
    gk.gk_sync(gkctx)
    first = y.clone()
    w = serving.dequant_w4(packed, scales, group)
    ref = x.astype(np.float64) @ w.T + (bias + res.astype(np.float64) if extra else 0)
    size = np.abs(x).astype(np.float64) @ np.abs(w).T + (np.abs(bias) + np.abs(res) if extra else 0)
    got = y.float().cpu().numpy()
    tol = (K + 4) * 2.0 ** -24 * size + (2.0 ** -24 if f32 else U) * np.abs(ref)
    assert (np.abs(got[:, :M] - ref) <= tol).all()
    assert (got[:, M:] == 3).all()
    call()
    gk.gk_sync(gkctx)
    assert t.equal(first, y)


def test_matvec_w4_in_place_residual_and_odd_values(gkctx):
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(1)
    N, K, M, G = 4, 256, 40, 64
    packed = rng.integers(0, 256, (M, K // 2), dtype=np.uint8)
    scales = serving.bf16(rng.uniform(0.5, 1.5, (M, K // G)))
    scales[7, 2] = np.nan
    x = serving.bf16(rng.standard_normal((N, K)))
    x[2, 100] = np.inf
    x[3, :] = 0
    y0 = rng.standard_normal((N, M)).astype(np.float32)
    y = dev(y0)
    gk.gk_matvec_w4(gkctx, gk.GK_BF16, dev(x, t.bfloat16), K, dev(packed), dev(scales, t.bfloat16), G, None, y, M, y, M,
                    gk.GK_F32, N, K, M)
    gk.gk_sync(gkctx)
    got = y.cpu().numpy()
    ok = np.ones((N, M), bool)
    ok[:, 7], ok[2] = False, False
    w = serving.dequant_w4(packed, np.nan_to_num(scales), G)
    with np.errstate(all="ignore"):
        ref = x.astype(np.float64) @ w.T + y0
    assert np.isnan(got[:, 7]).all() and not np.isfinite(got[2]).any()
    assert np.abs(got - ref)[ok].max() < 1e-4 and np.array_equal(got[3][ok[3]], y0[3][ok[3]])


# ---------------------------------------------------------------------------------------- sampling
def pick(gkctx, x, u, temp=None, k=None, p=None, m=None, bf16=False, ld=None, prob=True):
    from gpt_decoder_gb300 import gk

    t = _t()
    R, V = x.shape
    ld = ld or V
    buf = t.full((R, ld), float("inf"), dtype=t.bfloat16 if bf16 else t.float32, device="cuda")
    buf[:, :V] = dev(x, buf.dtype)
    f = lambda a, dt: None if a is None else dev(np.broadcast_to(np.asarray(a, dt), (R,)).copy())  # noqa: E731
    nx, pr = t.full((R,), -5, dtype=t.int32, device="cuda"), t.full((R,), -5.0, device="cuda")
    gk.gk_sample_rows(gkctx, gk.GK_BF16 if bf16 else gk.GK_F32, buf, ld, R, V, f(u, np.float32), f(temp, np.float32),
                      f(k, np.int32), f(p, np.float32), f(m, np.float32), nx, pr if prob else None)
    gk.gk_sync(gkctx)
    return nx.cpu().numpy(), pr.cpu().numpy()


def agree(got, x, u, temp=None, k=None, p=None, m=None):
    R = x.shape[0]
    at = lambda a, r: None if a is None else np.broadcast_to(np.asarray(a), (R,))[r]  # noqa: E731
    for r in range(R):
        f = [None if a is None else np.float32(at(a, r)) for a in (temp, p, m)]
        i, pr, near = serving.sample_row(x[r], np.float32(at(u, r)), f[0], at(k, r), f[1], f[2])
        assert near > 1e-9, r
        assert got[0][r] == i, (r, got[0][r], i, near)
        assert abs(got[1][r] - pr) <= 2.0 ** -22 * max(pr, 2.0 ** -20), (r, got[1][r], pr)


@pytest.mark.parametrize("V", [1, 2, 33, 1000, 50257, 131072, 262144])
@pytest.mark.parametrize("bf16", [False, True])
def test_sampling_filters(gkctx, V, bf16):
    rng = np.random.default_rng(V + bf16)
    R = 24
    x = (rng.standard_normal((R, V)) * rng.choice([0.5, 2, 6], (R, 1))).astype(np.float32)
    x = serving.bf16(x) if bf16 else x
    u = rng.random(R).astype(np.float32)
    temp = rng.uniform(0.3, 2, R).astype(np.float32)
    k = rng.choice([0, 1, 2, 7, 40, 900, V, V + 5], R).astype(np.int32)
    p = rng.choice([0.1, 0.5, 0.9, 0.999, 1.0, 0.0], R).astype(np.float32)
    m = rng.choice([0.0, 0.003, 0.05, 0.5], R).astype(np.float32)
    for f in ({}, dict(temp=temp), dict(temp=temp, k=k), dict(p=p), dict(m=m), dict(temp=temp, k=k, p=p, m=m)):
        agree(pick(gkctx, x, u, bf16=bf16, ld=V + 7 * (V % 2), **f), x, u, **f)


def test_sampling_ties_and_extremes(gkctx):
    inf, nan = np.inf, np.nan
    V = 3000
    rng = np.random.default_rng(2)
    x = np.zeros((16, V), np.float32)
    x[1, :] = -0.0
    x[1, 5] = 0.0
    x[2, 100:200] = 2  # one hundred equal maxima
    x[3] = rng.integers(0, 3, V)  # three values, many ties
    x[4] = rng.integers(0, 3, V)
    x[5, 7] = inf
    x[6, [7, 9]] = inf
    x[7] = nan
    x[8] = -inf
    x[9], x[9, 2999] = -inf, -3.4e38
    x[10], x[10, [3, 2000]] = nan, (1.0, 2.0)
    x[11] = rng.standard_normal(V) * 1e30
    x[12] = np.exp2(-(np.arange(V) % 140.0)).astype(np.float32)  # magnitudes over the whole range of exponents
    x[13] = -np.exp2(np.arange(V) % 120).astype(np.float32)
    x[14] = rng.standard_normal(V) * 1e-30
    x[15] = rng.standard_normal(V)
    u = (0.317 + 0.041 * np.arange(16)).astype(np.float32)
    u = np.where(u >= 1, 0.123, u).astype(np.float32)
    for f in ({}, dict(k=50), dict(p=0.777), dict(m=0.3), dict(k=50, p=0.613, m=0.01), dict(temp=1e-30, k=3), dict(temp=np.inf, p=0.4321)):
        agree(pick(gkctx, x, u, **f), x, u, **f)
    got = pick(gkctx, x, u, temp=0.0, k=5)
    assert got[0].tolist()[:7] == [0, 0, 100, int(x[3].argmax()), int(x[4].argmax()), 7, 7] and got[0][7] == -1
    assert (got[1][[0, 2, 5]] == 1).all() and got[1][7] == 0 and got[1][8] == 0
    # uniform numbers outside [0, 1): the first, and the last kept, index
    one = pick(gkctx, x[15:], np.array([1.0], np.float32), k=10)
    kept = np.flatnonzero(x[15] >= np.sort(x[15])[-10])
    assert one[0][0] == kept[-1] and pick(gkctx, x[15:], np.array([nan], np.float32), k=10)[0][0] == kept[-1]
    assert pick(gkctx, x[15:], np.array([-1.0], np.float32), k=10)[0][0] == kept[0]
    assert pick(gkctx, x[15:], np.array([0.0], np.float32), k=10, prob=False)[0][0] == kept[0]


def test_sampling_many_rows_and_repeat(gkctx):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((700, 257)) * 2).astype(np.float32)
    u = rng.random(700).astype(np.float32)
    a = pick(gkctx, x, u, temp=0.8, k=40, p=0.9)
    agree(a, x, u, temp=0.8, k=40, p=0.9)
    b = pick(gkctx, x, u, temp=0.8, k=40, p=0.9)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


# ------------------------------------------------------------------------------- a run of them together
def test_serving_step_of_a_block(gkctx):
    """Two decode steps of one attention block as a served model runs them: 4-bit q, k, v projection, the cache
    write, attention, 4-bit output projection with the residual, a 4-bit head, filtered sampling, against the same
    chain in float64 with the device's roundings of the tensors in between."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(11)
    H, Hkv, hs, V, page, B, G = 4, 2, 64, 500, 16, 3, 64
    C, W = H * hs, (H + 2 * Hkv) * hs

    def quantised(K, M):
        w = (rng.standard_normal((K, M)) / math.sqrt(K)).astype(np.float32)
        q, s = t.zeros(M, K // 2, dtype=t.uint8, device="cuda"), t.zeros(M, K // G, dtype=t.bfloat16, device="cuda")
        gk.gk_quant_w4(gkctx, dev(w), M, 0, q, s, G, K, M)
        return q, s, serving.dequant_w4(*serving.quant_w4(np.ascontiguousarray(w.T), G), G)

    wqkv, wo, wv = quantised(C, W), quantised(C, C), quantised(C, V)
    lens = np.array([30, 0, 47], np.int32)
    c = cache(rng, [64, 16, 64], Hkv, hs, page, True)
    c.kv_len = lens.copy()
    d = Dev(c, poison=False)
    d.kv_len.copy_(dev(lens))
    for step in range(2):
        n = [5, 3, 1] if step == 0 else [1, 1, 1]
        rows, qs = sum(n), starts(n)
        c.kv_len += np.array(n, np.int32)
        d.kv_len.copy_(dev(c.kv_len))
        x = serving.bf16(rng.standard_normal((rows, C)))
        xr = rng.standard_normal((rows, C)).astype(np.float32)
        xd, res, qkv = dev(x, t.bfloat16), dev(xr), t.empty(rows, W, dtype=t.bfloat16, device="cuda")
        y, h, logits = (t.empty(rows, C, dtype=t.bfloat16, device="cuda"), t.empty(rows, C, dtype=t.bfloat16, device="cuda"),
                        t.empty(rows, V, device="cuda"))
        u, nx = dev(rng.random(rows).astype(np.float32)), t.empty(rows, dtype=t.int32, device="cuda")
        qsd = dev(qs)
        gk.gk_matvec_w4(gkctx, gk.GK_BF16, xd, C, wqkv[0], wqkv[1], G, None, None, 0, qkv, W, gk.GK_BF16, rows, C, W)
        gk.gk_paged_write(gkctx, d.h, gk.GK_BF16, qkv[:, C:], W, qkv[:, C + Hkv * hs :], W, qsd, B, rows)
        gk.gk_paged_attn(gkctx, d.h, gk.GK_BF16, qkv, W, y, C, None, qsd, B, H, rows, max(n), 0.125)
        gk.gk_matvec_w4(gkctx, gk.GK_BF16, y, C, wo[0], wo[1], G, None, res, C, res, C, gk.GK_F32, rows, C, C)
        gk.gk_to_bf16(gkctx, res, h, rows * C)
        gk.gk_matvec_w4(gkctx, gk.GK_BF16, h, C, wv[0], wv[1], G, None, None, 0, logits, V, gk.GK_F32, rows, C, V)
        gk.gk_sample_rows(gkctx, gk.GK_F32, logits, V, rows, V, u, None, None, dev(np.full(rows, 0.9, np.float32)), None, nx)
        gk.gk_sync(gkctx)
        got = {k: a.float().cpu().numpy().astype(np.float64) for k, a in dict(qkv=qkv, y=y, res=res, h=h, logits=logits).items()}

        def close(a, b, size, bits, K):
            assert (np.abs(a - b) <= bits * np.abs(b) + (K + 4) * 2.0 ** -24 * size).all()

        close(got["qkv"], x @ wqkv[2].T, np.abs(x) @ np.abs(wqkv[2]).T, U, C)
        q3 = got["qkv"].reshape(rows, -1, hs)
        serving.paged_write(c, q3[:, H : H + Hkv].astype(np.float32), q3[:, H + Hkv :].astype(np.float32), qs)
        assert np.array_equal(d.k.cpu().numpy(), c.k) and np.array_equal(d.vs.cpu().numpy(), c.v_scale)
        ref = serving.paged_attn(c, q3[:, :H].astype(np.float32), qs, 0.125)
        check_attention(got["y"].reshape(rows, H, hs), ref[1], ref)
        close(got["res"], got["y"] @ wo[2].T + xr, np.abs(got["y"]) @ np.abs(wo[2]).T + np.abs(xr), 2.0 ** -24, C)
        close(got["logits"], got["h"] @ wv[2].T, np.abs(got["h"]) @ np.abs(wv[2]).T, 2.0 ** -24, C)
        for r in range(rows):
            assert nx[r].item() == serving.sample_row(got["logits"][r], u[r].item(), None, None, np.float32(0.9))[0]


# ---------------------------------------------------------------------------------------- refusals
def refused(status, fn, *args):
    from gpt_decoder_gb300 import gk

    with pytest.raises(gk.GkError) as e:
        fn(*args)
    assert e.value.status == status, e.value


def test_paged_calls_refuse(gkctx):
    from gpt_decoder_gb300 import gk

    t = _t()
    c = cache(np.random.default_rng(1), [20], 2, 32, 16, True)
    d = Dev(c)
    x, y, qs = t.zeros(4, 64, device="cuda"), t.zeros(4, 64, dtype=t.bfloat16, device="cuda"), dev(starts([4]))
    A, L, UN = gk.GK_ERR_ARG, gk.GK_ERR_ALIGN, gk.GK_ERR_UNSUPPORTED
    for fn in (gk.gk_paged_write, gk.gk_paged_read):
        refused(A, fn, gkctx, d.h, gk.GK_BF16X2, x, 64, x, 64, qs, 1, 4)
        refused(A, fn, gkctx, d.h, gk.GK_F32, None, 64, x, 64, qs, 1, 4)
        refused(A, fn, gkctx, d.h, gk.GK_F32, x, 56, x, 64, qs, 1, 4)
        refused(A, fn, gkctx, d.h, gk.GK_F32, x, 64, x, 64, None, 1, 4)
        refused(A, fn, gkctx, d.h, gk.GK_F32, x, 64, x, 64, qs, 0, 4)
        refused(A, fn, gkctx, d.h, gk.GK_F32, x, 64, x, 64, qs, 1, -1)
        refused(L, fn, gkctx, d.h, gk.GK_F32, x, 68, x, 64, qs, 1, 4)
        refused(L, fn, gkctx, d.h, gk.GK_F32, x.data_ptr() + 4, 64, x, 64, qs, 1, 4)
        fn(gkctx, d.h, gk.GK_F32, x, 64, x, 64, qs, 1, 0)
    att = lambda dt=gk.GK_BF16, q=y, ldq=64, o=y, H=2, mq=4, s=1.0: (gkctx, d.h, dt, q, ldq, o, 64, None, qs, 1, H, 4, mq, s)  # noqa: E731
    refused(UN, gk.gk_paged_attn, *att(dt=gk.GK_F32))
    refused(A, gk.gk_paged_attn, *att(q=None))
    refused(A, gk.gk_paged_attn, *att(H=3))
    refused(A, gk.gk_paged_attn, *att(H=0))
    refused(A, gk.gk_paged_attn, *att(H=4))  # rows of 4 heads do not fit the stride
    refused(A, gk.gk_paged_attn, *att(mq=0))
    refused(A, gk.gk_paged_attn, *att(s=float("nan")))
    refused(A, gk.gk_paged_attn, *att(s=0.0))
    refused(A, gk.gk_paged_attn, *att(s=float("inf")))
    refused(L, gk.gk_paged_attn, *att(ldq=68))
    refused(L, gk.gk_paged_attn, *att(o=y.data_ptr() + 2))
    s = d.h.struct
    for name, bad, status in (("page_size", 24, UN), ("page_size", 512, UN), ("page_size", 8, UN), ("hs", 24, UN), ("hs", 144, UN),
                              ("dtype", gk.GK_F32, A), ("k_scale", None, A), ("n_pages", 0, A), ("max_pages", 0, A),
                              ("ld_table", 1, A), ("k", s.k + 2, L), ("kv_len", None, A), ("max_pages", 1 << 27, A)):
        old = getattr(s, name)
        setattr(s, name, bad)
        refused(status, gk.gk_paged_read, gkctx, d.h, gk.GK_F32, x, 1024, x, 1024, qs, 1, 4)
        refused(status, gk.gk_paged_attn, gkctx, d.h, gk.GK_BF16, y, 1024, y, 1024, None, qs, 1, 2, 4, 4, 1.0)
        setattr(s, name, old)
    gk.gk_sync(gkctx)


def test_w4_and_sampling_refuse(gkctx):
    from gpt_decoder_gb300 import gk

    t = _t()
    A, L, UN = gk.GK_ERR_ARG, gk.GK_ERR_ALIGN, gk.GK_ERR_UNSUPPORTED
    x, w, s = t.zeros(40, 64, dtype=t.bfloat16, device="cuda"), t.zeros(8, 32, dtype=t.uint8, device="cuda"), t.zeros(8, 2, dtype=t.bfloat16, device="cuda")
    y = t.zeros(40, 8, device="cuda")
    mv = lambda dt=gk.GK_BF16, x=x, ldx=64, w=w, g=32, res=None, ldr=8, ldy=8, yd=gk.GK_F32, N=2, K=64: (  # noqa: E731
        gkctx, dt, x, ldx, w, s, g, None, res, ldr, y, ldy, yd, N, K, 8)
    for bad, status in ((dict(dt=gk.GK_F32), UN), (dict(x=None), A), (dict(ldx=56), A), (dict(g=16), UN), (dict(g=128), A),
                        (dict(N=33), UN), (dict(N=-1), A), (dict(yd=gk.GK_BF16X2), A), (dict(ldy=7), A), (dict(ldx=68), L),
                        (dict(w=w.data_ptr() + 1), L), (dict(x=x.data_ptr() + 2), L), (dict(res=y, ldr=9), A),
                        (dict(res=y, yd=gk.GK_BF16), A), (dict(res=x, ldr=7), A), (dict(K=0), A)):
        refused(status, gk.gk_matvec_w4, *mv(**bad))
    gk.gk_matvec_w4(*mv(N=0))
    refused(A, gk.gk_quant_w4, gkctx, y, 7, 0, w, s, 32, 64, 8)
    refused(A, gk.gk_quant_w4, gkctx, None, 8, 0, w, s, 32, 64, 8)
    refused(UN, gk.gk_quant_w4, gkctx, y, 8, 0, w, s, 48, 96, 8)
    n, u = t.zeros(4, dtype=t.int32, device="cuda"), t.zeros(4, device="cuda")
    sr = lambda dt=gk.GK_F32, x=y, ld=8, V=8, u=u, n=n, rows=4: (gkctx, dt, x, ld, rows, V, u, None, None, None, None, n)  # noqa: E731
    for bad, status in ((dict(dt=gk.GK_I8), A), (dict(x=None), A), (dict(ld=7), A), (dict(V=0), A), (dict(u=None), A), (dict(n=None), A),
                        (dict(rows=-1), A), (dict(V=(1 << 18) + 1, ld=1 << 20), UN)):
        refused(status, gk.gk_sample_rows, *sr(**bad))
    gk.gk_sample_rows(*sr(rows=0))
    gk.gk_sync(gkctx)


def test_serving_calls_refuse_sizes_past_their_indices(gkctx):
    from gpt_decoder_gb300 import gk

    t = _t()
    c = cache(np.random.default_rng(2), [20], 2, 32, 16, False)
    d, y, qs = Dev(c), t.zeros(4, 128, dtype=t.bfloat16, device="cuda"), dev(starts([4]))
    refused(gk.GK_ERR_UNSUPPORTED, gk.gk_paged_attn, gkctx, d.h, gk.GK_BF16, y, 128, y, 128, None, qs, 1, 4, 1 << 30, 1 << 30, 1.0)
    w, s = t.zeros(8, 32, dtype=t.uint8, device="cuda"), t.zeros(8, 2, dtype=t.bfloat16, device="cuda")
    M = 1 << 30
    refused(gk.GK_ERR_UNSUPPORTED, gk.gk_matvec_w4, gkctx, gk.GK_BF16, y, 128, w, s, 32, None, None, 0, y, M, gk.GK_F32, 2, 64, M)
    gk.gk_sync(gkctx)


@pytest.mark.parametrize("n", [1, 40, 200])
def test_attention_of_sequences_that_share_pages(gkctx, n):
    """A common prefix kept once: two tables name the same pages (nothing is written meanwhile)."""
    rng = np.random.default_rng(700 + n)
    for q8 in (False, True):
        c = cache(rng, [1000, 1000, 700], 2, 64, 32, q8)
        c.table[1, :20] = c.table[0, :20]
        c.table[2, :c.table.shape[1]] = c.table[0]
        q = serving.bf16(rng.standard_normal((3 * n, 4, 64)))
        ref = serving.paged_attn(c, q, starts([n] * 3), 0.125)
        check_attention(*attend(gkctx, c, q, [n] * 3, 0.125), ref, (n, q8))


@pytest.mark.parametrize("q8", [False, True])
def test_cache_offsets_past_32_bits(gkctx, q8):
    """Pages whose first element lies past 2^32 elements of the cache: write, read back and attention."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(800)
    Hkv, hs, page, n_pages = 8, 128, 128, 33000
    assert (n_pages - 200) * Hkv * hs * page > 1 << 32
    c = cache(rng, [1500, 333], Hkv, hs, page, q8)
    d = Dev(c)

    def big(x):  # the last pages are the small cache's
        if x is None:
            return None
        y = t.empty(n_pages, *x.shape[1:], dtype=x.dtype, device="cuda")
        y[n_pages - c.n_pages:].copy_(x)
        return y

    k, v, ks, vs = (big(x) for x in (d.k, d.v, d.ks, d.vs))
    h = gk.PagedKv(k, v, ks, vs, d.table + (n_pages - c.n_pages), d.kv_len)
    w = Hkv * hs
    for n in (1, 300):
        q = serving.bf16(rng.standard_normal((2 * n, Hkv, hs)))
        ref = serving.paged_attn(c, q, starts([n, n]), 0.088)
        y = t.zeros(2 * n, w, dtype=t.bfloat16, device="cuda")
        lse = t.zeros(2 * n, Hkv, device="cuda")
        qd, qs = dev(q.reshape(2 * n, w), t.bfloat16), dev(starts([n, n]))
        gk.gk_paged_attn(gkctx, h, gk.GK_BF16, qd, w, y, w, lse, qs, 2, Hkv, 2 * n, n, 0.088)
        gk.gk_sync(gkctx)
        check_attention(y.float().cpu().numpy().reshape(ref[0].shape), lse.cpu().numpy(), ref, n)
    # write and read at the same places as in the small cache: the same bits
    new = t.from_numpy(rng.standard_normal((2, 200, w)).astype(np.float32)).cuda()
    qs = dev(starts([100, 100]))
    out = []
    for cache_h in (h, d.h):
        gk.gk_paged_write(gkctx, cache_h, gk.GK_F32, new[0], w, new[1], w, qs, 2, 200)
        o = t.zeros(2, 200, w, device="cuda")
        gk.gk_paged_read(gkctx, cache_h, gk.GK_F32, o[0], w, o[1], w, qs, 2, 200)
        gk.gk_sync(gkctx)
        out.append(o)
    assert t.equal(out[0], out[1])
    assert float((out[0] - new).abs().max()) < 0.05  # half a step of values below 6, or bf16's rounding of them


def test_two_contexts_at_once(gkctx):
    """Calls of two contexts on two streams run together, each with a workspace of its own: the bits of one alone."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(900)
    jobs = []
    for n, hs, q8 in ((300, 128, True), (260, 64, False), (1, 64, True), (1, 128, False)):
        c = cache(rng, [3000, 900], 2, hs, 64, q8)
        q = dev(rng.standard_normal((2 * n, 8 * hs)), t.bfloat16)
        jobs.append((Dev(c), q, dev(starts([n, n])), n, 8 * hs))
    W = dev(rng.standard_normal((512, 1000)).astype(np.float32))
    wq, sc = t.zeros(1000, 256, dtype=t.uint8, device="cuda"), t.zeros(1000, 16, dtype=t.bfloat16, device="cuda")
    gk.gk_quant_w4(gkctx, W, 1000, 0, wq, sc, 32, 512, 1000)
    x, u = dev(rng.standard_normal((5, 512)), t.bfloat16), dev(rng.random(5).astype(np.float32))
    p = dev(np.full(5, 0.9, np.float32))
    gk.gk_sync(gkctx)

    def outputs():
        return [t.zeros(q.shape, dtype=t.bfloat16, device="cuda") for _, q, _, _, _ in jobs] + [
            t.zeros(5, 1000, device="cuda"), t.zeros(5, dtype=t.int32, device="cuda")]

    def run(ctx, out):
        for (d, q, qs, n, w), y in zip(jobs, out):
            gk.gk_paged_attn(ctx, d.h, gk.GK_BF16, q, w, y, w, None, qs, 2, 8, 2 * n, n, 0.1)
        gk.gk_matvec_w4(ctx, gk.GK_BF16, x, 512, wq, sc, 32, None, None, 0, out[-2], 1000, gk.GK_F32, 5, 512, 1000)
        gk.gk_sample_rows(ctx, gk.GK_F32, out[-2], 1000, 5, 1000, u, None, None, p, None, out[-1])

    want = outputs()
    t.cuda.synchronize()
    run(gkctx, want)
    gk.gk_sync(gkctx)
    ctxs = [gk.Ctx(t.cuda.Stream(), workspace_bytes=64 << 20) for _ in range(2)]
    got = [[outputs() for _ in range(10)] for _ in ctxs]
    t.cuda.synchronize()
    for i in range(10):
        for ctx, o in zip(ctxs, got):
            run(ctx, o[i])
    for ctx in ctxs:
        gk.gk_sync(ctx)
        ctx.close()
    for o in got:
        for each in o:
            for a, b in zip(each, want):
                assert t.equal(a, b)


@pytest.mark.parametrize("n, hs, ws", [(1100, 64, 2 << 20), (600, 128, 4 << 20)])
def test_attention_of_8_bit_chunks_a_few_heads_at_a_time(gkctx, n, hs, ws):
    """A workspace with room for the codes of two of five heads as bf16: three turns, the last of one head."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(1000 + hs)
    Hkv, G, kv = 5, 8, [1300, 1200]
    c = cache(rng, kv, Hkv, hs, 64, True)
    a_head = 2 * 2 * 1408 * hs * 2  # keys and values, two sequences in whole tiles of 128
    assert 2 * a_head <= ws * 3 // 4 < 3 * a_head and 2 * 2 * 2 * -(-n * G // 256) >= 152
    q = serving.bf16(rng.standard_normal((2 * n, Hkv * G, hs)))
    ref = serving.paged_attn(c, q, starts([n, n]), 0.1)
    ctx = gk.Ctx(t.cuda.current_stream().cuda_stream, workspace_bytes=ws)
    check_attention(*attend(ctx, c, q, [n, n], 0.1), ref, hs)
    ctx.close()


@pytest.mark.parametrize("n, hs, q8", [(1, 64, False), (1, 128, True), (6, 48, True), (9, 128, False)])
def test_attention_of_few_short_sequences_captured(gkctx, n, hs, q8):
    """Pieces joined inside a cluster: no workspace, sequences of one piece and of several, a padding row, replays on
    lengths that change between them."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(1100 + n)
    c = cache(rng, [1000, 40, 129, 0], 2, hs, 16, q8)
    q = serving.bf16(rng.standard_normal((4 * n, 6, hs)))
    w, qs = 6 * hs, dev(starts([n] * 4))
    s = t.cuda.Stream()
    ctx = gk.Ctx(s, workspace_bytes=0)
    d, qd = Dev(c, poison=False), dev(q.reshape(4 * n, w), t.bfloat16)
    y, lse = t.zeros(4 * n, w, dtype=t.bfloat16, device="cuda"), t.zeros(4 * n, 6, device="cuda")
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=s):
        gk.gk_paged_attn(ctx, d.h, gk.GK_BF16, qd, w, y, w, lse, qs, 4, 6, 4 * n, n, 0.2)
    for lens in ([1000, 40, 129, 0], [777, 12, 128, 0], [129, 1, 0, 0], [1000, 40, 129, 0]):
        c.kv_len[:] = lens
        d.kv_len.copy_(dev(c.kv_len))
        y.fill_(7.0)
        g.replay()
        t.cuda.synchronize()
        ref = serving.paged_attn(c, q, starts([n] * 4), 0.2)
        check_attention(y.float().cpu().numpy().reshape(ref[0].shape), lse.cpu().numpy(), ref, (lens, n))
    gk.gk_sync(ctx)
    ctx.close()


# ------------------------------------------------------- what is not finite where it is seen, and scores far apart
def attend_odd(gkctx, c, q, n, scale, refused=False):
    """Attention with infinities or NaN among what rows see: they are in the result exactly where the oracle has
    them (a NaN or an infinity, not which of the two), and the rest is within the bounds above."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rows, H, hs = q.shape
    w, d = H * hs, Dev(c)
    y, lse = t.full((rows, w), 3.0, dtype=t.bfloat16, device="cuda"), t.full((rows, H), 3.0, device="cuda")
    gk.gk_paged_attn(gkctx, d.h, gk.GK_BF16, dev(q.reshape(rows, w), t.bfloat16), w, y, w, lse, dev(starts(n)), len(n), H, rows, max(n), scale)
    if refused:
        with pytest.raises(gk.GkError) as e:
            gk.gk_sync(gkctx)
        assert e.value.status == gk.GK_ERR_INDEX
    else:
        gk.gk_sync(gkctx)
    y, lse = y.float().cpu().numpy().reshape(q.shape).astype(np.float64), lse.cpu().numpy()
    yr, lr, spread = serving.paged_attn(c, q, starts(n), scale)
    odd = ~np.isfinite(yr)
    assert odd.any() and not odd.all()
    assert np.array_equal(odd, ~np.isfinite(y)), np.argwhere(odd != ~np.isfinite(y))[:4].tolist()
    # a weight below float32's smallest normal number, 2^-126, is zero on the device: each of up to 2^14 keys is off by at
    # most that times its value (below 2^3 here), which shows where the weights above it meet values of zero
    tol = U * (np.abs(yr) + spread) + 2.0 ** -10 * spread + 2.0 ** (14 - 126 + 3)
    assert (np.abs(y[~odd] - yr[~odd]) <= tol[~odd]).all()
    assert np.abs(lse - lr).max() < 2.0 ** -10 * max(1.0, np.abs(lr).max() / 64)


def make_odd(c, b, pos):
    """Infinities and a NaN in the value at a position: of the first and the last head (8 bits: the head's scale)."""
    p, r = c.place(b, pos)
    if c.v_scale is not None:
        c.v_scale[p, 0, r] = np.nan
    else:
        c.v[p, 0, r, 5], c.v[p, 0, r, 9], c.v[p, -1, r, 0] = np.inf, np.nan, -np.inf


SEEN_FEW = [  # kv_len, new tokens, H, Hkv, hs, page; sequence b's value this far before its last token is not finite (and the last sequence's all are)
    (777, 1, 2, 2, 64, 16, [0, 3, 8, 9, 700]),  # the last tile of 16 keys begins 8 before the last of 777
    (130, 1, 4, 1, 128, 64, [0, 1, 2, 100]),
    (144, 1, 4, 2, 80, 16, [0, 15, 16]),
    (5000, 1, 2, 2, 64, 16, [0, 7, 8, 4900]),  # in pieces
    (130, 5, 2, 2, 48, 32, [0, 3, 4, 5, 17, 18, 90]),  # the first of the new tokens is 4 before the last
    (128, 3, 4, 2, 64, 16, [0, 2, 3, 15, 16]),  # 16 rows of a key / value head: see also the next
    (1000, 8, 4, 2, 64, 16, [0, 7, 8, 9, 23, 24]),
    (300, 16, 2, 1, 128, 16, [0, 15, 16, 27, 28]),  # and 32
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("case", range(len(SEEN_FEW)))
def test_attention_seen_infinities_and_nan_few_rows(gkctx, case, q8):
    kv, n, H, Hkv, hs, page, backs = SEEN_FEW[case]
    rng = np.random.default_rng(1200 + case)
    c = cache(rng, [kv] * (len(backs) + 1), Hkv, hs, page, q8)
    for b, back in enumerate(backs):
        make_odd(c, b, kv - 1 - back)
    q = serving.bf16(rng.standard_normal((n * (len(backs) + 1), H, hs)))
    attend_odd(gkctx, c, q, [n] * (len(backs) + 1), 0.125)


def test_attention_seen_infinities_few_rows_of_refused_pages(gkctx):
    """Values that are not finite on both sides of a refused page, and in the last tile behind one."""
    rng = np.random.default_rng(1300)
    c = cache(rng, [203] * 3, 2, 64, 16, False)
    for b, pos in enumerate((150, 176, 202)):
        make_odd(c, b, pos)
    c.table[0, 10], c.table[1, 10], c.table[2, 11] = -1, c.n_pages, -5
    for n in (1, 5):
        attend_odd(gkctx, c, serving.bf16(rng.standard_normal((3 * n, 4, 64))), [n] * 3, 0.125, refused=True)


SEEN_TILES = [  # as SEEN_FEW
    (300, 40, 1, 1, 64, 16, [0, 39, 40, 43, 44, 200]),  # the first new token is at 260, its tile of 128 keys at 256
    (777, 100, 2, 1, 128, 64, [0, 99, 100, 136, 137, 500]),  # 200 rows
    (500, 200, 2, 1, 64, 32, [0, 199, 200, 243, 244, 71, 72]),  # 400 rows: two blocks, the second's first token 72 before the last
    (6000, 70, 1, 1, 80, 128, [0, 69, 70, 111, 112, 5000]),  # in pieces
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("case", range(len(SEEN_TILES)))
def test_attention_seen_infinities_and_nan_tiles(gkctx, case, q8):
    kv, n, H, Hkv, hs, page, backs = SEEN_TILES[case]
    rng = np.random.default_rng(1400 + case)
    c = cache(rng, [kv] * (len(backs) + 1), Hkv, hs, page, q8)
    for b, back in enumerate(backs):
        make_odd(c, b, kv - 1 - back)
    q = serving.bf16(rng.standard_normal((n * (len(backs) + 1), H, hs)))
    attend_odd(gkctx, c, q, [n] * (len(backs) + 1), 0.125)


@pytest.mark.parametrize("hs", [64, 128])
def test_attention_seen_infinities_in_tiles_of_refused_pages(gkctx, hs):
    """A refused page in a tile of keys that every row sees: its neighbours' infinities and NaN stay."""
    rng = np.random.default_rng(1500 + hs)
    c = cache(rng, [700] * 4, 1, hs, 16, False)
    for b, pos in enumerate((150, 180, 120)):
        make_odd(c, b, pos)
    c.table[:3, 10] = -1, c.n_pages, -5  # positions 160 .. 175
    attend_odd(gkctx, c, serving.bf16(rng.standard_normal((4 * 70, 1, hs))), [70] * 4, 0.125, refused=True)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kv,n,high", [(100, 1, 20), (1000, 1, 500), (9000, 1, 5000), (9000, 33, 5000), (9000, 70, 5000)])
def test_attention_seen_infinities_behind_far_larger_scores(gkctx, kv, n, high, q8):
    """The weight of a value that is not finite may lie below float32's smallest, in another warp's keys or another
    piece than the row's largest score: the result is not finite all the same. (Scores are exact here: q has one
    element of 1, and keys hold 508 there or nothing; exp(-508) is above float64's smallest.)"""
    rng = np.random.default_rng(1600 + n)
    c = cache(rng, [kv, kv], 2, 64, 16, q8)
    c.k[:] = 0
    for b in range(2):
        p, r = c.place(b, high)
        c.k[p, :, r, 0] = 127 if q8 else 508
    if q8:
        c.k_scale[:] = 4
    make_odd(c, 0, 3)
    q = np.zeros((2 * n, 2, 64), np.float32)
    q[:, :, 0] = 1
    attend_odd(gkctx, c, q, [n, n], 1.0)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kv,n,high", [(100, 1, 20), (1000, 1, 500), (9000, 1, 5000), (9000, 33, 5000), (9000, 70, 5000)])
def test_attention_of_a_nan_key_behind_far_larger_scores(gkctx, kv, n, high, q8):
    """The same of a key: its score is NaN, and so are the results and log sums of every row that sees it."""
    rng = np.random.default_rng(1650 + n)
    c = cache(rng, [kv, kv], 2, 64, 16, q8)
    c.k[:] = 0
    for b in range(2):
        p, r = c.place(b, high)
        c.k[p, :, r, 0] = 127 if q8 else 508
    p, r = c.place(0, 3)
    if q8:
        c.k_scale[:] = 4
        c.k_scale[p, 0, r] = np.nan
    else:
        c.k[p, 0, r, 7] = np.nan
    q = np.zeros((2 * n, 2, 64), np.float32)
    q[:, :, 0] = 1
    y, lse = attend(gkctx, c, q, [n, n], 1.0)
    assert np.isnan(y[:n, 0]).all() and np.isnan(lse[:n, 0]).all()
    ref = serving.paged_attn(c, q, starts([n, n]), 1.0)
    fine = ~np.isnan(ref[0])
    assert not fine[:n, 0].any() and fine[:n, 1].all() and fine[n:].all()
    tol = U * (np.abs(ref[0]) + ref[2]) + 2.0 ** -10 * ref[2] + 2.0 ** (14 - 126 + 3)  # (as in attend_odd)
    assert (np.abs(y - ref[0])[fine] <= tol[fine]).all()
    assert np.abs(lse - ref[1])[np.isfinite(ref[1])].max() < 508 / 64 * 2.0 ** -10


def test_attention_scale_past_its_unit_is_refused(gkctx):
    """Scores are kept in powers of two: scale * log2(e) has to be a finite float32 too."""
    from gpt_decoder_gb300 import gk

    t = _t()
    c = cache(np.random.default_rng(3), [20], 2, 32, 16, False)
    d, q, qs = Dev(c), t.zeros(4, 64, dtype=t.bfloat16, device="cuda"), dev(starts([4]))
    y = t.full((4, 64), 3.0, dtype=t.bfloat16, device="cuda")
    refused(gk.GK_ERR_ARG, gk.gk_paged_attn, gkctx, d.h, gk.GK_BF16, q, 64, y, 64, None, qs, 1, 2, 4, 4, 3e38)
    gk.gk_sync(gkctx)
    assert (y == 3).all()
    gk.gk_paged_attn(gkctx, d.h, gk.GK_BF16, q, 64, y, 64, None, qs, 1, 2, 4, 4, 2.0 ** 127)  # scores of zero: plain means
    gk.gk_sync(gkctx)
    ref = serving.paged_attn(c, np.zeros((4, 2, 32)), starts([4]), 1.0)
    yr, spread = ref[0].reshape(4, 64), ref[2].reshape(4, 64)
    assert (np.abs(y.float().cpu().numpy() - yr) <= U * (np.abs(yr) + spread) + 2.0 ** -10 * spread).all()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("n,H", [(1, 2), (10, 2), (40, 4), (200, 2)])
def test_attention_of_lengths_past_the_table(gkctx, n, H, q8):
    """Rows at positions that the table has no room for: reported, and every token that is there is attended."""
    from gpt_decoder_gb300 import gk

    t = _t()
    rng = np.random.default_rng(1700 + n)
    c = cache(rng, [320, 100], 2, 64, 16, q8)
    d = Dev(c)
    c.kv_len[0] = 325
    d.kv_len.copy_(dev(c.kv_len))
    q = serving.bf16(rng.standard_normal((2 * n, H, 64)))
    w, ref = H * 64, serving.paged_attn(c, q, starts([n, n]), 0.125)
    y, lse = t.full((2 * n, w), 9.0, dtype=t.bfloat16, device="cuda"), t.full((2 * n, H), 9.0, device="cuda")
    gk.gk_paged_attn(gkctx, d.h, gk.GK_BF16, dev(q.reshape(2 * n, w), t.bfloat16), w, y, w, lse, dev(starts([n, n])), 2, H, 2 * n, n, 0.125)
    with pytest.raises(gk.GkError) as e:
        gk.gk_sync(gkctx)
    assert e.value.status == gk.GK_ERR_INDEX
    check_attention(y.float().cpu().numpy().reshape(q.shape), lse.cpu().numpy(), ref)
