"""Pins of the serving oracle: attention against torch in float64, the quantisers against their error
bounds and by hand, the sampler against frequencies and hand cases, and what the binding refuses."""
import numpy as np
import pytest

from oracle import sampling, serving


def cache(rng, kv_len, Hkv, hs, page, q8, spare=2):
    need = [max(0, -(-int(n) // page)) for n in kv_len]
    n_pages = sum(need) + spare
    width = max(1, max(need))
    ids = rng.permutation(n_pages)[: sum(need)]
    table = np.full((len(kv_len), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at : at + n]
        at += n
    shape = (n_pages, Hkv, page, hs)
    k, v = (rng.standard_normal(shape).astype(np.float32) for _ in range(2))
    if q8:
        (kc, ks), (vc, vs) = serving.quantise(k), serving.quantise(v)
        return serving.Pages(kc, vc, ks, vs, table, np.asarray(kv_len, np.int32))
    return serving.Pages(serving.bf16(k), serving.bf16(v), None, None, table, np.asarray(kv_len, np.int32))


@pytest.mark.parametrize("q8", [False, True])
def test_attention_matches_torch(q8):
    import torch

    rng = np.random.default_rng(3)
    kv_len, n, H, Hkv, hs = [37, 16, 5], [4, 16, 1], 4, 2, 16
    c = cache(rng, kv_len, Hkv, hs, 16, q8)
    q_start = np.concatenate([[0], np.cumsum(n)])
    q = serving.bf16(rng.standard_normal((sum(n), H, hs)))
    y, lse, spread = serving.paged_attn(c, q, q_start, 0.3)
    every = np.concatenate([[0], np.cumsum(kv_len)])  # every whole sequence read back
    k, v = serving.paged_read(c, every, every[-1]).astype(np.float64)
    for b in range(3):
        kb, vb = (torch.tensor(a[every[b] : every[b + 1]]).repeat_interleave(H // Hkv, 1).permute(1, 0, 2) for a in (k, v))
        qb = torch.tensor(q[q_start[b] : q_start[b + 1]].astype(np.float64)).permute(1, 0, 2)
        mask = torch.ones(n[b], kv_len[b], dtype=torch.bool).tril(kv_len[b] - n[b])
        ref = torch.nn.functional.scaled_dot_product_attention(qb, kb, vb, attn_mask=mask, scale=0.3)
        got = y[q_start[b] : q_start[b + 1]]
        assert np.abs(got - ref.permute(1, 0, 2).numpy()).max() < 1e-12
        z = (qb @ kb.transpose(1, 2) * 0.3).masked_fill(~mask, -np.inf).logsumexp(-1)
        assert np.abs(lse[q_start[b] : q_start[b + 1]] - z.T.numpy()).max() < 1e-12
    assert (spread >= np.abs(y) - 1e-12).all()


def test_padding_rows_see_nothing():
    rng = np.random.default_rng(4)
    c = cache(rng, [2, 0], 1, 16, 16, False)
    y, lse, _ = serving.paged_attn(c, np.ones((5, 1, 16)), [0, 4, 5], 1.0)
    assert (y[[0, 1, 4]] == 0).all() and (lse[[0, 1, 4]] == -np.inf).all() and np.isfinite(lse[2:4]).all()


def test_quantiser_bounds_and_edges():
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((50, 64)) * np.exp(rng.uniform(-20, 20, (50, 1)))).astype(np.float32)
    c, s = serving.quantise(x)
    # half a step, plus the float32 roundings of 127 / amax, of the product (2 x 2^-24 of up to 127
    # steps) and of the scale (2^-24 of up to 127 steps)
    assert (np.abs(c * s.astype(np.float64)[:, None] - x) <= s[:, None] * (0.5 + 127 * 3 * 2.0 ** -24)).all()
    assert (np.abs(c).max(1) == 127).all()
    e = np.zeros((4, 16), np.float32)
    e[1, 3], e[2, 0], e[3, 5] = 1e-38, np.inf, np.nan
    c, s = serving.quantise(e)
    assert (c == 0).all() and s[0] == 0 and s[1] == 0 and np.isnan(s[2:]).all()


def test_write_then_read_returns_the_stored_values():
    rng = np.random.default_rng(6)
    for q8 in (False, True):
        c = cache(rng, [21, 0, 40], 2, 16, 16, q8)
        q_start = [0, 5, 6, 26]
        k, v = (rng.standard_normal((26, 2, 16)).astype(np.float32) for _ in range(2))
        serving.paged_write(c, k, v, q_start)
        rk, rv = serving.paged_read(c, q_start, 27)
        assert (rk[5] == 0).all() and np.isnan(rk[26]).all()  # a padding row; a row of no sequence
        live = [r for r in range(26) if r != 5]
        if q8:
            codes, s = serving.quantise(v[live])
            assert np.array_equal(rv[live], codes.astype(np.float32) * s[..., None])
        else:
            assert np.array_equal(rk[live], serving.bf16(k[live]))


def test_bad_pages_are_not_followed():
    rng = np.random.default_rng(7)
    c = cache(rng, [40], 1, 16, 16, False)
    c.table[0, 1] = 99
    y, lse, _ = serving.paged_attn(c, np.ones((1, 1, 16)), [0, 1], 0.5)
    good = [j for j in range(40) if not 16 <= j < 32]
    z = np.array([0.5 * c.vector("k", *c.place(0, j))[0].sum() for j in good])
    assert abs(lse[0, 0] - np.log(np.exp(z).sum())) < 1e-12
    assert c.place(0, 20) is None and c.place(0, 48) is None and c.place(0, -1) is None


def test_w4_round_trip_and_edges():
    rng = np.random.default_rng(8)
    w = rng.standard_normal((5, 128)).astype(np.float32)
    w[0, :64], w[1, 3], w[2, 70] = 0, np.inf, np.nan
    p, s = serving.quant_w4(w, 64)
    d = serving.dequant_w4(p, s, 64)
    assert s[0, 0] == 0 and (d[0, :64] == 0).all() and np.isnan(s[1, 0]) and np.isnan(s[2, 1])
    # half a step, and the largest value may be cut by the scale's rounding (7 steps x 2^-8)
    fine = np.isfinite(s).repeat(64, 1)
    assert (np.abs(d - w)[fine] <= (s.repeat(64, 1) * (0.5 + 7 * 2.0 ** -8))[fine]).all()
    x = serving.dequant_w4(np.array([[0x8F, 0x10]], np.uint8).repeat(16, 1), np.array([[2.0]]), 64)
    assert x[0, 0] == 14 and x[0, 1] == 0


def test_sampler_agrees_with_the_top_k_oracle():
    rng = np.random.default_rng(9)
    for i in range(200):
        x, u, k = rng.standard_normal(50).round(1), rng.random(), int(rng.integers(1, 60))
        assert serving.sample_row(x, u, 0.7, k)[0] == sampling.topk_sample(x, k, 0.7, u)


def test_sampler_frequencies_and_filters():
    p = np.array([0.5, 0.25, 0.15, 0.07, 0.03])
    x = np.log(p[[3, 0, 2, 4, 1]])
    us = (np.arange(2000) + 0.5) / 2000
    share = np.bincount([serving.sample_row(x, u)[0] for u in us], minlength=5) / 2000
    assert np.abs(share - p[[3, 0, 2, 4, 1]]).max() < 1e-3
    assert {serving.sample_row(x, u, top_p=0.8)[0] for u in us} == {1, 2, 4}
    assert {serving.sample_row(x, u, min_p=0.2)[0] for u in us} == {1, 2, 4}
    assert {serving.sample_row(x, u, top_p=0.0)[0] for u in us} == {1}
    # top_p is a share of what top_k left: 0.8 of (0.5 + 0.25) needs both
    assert {serving.sample_row(x, u, top_k=2, top_p=0.8)[0] for u in us} == {1, 4}
    assert {serving.sample_row(x, u, top_k=2, top_p=0.6)[0] for u in us} == {1}


def test_sampler_edges():
    inf, nan = np.inf, np.nan
    assert serving.sample_row([-inf, nan], 0.5)[:2] == (-1, 0.0)
    assert serving.sample_row([1, inf, inf, nan], 0.6)[:2] == (2, 0.5)
    assert serving.sample_row([1, 3, 3], 0.9, temperature=0.0)[:2] == (1, 1.0)
    assert serving.sample_row([1, 3, 3], 0.9, temperature=nan)[0] == 1
    assert serving.sample_row([1.0, 2.0, -inf], 1.0)[0] == 1  # no running sum exceeds the total: the last kept
    assert serving.sample_row([1, 2, 3], 0.0)[0] == 0


def test_binding_refuses_mismatched_cache_tensors():
    import torch

    from gpt_decoder_gb300 import gk

    k = torch.zeros(3, 2, 16, 32, dtype=torch.int8)
    s = torch.zeros(3, 2, 16)
    t, n = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    c = gk.PagedKv(k, k.clone(), s, s.clone(), t, n)
    assert (c.struct.n_pages, c.struct.Hkv, c.struct.page_size, c.struct.hs, c.struct.max_pages) == (3, 2, 16, 32, 4)
    for bad in ((k, k[:2], s, s, t, n), (k, k, None, None, t, n), (k.bfloat16(), k.bfloat16(), s, s, t, n), (k.half(), k.half(), None, None, t, n),
                (k, k, s[:2], s, t, n), (k, k, s, s, t.long(), n), (k, k, s, s, t[0], n), (k.float(), k.float(), None, None, t, n),
                (k.transpose(0, 1), k.transpose(0, 1), s, s, t, n)):
        with pytest.raises(ValueError):
            gk.PagedKv(*bad)
    with pytest.raises(ValueError):
        gk._batch(c, 3, "gk_paged_read")


def test_binding_refuses_cache_tensors_on_different_devices():
    import torch

    from gpt_decoder_gb300 import gk

    k = torch.zeros(3, 2, 16, 32, dtype=torch.bfloat16)
    t, n = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    gk.PagedKv(k, k.clone(), None, None, t, n)
    with pytest.raises(ValueError):
        gk.PagedKv(k, k.clone(), None, None, t.to("meta"), n)


def test_calls_without_a_context_are_refused():
    import ctypes as ct

    from gpt_decoder_gb300 import gk

    c = gk.gk_paged_kv()
    assert gk._lib.gk_paged_write(None, ct.byref(c), 0, None, 0, None, 0, None, 1, 1) == gk.GK_ERR_ARG
    assert gk._lib.gk_paged_read(None, ct.byref(c), 0, None, 0, None, 0, None, 1, 1) == gk.GK_ERR_ARG
    assert gk._lib.gk_paged_attn(None, ct.byref(c), 1, None, 0, None, 0, None, None, 1, 1, 1, 1, 1.0) == gk.GK_ERR_ARG
    assert gk._lib.gk_quant_w4(None, None, 0, 0, None, None, 32, 32, 1) == gk.GK_ERR_ARG
    assert gk._lib.gk_matvec_w4(None, 1, None, 0, None, None, 32, None, None, 0, None, 0, 0, 1, 32, 1) == gk.GK_ERR_ARG
    assert gk._lib.gk_sample_rows(None, 0, None, 0, 1, 1, None, None, None, None, None, None, None) == gk.GK_ERR_ARG
