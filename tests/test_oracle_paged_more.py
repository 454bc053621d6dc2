"""Pins of the oracle's shared prefixes, attention weights and eviction: against torch in float64 and by hand; and what the
binding refuses without a GPU."""
import numpy as np
import pytest

from oracle import serving
from tests.test_oracle_serving import cache


@pytest.mark.parametrize("q8", [False, True])
def test_mass_is_the_softmax_columns(q8):
    import torch

    rng = np.random.default_rng(1)
    kv_len, n, H, Hkv, hs = [37, 16, 5], [4, 16, 1], 4, 2, 16
    c = cache(rng, kv_len, Hkv, hs, 16, q8)
    qs = np.concatenate([[0], np.cumsum(n)])
    q = serving.bf16(rng.standard_normal((sum(n), H, hs)))
    lse = serving.paged_attn(c, q, qs, 0.3)[1]
    old = rng.random((c.n_pages, Hkv, 16))
    got = serving.paged_mass(c, q, lse, qs, 0.3, old=old, decay=0.5, first=[3, 0, 9])
    every = np.concatenate([[0], np.cumsum(kv_len)])
    k = serving.paged_read(c, every, every[-1])[0].astype(np.float64)
    seen = 0
    for b in range(3):
        kb = torch.tensor(k[every[b] : every[b + 1]]).repeat_interleave(H // Hkv, 1)
        z = torch.einsum("ihd,jhd->hij", torch.tensor(q[qs[b] : qs[b + 1]].astype(np.float64)), kb) * 0.3
        mask = torch.ones(n[b], kv_len[b], dtype=torch.bool).tril(kv_len[b] - n[b])
        w = z.masked_fill(~mask, -np.inf).softmax(-1).sum(1).view(Hkv, H // Hkv, -1).sum(1).numpy()
        for j in range([3, 0, 9][b], kv_len[b]):
            p, r = c.place(b, j)
            for h in range(Hkv):
                want = w[h, j] + (0.5 * old[p, h, r] if j < kv_len[b] - n[b] else 0)
                assert abs(got[p, h, r][0] - want) < 1e-12 and got[p, h, r][1] >= w[h, j]
                seen += 1
    assert seen == len(got) == Hkv * (34 + 16)


def test_rows_without_weight_and_nan():
    rng = np.random.default_rng(2)
    c = cache(rng, [3], 1, 16, 16, False)
    q = np.ones((2, 1, 16), np.float32)
    got = serving.paged_mass(c, q, np.array([[-np.inf], [1.0]]), [0, 2], 0.1)
    alone = serving.paged_mass(c, q[1:], np.array([[1.0]]), [0, 1], 0.1)
    assert {at: m for at, (m, _) in got.items()} == {at: m for at, (m, _) in alone.items()}
    got = serving.paged_mass(c, q, np.array([[np.nan], [1.0]]), [0, 2], 0.1)
    assert [np.isnan(got[c.place(0, j)[0], 0, j][0]) for j in range(3)] == [True, True, False]  # the first row sees two


def test_evict_by_hand():
    table = np.array([[1, 0]], np.int32)
    k = np.arange(2 * 16, dtype=np.float32).reshape(2, 1, 16, 1).repeat(16, 3)
    c = serving.Pages(k, -k, None, None, table, np.array([20], np.int32))
    mass = np.zeros((2, 1, 16), np.float32)
    mass[1, 0, 3], mass[1, 0, 7], mass[0, 0, 0], mass[1, 0, 0] = 2, np.nan, 1, 9  # positions 3, 7, 16, 0
    to = serving.Pages(np.zeros_like(k), np.zeros_like(k), None, None, np.array([[0]], np.int32), np.array([0], np.int32))
    to_mass = np.full((2, 1, 16), 5, np.float32)
    new_len, kept = serving.paged_evict(c, mass, to, to_mass, [1], 6, 2)
    # behind position 0: the last two, then 3 and 16, then of the zeros the lowest positions
    assert new_len.tolist() == [7] and kept.tolist() == [[[1, 2, 3, 16, 18, 19]]]
    assert to.k[0, 0, :8, 0].tolist() == [16, 17, 18, 19, 0, 2, 3, 0] and to.v[0, 0, 3, 0] == -19
    assert to_mass[0, 0].tolist() == [9, 0, 0, 2, 1, 0, 0] + [5] * 9
    new_len, kept = serving.paged_evict(c, mass, to, to_mass, None, 30, 2)  # nothing to cut; 20 tokens, room for 16
    assert new_len.tolist() == [20] and kept[0, 0].tolist() == list(range(20)) + [-1] * 10


def test_shared_prefix_is_looked_up_in_the_first_row():
    rng = np.random.default_rng(3)
    c = cache(rng, [40, 37, 36], 1, 16, 16, False)
    c.table[1, :2], c.table[2, :2] = c.table[0, :2], c.table[0, :2]
    q = serving.bf16(rng.standard_normal((3, 2, 16)))
    qs = [0, 1, 2, 3]
    want = serving.paged_attn(c, q, qs, 0.2)
    other = serving.Pages(c.k, c.v, None, None, c.table.copy(), c.kv_len)
    other.table[1, 0] = -1
    view = serving.SharedPages(other, [(0, 3, 32)], qs)
    assert view.place(1, 3) == c.place(0, 3) and view.place(1, 33) == c.place(1, 33)
    for a, b in zip(serving.paged_attn(view, q, qs, 0.2), want):
        assert np.array_equal(a, b)
    assert not serving.SharedPages(other, [(0, 3, 37)], qs).lead.get(1)  # its row lies in the prefix


def test_binding_checks_the_batch():
    from types import SimpleNamespace

    import torch

    from gpt_decoder_gb300 import gk

    ctx = SimpleNamespace(handle=None)
    k = torch.zeros(2, 1, 16, 16, dtype=torch.bfloat16)
    h = gk.PagedKv(k, k, None, None, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    for fn, args in ((gk.gk_paged_attn_shared, (ctx, h, 1, None, 0, None, 0, None, None, 2, None, None, 1, 1, 1, 1, 1, 1.0)),
                     (gk.gk_paged_mass, (ctx, h, 1, None, 0, None, None, 1.0, None, None, None, 2, 1, 1, 1, 1.0)),
                     (gk.gk_paged_evict, (ctx, h, None, h, None, None, 8, 2, None, None, 2))):
        with pytest.raises(ValueError):
            fn(*args)
