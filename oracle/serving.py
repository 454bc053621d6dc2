"""Oracle of the serving operators: the paged cache, attention over it, 4-bit products, filtered sampling.

TEST INFRASTRUCTURE ONLY (see the package docstring): never imported by the product path.

Arrays are numpy; arithmetic is float64 except where the stored codes define a float32 order of
operations (the cache's quantiser and the weight quantiser round step by step in float32, as their
definitions say). bfloat16 values are passed as the float32 numbers they stand for.
"""
from __future__ import annotations

import numpy as np


def bf16(x):
    """Round float32 to bfloat16 (nearest even), kept as float32; NaN stays NaN."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), x, r)


# ---------------------------------------------------------------------------------- paged cache
def quantise(x):
    """(codes, scales) of vectors x [..., hs] in float32: scale = amax / 127, code = rint(x * (127 / amax))."""
    x = np.asarray(x, np.float32)
    m = np.abs(x).max(-1)
    odd = ~np.isfinite(x).all(-1)
    none = ~(m >= np.float32(2.0 ** -100)) | odd
    with np.errstate(all="ignore"):
        inv = np.where(none, np.float32(0), np.float32(127) / m)
        c = np.rint(np.where(odd[..., None], np.float32(0), x) * inv[..., None])
        scale = np.where(odd, np.float32(np.nan), np.where(none, np.float32(0), m / np.float32(127)))
    return np.clip(c, -127, 127).astype(np.int8), scale.astype(np.float32)


class Pages:
    """A paged cache on the host: k, v [n_pages, Hkv, page, hs] (int8 with scales, or bf16 values as float32)."""

    def __init__(self, k, v, k_scale, v_scale, table, kv_len):
        self.k, self.v, self.k_scale, self.v_scale = (None if a is None else a.copy() for a in (k, v, k_scale, v_scale))
        self.table, self.kv_len = table, kv_len
        self.n_pages, self.Hkv, self.page, self.hs = k.shape

    def place(self, b, pos):
        """(page, row) of a position, or None where the device refuses it."""
        if pos < 0 or pos >= self.table.shape[1] * self.page:
            return None
        i = int(self.table[b, pos // self.page])
        return (i, pos % self.page) if 0 <= i < self.n_pages else None

    def vector(self, which, page, row):
        a, s = (self.k, self.k_scale) if which == "k" else (self.v, self.v_scale)
        if s is None:
            return a[page, :, row].astype(np.float64)
        return (a[page, :, row].astype(np.float32) * s[page, :, row, None]).astype(np.float64)


def rows_of(q_start, kv_len):
    """(row, sequence, position) of every row of a call."""
    for b in range(len(q_start) - 1):
        n = int(q_start[b + 1]) - int(q_start[b])
        for i in range(n):
            yield int(q_start[b]) + i, b, int(kv_len[b]) - n + i


def paged_write(c, k, v, q_start):
    """k, v [rows, Hkv, hs] into the cache."""
    for r, b, pos in rows_of(q_start, c.kv_len):
        at = c.place(b, pos)
        if at is None:
            continue
        for a, s, x in ((c.k, c.k_scale, k), (c.v, c.v_scale, v)):
            if s is None:
                a[at[0], :, at[1]] = bf16(x[r])
            else:
                a[at[0], :, at[1]], s[at[0], :, at[1]] = quantise(x[r])


def paged_read(c, q_start, rows):
    """(k, v) [rows, Hkv, hs] in float32; rows of no sequence are NaN here (the device leaves them)."""
    out = np.full((2, rows, c.Hkv, c.hs), np.nan, np.float32)
    for r, b, pos in rows_of(q_start, c.kv_len):
        at = c.place(b, pos)
        for j, which in enumerate("kv"):
            out[j, r] = 0 if at is None else c.vector(which, *at)
    return out


def paged_attn(c, q, q_start, scale):
    """q [rows, H, hs] -> (y, lse, spread): y [rows, H, hs], lse [rows, H] and spread = sum_j p_j |v_j|, the
    size that errors of the weights go by. Only visible keys are touched."""
    rows, H, hs = q.shape
    y, spread, lse = np.zeros((rows, H, hs)), np.zeros((rows, H, hs)), np.full((rows, H), -np.inf)
    G = H // c.Hkv
    for b in range(len(q_start) - 1):
        s0, n = int(q_start[b]), int(q_start[b + 1]) - int(q_start[b])
        kv = int(c.kv_len[b])
        places = [(j, c.place(b, j)) for j in range(kv)] if n else []
        at = [(j, p) for j, p in places if p is not None]
        if not at:
            continue
        pos = np.array([j for j, _ in at])
        pg, rw = np.array([p[0] for _, p in at]), np.array([p[1] for _, p in at])

        def held(a, s):
            x = a[pg, :, rw].astype(np.float32)
            return (x if s is None else x * s[pg, :, rw][..., None]).astype(np.float64)

        k, v = held(c.k, c.k_scale), held(c.v, c.v_scale)  # [kv, Hkv, hs]
        for i in range(n):
            m = int(np.searchsorted(pos, kv - n + i, side="right"))
            if m == 0:
                continue
            for h in range(H):
                with np.errstate(all="ignore"):
                    z = scale * (k[:m, h // G] @ q[s0 + i, h].astype(np.float64))
                    t = z.max()
                    w = np.exp(z - t)
                    l = w.sum()
                    y[s0 + i, h] = w @ v[:m, h // G] / l
                    spread[s0 + i, h] = w @ np.abs(v[:m, h // G]) / l
                    lse[s0 + i, h] = t + np.log(l)
    return y, lse, spread


# -------------------------------------------------------------------------------- 4-bit weights
def quant_w4(w, group):
    """(packed uint8 [M, K/2], scales as float32 [M, K/group]) of w [M, K] float32."""
    M, K = w.shape
    g = w.astype(np.float32).reshape(M, K // group, group)
    odd = ~np.isfinite(g).all(-1)
    with np.errstate(all="ignore"):
        s = bf16(np.where(odd, np.float32(np.nan), np.abs(g).max(-1) / np.float32(7)))
        c = np.where((s > 0)[..., None], np.clip(np.rint(g / s[..., None]), -7, 7), 0)
    c = (np.where(odd[..., None], 0, c) + 8).astype(np.uint8).reshape(M, K)
    return c[:, 0::2] | (c[:, 1::2] << 4), s


def dequant_w4(packed, scales, group):
    """float64 [M, K]."""
    M, K = packed.shape[0], packed.shape[1] * 2
    c = np.empty((M, K))
    c[:, 0::2], c[:, 1::2] = packed & 15, packed >> 4
    return (c - 8) * np.repeat(scales.astype(np.float64), group, axis=1)


# ------------------------------------------------------------------------------------- sampling
def sample_row(x, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """(index, probability, distance) for one row of logits; distance is how far, as a share of the kept
    weight, the decision was from going another way (rows nearer than rounding are not told apart)."""
    x = np.where(np.isnan(np.asarray(x, np.float64)), -np.inf, np.asarray(x, np.float64))
    V, t = x.size, 1.0 if temperature is None else float(temperature)
    top = x.max()
    if top == -np.inf:
        return -1, 0.0, np.inf
    if not t > 0:
        return int(np.argmax(x)), 1.0, np.inf
    w = np.where(x == top, 1.0, 0.0)
    if np.isfinite(top):
        with np.errstate(over="ignore"):
            w = np.where(x == -np.inf, 0.0, np.exp((x - top) / t))
    w[x == top] = 1.0
    least, near = -np.inf, np.inf
    down = np.sort(x)[::-1]
    if top_k is not None and 0 < top_k < V:
        least = down[top_k - 1]
    if top_p is not None and top_p < 1:
        order = np.argsort(-x, kind="stable")
        order = order[x[order] >= least]
        sums = np.cumsum(w[order])
        want = float(top_p) * sums[-1]
        j = min(int(np.searchsorted(sums, want)), order.size - 1) if top_p > 0 else 0
        least = max(least, x[order[j]])
        if top_p > 0:  # between which sums of distinct values the share falls
            ends = np.append(x[order][1:] != x[order][:-1], True)
            near = np.abs(sums[ends] - want).min() / sums[-1]
    keep = (x >= least) & (w > 0)
    if min_p is not None and min_p > 0:
        near = min(near, np.abs(w[keep] - min(min_p, 1.0)).min() if min_p < 1 else np.inf)
        keep &= w >= min(float(min_p), 1.0)
    where = np.flatnonzero(keep)
    sums = np.cumsum(w[where])
    over = np.flatnonzero(sums > float(u) * sums[-1])
    j = int(over[0]) if over.size else where.size - 1
    if 0 < float(u) < 1:
        near = min(near, np.abs(sums / sums[-1] - float(u)).min())
    return int(where[j]), float(w[where[j]] / sums[-1]), near
