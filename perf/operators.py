"""The serving operators as measured cases: attention of new tokens over a paged cache, the cache's
quantising write and its read back, products with 4-bit weights, and filtered sampling.

`run` computes each operator either in its plain form (elementary torch operations in 32 bits, 64
for the sampling weights, rounded once at the end) or, where `own` is true, through libgk's entry
points. `exact` is the operators' definition once more, in 64 bits and written apart.

Shared conventions of the paged cache: sequence b has tokens q_start[b] .. q_start[b+1]-1 in this
call, the last ones of the kv_len[b] tokens it then has; token i of n sits at position
kv_len[b] - n + i, in row pos % page of page page_table[b][pos // page]. A position below zero is
padding: nothing is stored for it, it reads back as zeros, and its attention output is zero.
"""
import math
import random

import torch

own = False

GROUPS = (32, 64, 128)
PAGES = (16, 32, 64, 128, 256)


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one sequence, one new token, the GPT-2-124M head layout: the latency of a single call
        dict(name="attn_one_token", op="attn", B=1, n=1, kv=777, H=12, Hkv=12, hs=64, page=16, q8=False, lens=1),
        # a decode batch of unequal lengths over an 8-bit cache with shared key/value heads
        dict(name="attn_decode_ragged", op="attn", B=48, n=1, kv=8191, H=32, Hkv=8, hs=128, page=64, q8=True, lens=2),
        # prompts continued in chunks, GPT-2-124M heads, bf16 cache
        dict(name="attn_chunk", op="attn", B=3, n=1000, kv=8100, H=12, Hkv=12, hs=64, page=32, q8=False, lens=3),
        # the largest: long chunks behind long prefixes over an 8-bit cache, shared heads
        dict(name="attn_chunk_long", op="attn", B=2, n=2048, kv=16384, H=32, Hkv=8, hs=128, page=64, q8=True, lens=4),
        # one new token for each of 16 sequences quantised into the cache and handed on as stored
        dict(name="store_decode", op="store", B=16, n=1, kv=1024, Hkv=12, hs=64, page=16, q8=True, f32=False, lens=5),
        # whole prompt chunks stored
        dict(name="store_chunk", op="store", B=7, n=4096, kv=8192, Hkv=8, hs=128, page=64, q8=True, f32=False, lens=6),
        # a short sequence read back
        dict(name="read_one", op="read", B=1, n=333, kv=333, Hkv=12, hs=64, page=16, q8=True, f32=True, lens=7),
        # a batch's whole sequences read back (to move them, or for an operator that takes plain rows)
        dict(name="read_batch", op="read", B=16, n=16384, kv=16384, Hkv=8, hs=128, page=128, q8=True, f32=False, lens=8),
        # one row, temperature and top-k, GPT-2's vocabulary with its padded row stride
        dict(name="sample_one", op="sample", R=1, V=50257, bf16=False, mode="topk"),
        # a served batch: every row with filters of its own
        dict(name="sample_batch", op="sample", R=192, V=50257, bf16=False, mode="mixed"),
        # GPT-2-124M's fused q, k, v projection for one token
        dict(name="w4_one", op="w4", N=1, K=768, M=2304, group=64, f32=False, extra=True),
        # a wide layer for a few rows: the weights' bytes are what counts
        dict(name="w4_wide", op="w4", N=5, K=8192, M=28672, group=128, f32=False, extra=False),
    ]


def _log(rng, lo, hi):
    """An integer from lo to hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attn", "attn", "store", "read", "sample", "w4"))
    seed = rng.randrange(1 << 30)
    if op == "sample":
        V = _log(rng, 1000, 131072)
        R = _log(rng, 1, max(1, min(256, 192 * 50257 // V)))
        return dict(op=op, R=R, V=V, bf16=rng.random() < 0.3, mode=rng.choice(("topk", "topp", "minp", "mixed", "plain")))
    if op == "w4":
        group = rng.choice(GROUPS)
        K = group * _log(rng, max(1, 256 // group), 16384 // group)
        M = _log(rng, 64, max(64, min(50257, 8192 * 28672 // K)))
        return dict(op=op, N=_log(rng, 1, 32), K=K, M=M, group=group, f32=rng.random() < 0.5, extra=rng.random() < 0.5)
    hs = rng.choice((32, 64, 64, 80, 128, 128))
    page, q8, Hkv = rng.choice(PAGES), rng.random() < 0.5, _log(rng, 1, 16)
    if op == "attn":
        H = Hkv * rng.choice((1, 1, 2, 4, 8) if Hkv <= 8 else (1, 2))
        n = 1 if rng.random() < 0.35 else _log(rng, 2, 2048)
        kv = _log(rng, max(n, 16), max(n, 65536 if n <= 64 else 16384))
        B = _log(rng, 1, 64)
        while B > 1 and (B * H * n * kv > 2 * 32 * 2048 * 16384 or B * Hkv * hs * kv > 48 * 8 * 128 * 8192):
            B -= 1
        while H * n * kv * hs > 2 * 32 * 2048 * 16384 * 128 or Hkv * hs * kv > 48 * 8 * 128 * 8192:
            kv = max(n, kv // 2)
        return dict(op=op, B=B, n=n, kv=kv, H=H, Hkv=Hkv, hs=hs, page=page, q8=q8, lens=seed)
    n = _log(rng, 1, 4096 if op == "store" else 16384)
    kv = n + rng.randrange(0, 2048)
    B = _log(rng, 1, 64)
    most = 7 * 4096 * 8 * 128 if op == "store" else 16 * 16384 * 8 * 128 // 4
    while B > 1 and B * n * Hkv * hs > most:
        B -= 1
    while n * Hkv * hs > most:
        n //= 2
    return dict(op=op, B=B, n=n, kv=kv, Hkv=Hkv, hs=hs, page=page, q8=q8, f32=op == "read" and rng.random() < 0.4, lens=seed)


def _lens(case):
    """Per sequence: (new tokens, cached tokens with them). The first has the case's own sizes; in a batch of eight
    and more the last is a padding row (a token, and nothing cached)."""
    r, got = random.Random(case["lens"]), []
    for b in range(case["B"]):
        if b == 0:
            got.append((case["n"], case["kv"]))
        elif case["B"] >= 8 and b == case["B"] - 1:
            got.append((1, 0))
        else:
            n = _log(r, max(1, case["n"] // 4), case["n"])
            got.append((n, _log(r, max(n, case["kv"] // 16), case["kv"])))
    return got


def work(case):
    op = case["op"]
    if op == "sample":
        return {"bytes": case["R"] * (case["V"] * (2 if case["bf16"] else 4) + 28), "flops": 8 * case["R"] * case["V"]}
    if op == "w4":
        N, K, M = case["N"], case["K"], case["M"]
        w = M * K // 2 + 2 * M * K // case["group"]
        y = N * M * (4 if case["f32"] else 2)
        return {"bytes": w + 2 * N * K + y + (4 * M + 4 * N * M if case["extra"] else 0), "flops": 2 * N * K * M}
    lens, hs, Hkv = _lens(case), case["hs"], case["Hkv"]
    held = hs + 4 if case["q8"] else 2 * hs  # bytes of one cached head vector
    if op == "attn":
        H = case["H"]
        pairs = sum(sum(max(0, kv - n + i + 1) for i in range(n)) for n, kv in lens)
        return {"bytes": sum(2 * kv * Hkv * held + 2 * 2 * n * H * hs for n, kv in lens), "flops": 4 * H * hs * pairs}
    rows = sum(n for n, _ in lens)
    stored = sum(min(n, kv) for n, kv in lens)
    if op == "store":  # rows read, written to the cache, and handed on as stored
        return {"bytes": 2 * Hkv * (rows * hs * 2 + stored * held + rows * hs * 2), "flops": 6 * rows * Hkv * hs}
    return {"bytes": 2 * Hkv * (stored * held + rows * hs * (4 if case["f32"] else 2)), "flops": 2 * rows * Hkv * hs}


# ------------------------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed % (1 << 62))


_contexts = {}


def _context():
    """The context of the current device and stream, kept as a program keeps it. (A state has the one of the stream that
    it was prepared on, and its passes run there.)"""
    from gpt_decoder_gb300 import gk

    stream = torch.cuda.current_stream()
    at = stream.device_index, stream.cuda_stream
    if at not in _contexts:
        _contexts[at] = gk.Ctx(stream.cuda_stream, workspace_bytes=256 << 20)
    return _contexts[at]


def prepare(case, seed):
    g, op, dev = _gen(seed), case["op"], "cuda"
    s = {"case": dict(case), "op": op}
    if op == "sample":
        R, V = case["R"], case["V"]
        ld = -(-V // 64) * 64
        x = torch.randn(R, ld, generator=g, device=dev) * 2.0
        hot = torch.randint(0, V, (R, 24), generator=g, device=dev)  # a few likely tokens, as a trained model's rows have
        x.scatter_add_(1, hot, torch.empty(R, 24, device=dev).exponential_(0.25, generator=g))
        mode = case["mode"]
        k = torch.randint(1, 100, (R,), generator=g, device=dev).to(torch.int32)
        p = torch.rand(R, generator=g, device=dev) * 0.5 + 0.5
        m = torch.rand(R, generator=g, device=dev) * 0.1
        t = torch.rand(R, generator=g, device=dev) * 0.7 + 0.5
        if mode == "mixed":  # each row has some of the filters on
            on = torch.randint(0, 8, (R,), generator=g, device=dev)
            k, p, m = torch.where(on % 2 == 1, k, 0), torch.where(on // 2 % 2 == 1, p, 1.0), torch.where(on // 4 == 1, m, 0.0)
        s.update(logits=x.to(torch.bfloat16) if case["bf16"] else x, ld=ld, u=torch.rand(R, generator=g, device=dev), t=t,
                 k=k if mode in ("topk", "mixed") else None, p=p if mode in ("topp", "mixed") else None,
                 m=m if mode in ("minp", "mixed") else None)
        s.update(next=torch.empty(R, dtype=torch.int32, device=dev), prob=torch.empty(R, device=dev))
    elif op == "w4":
        N, K, M, G = case["N"], case["K"], case["M"], case["group"]
        s["x"] = torch.randn(N, K, generator=g, device=dev).to(torch.bfloat16)
        # two 4-bit codes a byte (even k in the low half), code c stands for c - 8; bell-shaped as quantised weights are
        c = [(torch.randn(M, K // 2, generator=g, device=dev) * 2.4).round_().clamp_(-8, 7).add_(8).to(torch.uint8) for _ in range(2)]
        s["w"] = c[0] | (c[1] << 4)
        s["scales"] = ((torch.rand(M, K // G, generator=g, device=dev) + 0.5) * (0.4 / math.sqrt(K))).to(torch.bfloat16)
        s["bias"] = torch.randn(M, generator=g, device=dev) if case["extra"] else None
        s["res"] = torch.randn(N, M, generator=g, device=dev) if case["extra"] else None
        s["y"] = torch.empty(N, M, dtype=torch.float32 if case["f32"] else torch.bfloat16, device=dev)
    else:
        lens, B, Hkv, hs, page = _lens(case), case["B"], case["Hkv"], case["hs"], case["page"]
        rows = sum(n for n, _ in lens)
        width = max(1, max(-(-kv // page) for _, kv in lens))
        need = [-(-kv // page) for _, kv in lens]
        pages = max(1, sum(need))
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)  # pages lie anywhere in the pool
        valid = torch.arange(width, device=dev)[None] < torch.tensor(need, device=dev)[:, None]
        table = torch.zeros(B, width, dtype=torch.int32, device=dev)
        table[valid] = order[: sum(need)]
        shape = (pages, Hkv, page, hs)
        s.update(table=table, width=width, pages=pages, rows=rows)
        s["q_start"] = torch.tensor([0] + [n for n, _ in lens], device=dev).cumsum(0).to(torch.int32)
        s["kv_len"] = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=dev)
        for x in ("k", "v"):
            if case["q8"]:
                s[x] = (torch.randn(shape, generator=g, device=dev) * 32).round_().clamp_(-127, 127).to(torch.int8)
                s[x + "_scale"] = (torch.rand(shape[:3], generator=g, device=dev) + 0.5) / 32
            else:
                s[x], s[x + "_scale"] = torch.randn(shape, generator=g, device=dev).to(torch.bfloat16), None
        if op == "attn":
            s["q"] = (torch.randn(rows, case["H"] * hs, generator=g, device=dev) * 1.5).to(torch.bfloat16)
            s["y"] = torch.empty(rows, case["H"] * hs, dtype=torch.bfloat16, device=dev)
        else:
            if op == "store":  # side by side, as a fused projection leaves them
                s["new"] = torch.randn(rows, 2 * Hkv * hs, generator=g, device=dev).to(torch.bfloat16)
            t = torch.float32 if case["f32"] else torch.bfloat16
            s["ko"], s["vo"] = (torch.empty(rows, Hkv * hs, dtype=t, device=dev) for _ in range(2))
    if own:
        from gpt_decoder_gb300 import gk

        s["gk"], s["ctx"] = gk, _context()
        if "table" in s:
            s["cache"] = gk.PagedKv(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["kv_len"])
    return s


# ------------------------------------------------------------------------------------- the pass
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_attn(s):
    c = s["case"]
    s["gk"].gk_paged_attn(s["ctx"], s["cache"], s["gk"].GK_BF16, s["q"], c["H"] * c["hs"], s["y"], c["H"] * c["hs"], None, s["q_start"], c["B"],
                          c["H"], s["rows"], c["n"], 1.0 / math.sqrt(c["hs"]))
    return s["y"]


def _own_read(s):
    c, gk = s["case"], s["gk"]
    w = c["Hkv"] * c["hs"]
    gk.gk_paged_read(s["ctx"], s["cache"], gk.GK_F32 if c["f32"] else gk.GK_BF16, s["ko"], w, s["vo"], w, s["q_start"], c["B"], s["rows"])
    return s["ko"], s["vo"]


def _own_store(s):
    c, gk = s["case"], s["gk"]
    w = c["Hkv"] * c["hs"]
    gk.gk_paged_write(s["ctx"], s["cache"], gk.GK_BF16, s["new"], 2 * w, s["new"][:, w:], 2 * w, s["q_start"], c["B"], s["rows"])
    return _own_read(s)


def _own_sample(s):
    c, gk = s["case"], s["gk"]
    gk.gk_sample_rows(s["ctx"], gk.GK_BF16 if c["bf16"] else gk.GK_F32, s["logits"], s["ld"], c["R"], c["V"], s["u"], s["t"], s["k"], s["p"], s["m"],
                      s["next"], s["prob"])
    return s["next"], s["prob"]


def _own_w4(s):
    c, gk = s["case"], s["gk"]
    gk.gk_matvec_w4(s["ctx"], gk.GK_BF16, s["x"], c["K"], s["w"], s["scales"], c["group"], s["bias"], s["res"], c["M"], s["y"], c["M"],
                    gk.GK_F32 if c["f32"] else gk.GK_BF16, c["N"], c["K"], c["M"])
    return s["y"]


def _places(s):
    """Of every row of the call: its sequence, its position, and the page and row of the page where it is kept."""
    r = torch.arange(s["rows"], device="cuda")
    start, kv = s["q_start"].long(), s["kv_len"].long()
    b = torch.searchsorted(start, r, right=True) - 1
    pos = kv[b] - start[b + 1] + r
    at = pos.clamp(min=0)
    page = s["case"]["page"]
    return b, pos, s["table"].long()[b, at // page], at % page


def _held(s, x):
    """The whole cache in 32 bits."""
    v = s[x].float()
    return v if s[x + "_scale"] is None else v * s[x + "_scale"][..., None]


def _plain_attn(s):
    c = s["case"]
    B, n, H, Hkv, hs, page = c["B"], c["n"], c["H"], c["Hkv"], c["hs"], c["page"]
    b, pos, _, _ = _places(s)
    i = torch.arange(s["rows"], device="cuda") - s["q_start"].long()[b]
    q = torch.zeros(B, n, H, hs, device="cuda")  # the chunks side by side, padded
    q[b, i] = s["q"].float().view(-1, H, hs)
    at = torch.full((B, n), -1, device="cuda")
    at[b, i] = pos
    q = q.view(B, n, Hkv, H // Hkv, hs).permute(0, 2, 3, 1, 4).reshape(B, Hkv, H // Hkv * n, hs)
    keys = s["table"].long()
    k, v = (_held(s, x)[keys].permute(0, 2, 1, 3, 4).reshape(B, Hkv, s["width"] * page, hs) for x in ("k", "v"))
    w = q @ k.transpose(2, 3)
    w *= 1.0 / math.sqrt(hs)
    seen = (torch.arange(s["width"] * page, device="cuda") <= at[:, :, None]).repeat(1, H // Hkv, 1)[:, None]
    w.masked_fill_(~seen, -math.inf)
    w -= w.amax(-1, keepdim=True).clamp(min=-3e38)  # a row that sees nothing stays at -inf
    w.exp_()
    y = (w @ v) / w.sum(-1, keepdim=True).clamp(min=1e-30)
    y = y.view(B, Hkv, H // Hkv, n, hs).permute(0, 3, 1, 2, 4).reshape(B, n, H * hs)
    s["y"].copy_(y[b, i])
    return s["y"]


def _plain_read(s):
    b, pos, page, row = _places(s)
    for x, out in (("k", "ko"), ("v", "vo")):
        v = s[x][page, :, row].float()
        if s[x + "_scale"] is not None:
            v *= s[x + "_scale"][page, :, row][..., None]
        s[out].copy_(torch.where(pos[:, None] < 0, 0.0, v.flatten(1)))
    return s["ko"], s["vo"]


def _plain_store(s):
    c = s["case"]
    _, pos, page, row = _places(s)
    page, row, kept = page[pos >= 0], row[pos >= 0], s["new"][pos >= 0]
    for x, v in zip(("k", "v"), kept.view(-1, 2, c["Hkv"], c["hs"]).unbind(1)):
        if c["q8"]:
            v = v.float()
            most = v.abs().amax(-1)
            s[x + "_scale"][page, :, row] = most / 127
            v = (v * (127 / most)[..., None]).round().to(torch.int8)
        s[x][page, :, row] = v
    return _plain_read(s)


def _plain_sample(s):
    V = s["case"]["V"]
    x = s["logits"][:, :V].double()
    R = x.shape[0]
    w = ((x - x.amax(1, keepdim=True)) / s["t"].double()[:, None]).exp()
    if s["k"] is not None or s["p"] is not None:
        down = x.sort(1, descending=True).values
    if s["k"] is not None:  # the k-th largest and all that equal it; k <= 0 keeps every token
        k = torch.where(s["k"] > 0, s["k"], V).clamp(max=V).long()
        w = torch.where(x < down.gather(1, k[:, None] - 1), 0.0, w)
    if s["p"] is not None:  # the fewest largest values (and all that equal the last) that reach the share p
        heavy = ((down - down[:, :1]) / s["t"].double()[:, None]).exp()
        if s["k"] is not None:
            heavy = torch.where(down < down.gather(1, k[:, None] - 1), 0.0, heavy)
        run_ = heavy.cumsum(1)
        first = (run_ < s["p"].double()[:, None] * run_[:, -1:]).sum(1).clamp(max=V - 1)
        w = torch.where((x < down.gather(1, first[:, None])) & (s["p"] < 1)[:, None], 0.0, w)
    if s["m"] is not None:  # at least the share m of the likeliest token
        w = torch.where(w < s["m"].double()[:, None], 0.0, w)
    run_ = w.cumsum(1)
    total = run_[:, -1:]
    pick = (run_ <= s["u"].double()[:, None] * total).sum(1).clamp(max=V - 1)
    s["next"].copy_(pick)
    s["prob"].copy_(w.gather(1, pick[:, None])[:, 0] / total[:, 0])
    return s["next"], s["prob"]


def _plain_w4(s):
    c = s["case"]
    M, K, G = c["M"], c["K"], c["group"]
    w = torch.stack((s["w"] & 15, s["w"] >> 4), 2).view(M, K // G, G).float() - 8
    w *= s["scales"].float()[..., None]
    y = s["x"].float() @ w.view(M, K).t()
    if s["bias"] is not None:
        y += s["bias"]
        y += s["res"]
    s["y"].copy_(y)
    return s["y"]


_own = dict(attn=_own_attn, read=_own_read, store=_own_store, sample=_own_sample, w4=_own_w4)
_plain = dict(attn=_plain_attn, read=_plain_read, store=_plain_store, sample=_plain_sample, w4=_plain_w4)


# --------------------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    if work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    return _exact[case["op"]](case, s)


def _sequence(case, s, b, x):
    """Sequence b's cached vectors [kv, Hkv, hs] in 64 bits."""
    kv = int(s["kv_len"][b])
    ids = [int(p) for p in s["table"][b, : -(-kv // case["page"])].tolist()]
    if not ids:
        return torch.zeros(0, case["Hkv"], case["hs"], dtype=torch.float64, device="cuda")
    at = torch.tensor(ids, device="cuda")
    v = s[x][at].double()
    if case["q8"]:
        v = v * s[x + "_scale"][at].double().unsqueeze(-1)
    return v.transpose(1, 2).reshape(-1, case["Hkv"], case["hs"])[:kv]


def _exact_attn(case, s):
    H, Hkv, hs = case["H"], case["Hkv"], case["hs"]
    y = torch.zeros(s["rows"], H, hs, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(-1, H, hs)
    base = 0
    for b, (n, kv) in enumerate(_lens(case)):
        k, v = _sequence(case, s, b, "k"), _sequence(case, s, b, "v")
        for lo in range(0, n if kv else 0, 512):
            hi = min(n, lo + 512)
            last = torch.arange(kv - n + lo, kv - n + hi, device="cuda")
            for h in range(H):
                z = q[base + lo : base + hi, h] @ k[:, h // (H // Hkv)].T / math.sqrt(hs)
                z[torch.arange(kv, device="cuda")[None, :] > last[:, None]] = -math.inf
                y[base + lo : base + hi, h] = torch.softmax(z, 1) @ v[:, h // (H // Hkv)]
        base += n
    return y.view(s["rows"], H * hs)


def _exact_rows(case, s, seqs):
    outs = []
    for x in ("k", "v"):
        parts = []
        for b, (n, kv) in enumerate(_lens(case)):
            got = seqs(b, x)[-n:].reshape(-1, case["Hkv"] * case["hs"])
            parts += [torch.zeros(n - got.shape[0], got.shape[1], dtype=torch.float64, device="cuda"), got]
        outs.append(torch.cat(parts))
    return tuple(outs)


def _exact_read(case, s):
    return _exact_rows(case, s, lambda b, x: _sequence(case, s, b, x))


def _exact_store(case, s):
    starts = s["q_start"].tolist()

    def stored(b, x):
        n, kv = _lens(case)[b]
        w = case["Hkv"] * case["hs"]
        new = s["new"][starts[b] : starts[b + 1], (0 if x == "k" else w) : (w if x == "k" else 2 * w)].double()
        new = new.view(n, case["Hkv"], case["hs"])[n - min(n, kv) :]
        if case["q8"] and new.numel():
            step = new.abs().max(dim=2, keepdim=True).values / 127
            new = torch.round(new / step) * step
        return new

    return _exact_rows(case, s, stored)


def _exact_sample(case, s):
    import numpy as np

    host = {k: None if s[k] is None else s[k].double().cpu().numpy() for k in ("u", "t", "k", "p", "m")}
    logits = s["logits"].double().cpu().numpy()
    ids, probs = [], []
    for r in range(case["R"]):
        x = logits[r, : case["V"]]
        order = np.argsort(-x, kind="stable")
        w = np.exp((x - x[order[0]]) / host["t"][r])
        least = -np.inf
        if host["k"] is not None and 0 < host["k"][r] < x.size:
            least = x[order[int(host["k"][r]) - 1]]
        if host["p"] is not None and host["p"][r] < 1:
            left = order[x[order] >= least]
            sums = np.cumsum(w[left])
            least = max(least, x[left[min(np.searchsorted(sums, host["p"][r] * sums[-1]), left.size - 1)]])
        keep = x >= least
        if host["m"] is not None:
            keep &= w >= host["m"][r]
        where = np.flatnonzero(keep)
        sums = np.cumsum(w[where])
        j = where[min(np.searchsorted(sums, host["u"][r] * sums[-1], side="right"), where.size - 1)]
        ids.append(j)
        probs.append(w[j] / sums[-1])
    return np.array(ids, dtype=np.int32), np.array(probs)


def _exact_w4(case, s):
    codes = torch.empty(case["M"], case["K"], dtype=torch.float64, device="cuda")
    codes[:, 0::2] = (s["w"] % 16).double() - 8
    codes[:, 1::2] = (s["w"] // 16).double() - 8
    w = codes * s["scales"].double().repeat_interleave(case["group"], dim=1)
    y = torch.einsum("nk,mk->nm", s["x"].double(), w)
    if case["extra"]:
        y = y + s["bias"].double() + s["res"].double()
    return y


_exact = dict(attn=_exact_attn, read=_exact_read, store=_exact_store, sample=_exact_sample, w4=_exact_w4)
