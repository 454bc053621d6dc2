"""More serving operators as measured cases, all of the paged cache: attention of a batch whose sequences share
long prefixes, the attention weight that each cached token receives, and the eviction of the lightest tokens.

`run` computes each operator either in its plain form (elementary torch operations in 32 bits, rounded once at
the end) or, where `own` is true, through libgk's entry points. `exact` is the operators' definition once more,
in 64 bits and written apart.

Shared conventions of the paged cache: sequence b has tokens q_start[b] .. q_start[b+1]-1 in this call, the last
ones of the kv_len[b] tokens it then has; token i of n sits at position kv_len[b] - n + i, in row pos % page of
page page_table[b][pos // page]. A position below zero is padding: its attention output is zero and it gives no
weight to any token.
* shared: sequences group_start[g] .. group_start[g+1]-1 hold the same first prefix_len[g] tokens; the others of
  a sequence are its own. The result is the attention over all of them.
* mass: per token and key / value head, decay * old (new tokens: nothing) + the sum of the softmax weights that the
  call's rows and the head's query heads give it; the softmax's log-sum-exp is an input, as attention leaves it.
* evict: per sequence and key / value head the first `first` tokens stay, the last `recent`, and of those between
  the heaviest (ties: the lowest position), `budget` behind the first ones in all; moved in their order to the
  pages of another table, with their mass. kept: their old positions, -1 behind the last.
"""
import math
import random

import torch

own = False

PAGES = (16, 32, 64, 128, 256)


# ------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a few continuations of one short prompt, a token each, GPT-2-124M heads: the latency of a single call
        dict(name="shared_few", op="shared", G=1, S=4, n=1, prefix=777, tail=40, H=12, Hkv=12, hs=64, page=16, q8=False, lens=1),
        # many samples of one long prompt over an 8-bit cache with shared key / value heads
        dict(name="shared_samples", op="shared", G=1, S=64, n=1, prefix=16384, tail=1024, H=32, Hkv=8, hs=128, page=64, q8=True, lens=2),
        # a served batch of several prompts with samples of each, a padding row at its end
        dict(name="shared_groups", op="shared", G=7, S=16, n=1, prefix=8100, tail=600, H=12, Hkv=12, hs=64, page=32, q8=False, lens=3),
        # the largest: chunks of new tokens (questions) behind two long shared documents
        dict(name="shared_chunks", op="shared", G=2, S=12, n=256, prefix=16384, tail=700, H=32, Hkv=8, hs=128, page=128, q8=False, lens=4),
        # one decoded token's weights added to a short sequence's
        dict(name="mass_one_token", op="mass", B=1, n=1, kv=777, H=12, Hkv=12, hs=64, page=16, q8=False, lens=5),
        # a decode batch of unequal lengths over an 8-bit cache with shared heads
        dict(name="mass_decode", op="mass", B=48, n=1, kv=8191, H=32, Hkv=8, hs=128, page=64, q8=True, lens=6),
        # prompts continued in chunks, GPT-2-124M heads, 8-bit cache
        dict(name="mass_chunk", op="mass", B=3, n=1000, kv=8100, H=12, Hkv=12, hs=64, page=32, q8=True, lens=7),
        # long chunks behind long prefixes, shared heads
        dict(name="mass_chunk_long", op="mass", B=2, n=2048, kv=16384, H=32, Hkv=8, hs=128, page=64, q8=False, lens=8),
        # one short sequence cut to its budget
        dict(name="evict_one", op="evict", B=1, kv=1100, first=4, budget=512, recent=64, Hkv=12, hs=64, page=16, q8=False, lens=9),
        # a decode batch that grew by a page a sequence and is cut back, 8-bit cache (handed on as stored)
        dict(name="evict_step", op="evict", B=16, kv=2116, first=4, budget=2048, recent=512, Hkv=12, hs=64, page=64, q8=True, lens=10),
        # a batch of prompts cut to a quarter after they were read
        dict(name="evict_batch", op="evict", B=48, kv=8191, first=16, budget=2048, recent=256, Hkv=8, hs=128, page=64, q8=False, lens=11),
        # long sequences cut to an eighth
        dict(name="evict_long", op="evict", B=3, kv=65536, first=64, budget=8192, recent=1024, Hkv=8, hs=128, page=128, q8=False, lens=12),
    ]


def _log(rng, lo, hi):
    """An integer from lo to hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("shared", "shared", "mass", "evict"))
    hs = rng.choice((32, 64, 64, 80, 128, 128))
    c = dict(op=op, hs=hs, page=rng.choice(PAGES), q8=rng.random() < 0.5, Hkv=_log(rng, 1, 16), lens=rng.randrange(1 << 30))
    Hkv = c["Hkv"]
    if op == "evict":
        c["budget"] = _log(rng, 8, 16384)
        c["recent"] = rng.randrange(0, c["budget"] + 1)
        c["first"] = rng.choice((0, 0, 4, rng.randrange(0, 200)))
        c["kv"], c["B"] = _log(rng, max(16, c["budget"] // 2), max(64, min(131072, c["budget"] * 64))), _log(rng, 1, 64)
        while c["B"] > 1 and c["B"] * Hkv * hs * c["kv"] > 3 * 65536 * 8 * 128:
            c["B"] -= 1
        while c["B"] * Hkv * hs * c["kv"] > 3 * 65536 * 8 * 128:
            c["kv"] //= 2
        return c
    c["H"] = H = Hkv * rng.choice((1, 1, 2, 4, 8) if Hkv <= 8 else (1, 2))
    if op == "mass":
        n = 1 if rng.random() < 0.35 else _log(rng, 2, 2048)
        kv = _log(rng, max(n, 16), max(n, 65536 if n <= 64 else 16384))
        B = _log(rng, 1, 64)
        while B > 1 and (B * H * n * kv > 2 * 32 * 2048 * 16384 or B * Hkv * hs * kv > 48 * 8 * 128 * 8192):
            B -= 1
        while H * n * kv * hs > 2 * 32 * 2048 * 16384 * 128 or Hkv * hs * kv > 48 * 8 * 128 * 8192:
            kv = max(n, kv // 2)
        c.update(B=B, n=n, kv=kv)
        return c
    n = 1 if rng.random() < 0.5 else _log(rng, 2, 512)
    G, S, prefix, tail = _log(rng, 1, 12), _log(rng, 2, 64), _log(rng, 16, 32768), n + _log(rng, 1, 2048)
    most, held = 24 * 256 * 32 * 16384, 64 * 1024 * 8 * 128 * 2

    def over():
        return (G * S * n * H * (prefix + tail) * hs > most * 128 or S * n * H * prefix > most // 2 or G * S * n * H * tail > most // 4
                or G * S * tail * Hkv * hs > held or G * prefix * Hkv * hs > held)

    while over() and G > 1:
        G -= 1
    while over() and S > 2:
        S -= 1
    while over() and prefix > 16:
        prefix //= 2
    c.update(G=G, S=S, n=n, prefix=prefix, tail=tail)
    return c


def _lens(case):
    """Per sequence: (new tokens, tokens with them). The first has the case's own sizes; in a batch of eight and more
    the last is a padding row (a token, and nothing cached)."""
    r, got = random.Random(case["lens"]), []
    most = case.get("n", 1)
    for b in range(case["B"]):
        if b == 0:
            got.append((most, case["kv"]))
        elif case["op"] == "mass" and case["B"] >= 8 and b == case["B"] - 1:
            got.append((1, 0))
        else:
            n = _log(r, max(1, most // 4), most)
            least = case["budget"] // 2 if case["op"] == "evict" else case["kv"] // 16
            got.append((n, _log(r, max(n, min(least, case["kv"])), case["kv"])))
    return got


def _groups(case):
    """Per group: (prefix, [(new tokens, tokens with the prefix and them) of each sequence]). The first group and its first
    sequence have the case's own sizes; with four groups and more the last sequence is a padding row."""
    r, got = random.Random(case["lens"]), []
    for g in range(case["G"]):
        prefix = case["prefix"] if g == 0 else _log(r, max(1, case["prefix"] // 8), case["prefix"])
        seqs = []
        for b in range(case["S"] if g == 0 else _log(r, 1, case["S"])):
            n = case["n"] if g + b == 0 else _log(r, max(1, case["n"] // 4), case["n"])
            tail = case["tail"] if g + b == 0 else _log(r, n, case["tail"])
            seqs.append((n, prefix + tail))
        if case["G"] >= 4 and g == case["G"] - 1:
            seqs.append((1, 0))
        got.append((prefix, seqs))
    return got


def _kept(case):
    """Tokens of each sequence after the eviction."""
    return [min(kv, case["first"] + case["budget"]) for _, kv in _lens(case)]


def _pairs(n, kv, start=0):
    """(row, key) pairs of n rows that see the keys from `start` on."""
    return sum(max(0, kv - n + i + 1 - start) for i in range(n))


def work(case):
    hs, Hkv = case["hs"], case["Hkv"]
    held = hs + 4 if case["q8"] else 2 * hs  # bytes of one cached head vector
    if case["op"] == "evict":  # all masses read; what is kept read and written, its mass and old position written
        kept = sum(_kept(case))
        back = 4 * hs + 2 * held if case["q8"] else 0  # 8-bit pages: handed on as stored
        return {"bytes": Hkv * (4 * sum(kv for _, kv in _lens(case)) + kept * (4 * held + 8 + back)), "flops": Hkv * sum(kv for _, kv in _lens(case))}
    H = case["H"]
    if case["op"] == "mass":  # keys, queries and their log-sum-exp, masses read and written
        lens = _lens(case)
        pairs = sum(_pairs(n, kv) for n, kv in lens)
        return {"bytes": sum(kv * Hkv * (held + 8) + n * H * (2 * hs + 4) for n, kv in lens), "flops": 2 * H * hs * pairs}
    total = {"bytes": 0, "flops": 0}
    for prefix, seqs in _groups(case):
        total["bytes"] += 2 * prefix * Hkv * held
        for n, kv in seqs:
            total["bytes"] += 2 * max(0, kv - prefix) * Hkv * held + 2 * 2 * n * H * hs
            total["flops"] += 4 * H * hs * _pairs(n, kv)
    return total


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


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pool(s, case, g, pages, prefix=""):
    """Keys and values of a pool of pages, as a model leaves them (8 bits: codes and their steps)."""
    shape = (pages, case["Hkv"], case["page"], case["hs"])
    for x in ("k", "v"):
        if case["q8"]:
            s[prefix + x] = (torch.randn(shape, generator=g, device="cuda") * 32).round_().clamp_(-127, 127).to(torch.int8)
            s[prefix + x + "_scale"] = (torch.rand(shape[:3], generator=g, device="cuda") + 0.5) / 32
        else:
            s[prefix + x], s[prefix + x + "_scale"] = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16), None


def _table(lens, page, g, shared=None):
    """Pages of a pool for sequences of these lengths, lying anywhere in it: (table, pages). shared[b] = (sequence, pages):
    the first `pages` pages are that sequence's."""
    own_pages = [max(0, -(-kv // page) - (shared[b][1] if shared and shared[b][0] != b else 0)) for b, kv in enumerate(lens)]
    width = max(1, max(-(-kv // page) for kv in lens))
    pages = max(1, sum(own_pages))
    order, at, rows = torch.randperm(pages, generator=g, device="cuda").tolist(), 0, []
    for b, need in enumerate(own_pages):
        lead = rows[shared[b][0]][: shared[b][1]] if shared and shared[b][0] != b and lens[b] else []
        row = lead + order[at : at + need]
        at += need
        rows.append(row + [0] * (width - len(row)))
    return _ints(rows), pages


def _places(s, table, b, pos):
    """Page and row of positions pos of sequences b."""
    page = s["case"]["page"]
    return s[table].long()[b, pos // page], pos % page


def _new_rows(s, seqs):
    s["rows"] = sum(n for n, _ in seqs)
    s["q_start"] = _ints([0] + [n for n, _ in seqs]).cumsum(0).to(torch.int32)
    s["kv_len"] = _ints([kv for _, kv in seqs])


def prepare(case, seed):
    g, op, dev = _gen(seed), case["op"], "cuda"
    s = {"case": dict(case), "op": op}
    Hkv, hs, page = case["Hkv"], case["hs"], case["page"]
    if op == "shared":
        groups = _groups(case)
        seqs = [x for _, members in groups for x in members]
        leaders, starts, shared = [], [0], []
        for prefix, members in groups:
            leaders.append(starts[-1])
            shared += [(starts[-1], prefix // page)] * len(members)
            starts.append(starts[-1] + len(members))
        _new_rows(s, seqs)
        s["table"], pages = _table([kv for _, kv in seqs], page, g, shared)
        _pool(s, case, g, pages)
        for (prefix, members), lead, end in zip(groups, leaders, starts[1:]):
            if prefix % page:  # the page in which a prefix ends is each sequence's own, with a copy of its tokens
                ids = s["table"][lead:end, prefix // page].long()
                ids = ids[torch.tensor([kv > 0 for _, kv in members], device=dev)]
                for x in ("k", "v", "k_scale", "v_scale"):
                    if s[x] is not None:
                        s[x][ids, :, : prefix % page] = s[x][ids[:1], :, : prefix % page]
        s["group_start"], s["prefix_len"] = _ints(starts), _ints([p for p, _ in groups])
        s["max_group"] = max(sum(n for n, _ in members) for _, members in groups)
        s["q"] = (torch.randn(s["rows"], case["H"] * hs, generator=g, device=dev) * 1.5).to(torch.bfloat16)
        s["y"] = torch.empty(s["rows"], case["H"] * hs, dtype=torch.bfloat16, device=dev)
    elif op == "mass":
        seqs = _lens(case)
        _new_rows(s, seqs)
        s["table"], pages = _table([kv for _, kv in seqs], page, g)
        _pool(s, case, g, pages)
        s["q"] = (torch.randn(s["rows"], case["H"] * hs, generator=g, device=dev) * 1.5).to(torch.bfloat16)
        s["old"] = torch.empty(pages, Hkv, page, device=dev).exponential_(20.0, generator=g)
        s["mass"], s["decay"] = torch.zeros(pages, Hkv, page, device=dev), 0.99
        s["lse"] = torch.empty(s["rows"], case["H"], device=dev)
        for b, (n, kv) in enumerate(seqs):  # as attention left it
            at = slice(int(s["q_start"][b]), int(s["q_start"][b + 1]))
            for lo in range(0, n, 512):
                z = _scores(s, b, kv, lo, min(n, lo + 512))
                s["lse"][at][lo : lo + 512] = z.logsumexp(2).permute(1, 0) if kv else -math.inf
    else:
        lens = [kv for _, kv in _lens(case)]
        s["kv_len"] = _ints(lens)
        s["table"], pages = _table(lens, page, g)
        _pool(s, case, g, pages)
        # weights as attention leaves them: over many orders of magnitude, some tokens never looked at
        m = (torch.randn(pages, Hkv, page, generator=g, device=dev) * 2.5 - 3).exp_()
        s["mass"] = m * (torch.rand(pages, Hkv, page, generator=g, device=dev) > 0.05)
        s["first"] = torch.full((case["B"],), case["first"], dtype=torch.int32, device=dev)
        kept = _kept(case)
        s["to_table"], s["to_pages"] = _table(kept, page, g)
        shape = (s["to_pages"], Hkv, page, hs)
        for x in ("k", "v"):
            s["to_" + x] = torch.zeros(shape, dtype=s[x].dtype, device=dev)
            s["to_" + x + "_scale"] = torch.zeros(shape[:3], device=dev) if case["q8"] else None
        s["to_mass"] = torch.zeros(shape[:3], device=dev)
        s["new_len"] = torch.zeros(case["B"], dtype=torch.int32, device=dev)
        s["kept"] = torch.empty(case["B"], Hkv, case["budget"], dtype=torch.int32, device=dev)
        if case["q8"]:
            s["rows"] = sum(kept)
            s["every"] = _ints([0] + kept).cumsum(0).to(torch.int32)
            s["ko"], s["vo"] = (torch.empty(s["rows"], Hkv * hs, dtype=torch.bfloat16, device=dev) for _ in range(2))
    if own:
        from gpt_decoder_gb300 import gk

        s["gk"], s["ctx"] = gk, _context()
        s["cache"] = gk.PagedKv(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["kv_len"])
        if op == "evict":
            s["to"] = gk.PagedKv(s["to_k"], s["to_v"], s["to_k_scale"], s["to_v_scale"], s["to_table"], s["new_len"])
    return s


def _scores(s, b, kv, lo, hi):
    """Scaled scores [H, rows lo .. hi-1, kv] of sequence b's new tokens, -inf where a key is not seen."""
    c = s["case"]
    H, Hkv, hs = c["H"], c["Hkv"], c["hs"]
    first, n = int(s["q_start"][b]), int(s["q_start"][b + 1] - s["q_start"][b])
    pos = torch.arange(kv, device="cuda")
    page, row = _places(s, "table", b, pos)
    k = s["k"][page, :, row].float()
    if s["k_scale"] is not None:
        k *= s["k_scale"][page, :, row][..., None]
    q = s["q"][first + lo : first + hi].float().view(hi - lo, Hkv, H // Hkv, hs).permute(1, 2, 0, 3).reshape(Hkv, -1, hs)
    z = (q @ k.permute(1, 2, 0)).view(H, hi - lo, kv) * (1.0 / math.sqrt(hs))
    return z.masked_fill_(pos > (kv - n + lo + torch.arange(hi - lo, device="cuda"))[:, None], -math.inf)


# ------------------------------------------------------------------------------------- the pass
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_shared(s):
    c, gk = s["case"], s["gk"]
    w = c["H"] * c["hs"]
    gk.gk_paged_attn_shared(s["ctx"], s["cache"], gk.GK_BF16, s["q"], w, s["y"], w, None, s["q_start"], s["kv_len"].shape[0],
                            s["group_start"], s["prefix_len"], s["prefix_len"].shape[0], c["H"], s["rows"], c["n"], s["max_group"],
                            1.0 / math.sqrt(c["hs"]))
    return s["y"]


def _own_mass(s):
    c, gk = s["case"], s["gk"]
    gk.gk_paged_mass(s["ctx"], s["cache"], gk.GK_BF16, s["q"], c["H"] * c["hs"], s["lse"], s["old"], s["decay"], s["mass"], None,
                     s["q_start"], c["B"], c["H"], s["rows"], c["n"], 1.0 / math.sqrt(c["hs"]))
    return s["mass"]


def _own_evict(s):
    c, gk = s["case"], s["gk"]
    gk.gk_paged_evict(s["ctx"], s["cache"], s["mass"], s["to"], s["to_mass"], s["first"], c["budget"], c["recent"], s["new_len"],
                      s["kept"], c["B"])
    if not c["q8"]:
        return s["to_k"], s["to_v"], s["to_mass"], s["new_len"], s["kept"]
    w = c["Hkv"] * c["hs"]
    gk.gk_paged_read(s["ctx"], s["to"], gk.GK_BF16, s["ko"], w, s["vo"], w, s["every"], c["B"], s["rows"])
    return s["ko"], s["vo"], s["to_mass"], s["new_len"], s["kept"]


def _held(s, x, page, row):
    """Cached vectors [..., Hkv, hs] in 32 bits."""
    v = s[x][page, :, row].float()
    return v if s[x + "_scale"] is None else v * s[x + "_scale"][page, :, row][..., None]


def _plain_shared(s):
    c = s["case"]
    H, Hkv, hs, n = c["H"], c["Hkv"], c["hs"], c["n"]
    G, base, row0 = H // Hkv, 0, 0
    for prefix, seqs in _groups(c):
        S, T = len(seqs), max(kv - prefix for _, kv in seqs)
        rows = sum(m for m, _ in seqs)
        m, kv = (torch.tensor([x[i] for x in seqs], device="cuda") for i in range(2))
        b, i = (torch.arange(n, device="cuda")[None] < m[:, None]).nonzero(as_tuple=True)  # the chunks side by side, padded
        at = torch.full((S, n), -1, device="cuda")
        at[b, i] = (kv - m)[b] + i
        q = torch.zeros(S, n, H, hs, device="cuda")
        q[b, i] = s["q"][row0 : row0 + rows].float().view(-1, H, hs)
        q = q.view(S, n, Hkv, G, hs)
        ids = torch.arange(S, device="cuda")[:, None] + base
        k, v = (_held(s, x, *_places(s, "table", base, torch.arange(prefix, device="cuda"))) for x in ("k", "v"))
        far = (prefix + torch.arange(T, device="cuda"))[None]  # the sequences' own tokens
        page, row = _places(s, "table", ids, far.clamp(max=s["table"].shape[1] * c["page"] - 1))
        k2, v2 = (_held(s, x, page, row) for x in ("k", "v"))
        z = q.permute(2, 0, 1, 3, 4).reshape(Hkv, S * n * G, hs) @ k.permute(1, 2, 0)
        z = z.view(Hkv, S, n, G, prefix)
        z *= 1.0 / math.sqrt(hs)
        z.masked_fill_(~(at[None, :, :, None, None] >= prefix), -math.inf)
        z2 = (q.permute(0, 2, 1, 3, 4).reshape(S, Hkv, n * G, hs) @ k2.permute(0, 2, 3, 1)).view(S, Hkv, n, G, T)
        z2 *= 1.0 / math.sqrt(hs)
        z2.masked_fill_(~(far[:, None, None, None] <= at[:, None, :, None, None]), -math.inf)
        z2 = z2.transpose(0, 1)  # [Hkv, S, n, G, T]
        top = torch.maximum(z.amax(-1, keepdim=True), z2.amax(-1, keepdim=True)).clamp(min=-3e38)
        z = z.sub_(top).exp_()
        z2 = (z2 - top).exp_()
        y = (z.reshape(Hkv, -1, prefix) @ v.transpose(0, 1)).view(Hkv, S, n, G, hs)
        y += (z2.transpose(0, 1).reshape(S, Hkv, n * G, T) @ v2.transpose(1, 2)).view(S, Hkv, n, G, hs).transpose(0, 1)
        y /= (z.sum(-1, keepdim=True) + z2.sum(-1, keepdim=True)).clamp(min=1e-30)
        s["y"][row0 : row0 + rows] = y.permute(1, 2, 0, 3, 4).reshape(S, n, H * hs)[b, i].to(torch.bfloat16)
        base, row0 = base + S, row0 + rows
    return s["y"]


def _plain_mass(s):
    c = s["case"]
    B, n, H, Hkv, hs = c["B"], c["n"], c["H"], c["Hkv"], c["hs"]
    start, kv = s["q_start"].long(), s["kv_len"].long()
    m = start[1:] - start[:-1]
    b, i = (torch.arange(n, device="cuda")[None] < m[:, None]).nonzero(as_tuple=True)
    q = torch.zeros(B, n, H, hs, device="cuda")  # the chunks side by side, padded
    q[b, i] = s["q"].float().view(-1, H, hs)
    lse = torch.full((B, n, H), math.inf, device="cuda")
    lse[b, i] = s["lse"]
    at = torch.full((B, n), -1, device="cuda")
    at[b, i] = (kv - m)[b] + i
    L = s["table"].shape[1] * c["page"]
    pos = torch.arange(L, device="cuda")
    page, row = _places(s, "table", torch.arange(B, device="cuda")[:, None], pos[None])
    k = _held(s, "k", page, row)  # [B, L, Hkv, hs]
    w = q.view(B, n, Hkv, H // Hkv, hs).permute(0, 2, 3, 1, 4).reshape(B, Hkv, H // Hkv * n, hs) @ k.permute(0, 2, 3, 1)
    w = w.view(B, Hkv, H // Hkv, n, L)
    w *= 1.0 / math.sqrt(hs)
    w -= lse.view(B, n, Hkv, H // Hkv).permute(0, 2, 3, 1)[..., None]
    w.exp_()
    w.masked_fill_(~(pos <= at[:, None, None, :, None]), 0)
    got = w.sum((2, 3)).transpose(1, 2)  # [B, L, Hkv]
    got += torch.where((pos < (kv - m)[:, None])[..., None], s["decay"] * s["old"][page, :, row], 0.0)
    held = pos < kv[:, None]
    s["mass"][page[held], :, row.expand(B, L)[held]] = got[held]
    return s["mass"]


def _plain_evict(s):
    c = s["case"]
    B, Hkv, budget, recent = c["B"], c["Hkv"], c["budget"], c["recent"]
    L = s["table"].shape[1] * c["page"]
    pos, kv, first = torch.arange(L, device="cuda"), s["kv_len"].long()[:, None], s["first"].long()[:, None]
    page, row = _places(s, "table", torch.arange(B, device="cuda")[:, None], pos[None])
    mass = s["mass"][page, :, row].transpose(1, 2)  # [B, Hkv, L]
    behind = (pos >= first) & (pos < kv)
    over = kv - first > budget
    between = (behind & (pos < kv - recent) & over)[:, None]
    order = torch.where(between, mass, -math.inf).sort(dim=2, descending=True, stable=True).indices
    stay = torch.zeros(B, Hkv, L, dtype=torch.bool, device="cuda")
    stay.scatter_(2, order[:, :, : budget - recent], True)
    stay &= between
    stay |= (behind & (~over | (pos >= kv - recent)))[:, None]
    new = torch.minimum(kv - first, torch.tensor(budget, device="cuda")).clamp(min=0) + torch.minimum(first, kv)
    kept = torch.where(stay, pos, L).sort(dim=2).values[:, :, :budget]
    if kept.shape[2] < budget:
        kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[2]), value=L)
    s["kept"].copy_(torch.where(kept < L, kept, -1))
    s["new_len"].copy_(new[:, 0])
    # what moves where: [B, Hkv, first + budget]
    slots = torch.arange(c["first"] + budget, device="cuda")
    src = torch.cat((slots[: c["first"]].expand(B, Hkv, -1), kept), 2)
    b, h, i = (slots < new)[:, None].expand(B, Hkv, -1).nonzero(as_tuple=True)
    src = src[b, h, i]
    p0, r0 = _places(s, "table", b, src)
    p1, r1 = _places(s, "to_table", b, i)
    for x in ("k", "v", "k_scale", "v_scale", "mass"):
        if s[x] is not None:
            s["to_" + x][p1, h, r1] = s[x][p0, h, r0]
    if not c["q8"]:
        return s["to_k"], s["to_v"], s["to_mass"], s["new_len"], s["kept"]
    b, i = (slots < new).nonzero(as_tuple=True)  # every token of every sequence, as stored
    p1, r1 = _places(s, "to_table", b, i)
    for x, out in (("k", "ko"), ("v", "vo")):
        s[out].copy_(_held(s, "to_" + x, p1, r1).flatten(1))
    return s["ko"], s["vo"], s["to_mass"], s["new_len"], s["kept"]


_own = dict(shared=_own_shared, mass=_own_mass, evict=_own_evict)
_plain = dict(shared=_plain_shared, mass=_plain_mass, evict=_plain_evict)


# --------------------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    if work(case)["flops"] > 2e12:
        return None
    return _exact[case["op"]](case, prepare(case, seed))


def _sequence(case, s, b, kv, x, table="table"):
    """Sequence b's cached vectors [kv, Hkv, hs] in 64 bits."""
    ids = s[table][b, : -(-kv // case["page"])].long()
    if ids.numel() == 0:
        return torch.zeros(0, case["Hkv"], case["hs"], dtype=torch.float64, device="cuda")
    v = s[x][ids].double()
    if case["q8"]:
        v = v * s[x + "_scale"][ids].double().unsqueeze(-1)
    return v.transpose(1, 2).reshape(-1, case["Hkv"], case["hs"])[:kv]


def _exact_shared(case, s):
    H, hs = case["H"], case["hs"]
    each = H // case["Hkv"]
    q = s["q"].double().view(-1, H, hs)
    out, at, b = [], 0, 0
    for prefix, seqs in _groups(case):
        doc = {x: _sequence(case, s, b, prefix, x) for x in ("k", "v")}
        for n, kv in seqs:
            y = torch.zeros(n, H, hs, dtype=torch.float64, device="cuda")
            if kv:
                k, v = (torch.cat((doc[x], _sequence(case, s, b, kv, x)[prefix:])) for x in ("k", "v"))
                hidden = torch.arange(kv, device="cuda")[None, :] > torch.arange(kv - n, kv, device="cuda")[:, None]
                for h in range(H):
                    z = torch.einsum("id,jd->ij", q[at : at + n, h], k[:, h // each]) / math.sqrt(hs)
                    z[hidden] = -math.inf
                    y[:, h] = torch.softmax(z, 1) @ v[:, h // each]
            out.append(y.reshape(n, H * hs))
            at, b = at + n, b + 1
    return torch.cat(out)


def _exact_mass(case, s):
    H, hs = case["H"], case["hs"]
    each = H // case["Hkv"]
    out = s["mass"].double()
    q, lse = s["q"].double().view(-1, H, hs), s["lse"].double()
    at = 0
    for b, (n, kv) in enumerate(_lens(case)):
        if kv:
            k = _sequence(case, s, b, kv, "k")
            ids = s["table"][b, : -(-kv // case["page"])].long()
            before = s["old"][ids].double().transpose(1, 2).reshape(-1, case["Hkv"])[:kv] * s["decay"]
            before[kv - n :] = 0
            for lo in range(0, n, 1024):
                hi = min(n, lo + 1024)
                hidden = torch.arange(kv, device="cuda")[None, :] > torch.arange(kv - n + lo, kv - n + hi, device="cuda")[:, None]
                for h in range(H):
                    z = torch.einsum("id,jd->ij", q[at + lo : at + hi, h], k[:, h // each]) / math.sqrt(hs)
                    p = torch.exp(z - lse[at + lo : at + hi, h, None])
                    p[hidden] = 0
                    before[:, h // each] += p.sum(0)
            for j, i in enumerate(ids.tolist()):
                part = before[j * case["page"] : (j + 1) * case["page"]]
                out[i, :, : part.shape[0]] = part.T
        at += n
    return out


def _exact_evict(case, s):
    import numpy as np

    budget, recent, page, Hkv = case["budget"], case["recent"], case["page"], case["Hkv"]
    kept = np.full((case["B"], Hkv, budget), -1, dtype=np.int32)
    to = {x: s["to_" + x].double() for x in ("k", "v", "mass")}
    read, lens = {"k": [], "v": []}, []
    for b, (_, kv) in enumerate(_lens(case)):
        first = min(case["first"], kv)
        ids = s["table"][b, : -(-kv // page)].long()
        held = s["mass"][ids].double().transpose(0, 1).reshape(Hkv, -1)[:, :kv]
        host = held.cpu().numpy()
        new = first + min(budget, kv - first)
        lens.append(new)
        rows = np.empty((Hkv, new), dtype=np.int64)
        for h in range(Hkv):
            stay = np.arange(first, kv)
            if stay.size > budget:
                old = stay[: stay.size - recent]
                heavy = old[np.argsort(-host[h, old], kind="stable")[: budget - recent]]
                stay = np.concatenate((np.sort(heavy), stay[stay.size - recent :]))
            kept[b, h, : stay.size] = stay
            rows[h] = np.concatenate((np.arange(first), stay))
        rows = torch.from_numpy(rows).cuda()
        vectors = {x: _sequence(case, s, b, kv, x).transpose(0, 1).gather(1, rows[..., None].expand(-1, -1, case["hs"])) for x in ("k", "v")}
        for x in ("k", "v"):
            read[x].append(vectors[x].transpose(0, 1).reshape(new, -1))
        for j, i in enumerate(s["to_table"][b, : -(-new // page)].tolist()):
            part = slice(j * page, min(new, (j + 1) * page))
            to["mass"][i, :, : part.stop - part.start] = held.gather(1, rows)[:, part]
            for x in ("k", "v"):
                to[x][i, :, : part.stop - part.start] = vectors[x][:, part]
    k, v = (torch.cat(read[x]) if case["q8"] else to[x] for x in ("k", "v"))
    return k, v, to["mass"], np.array(lens, dtype=np.int32), kept


_exact = dict(shared=_exact_shared, mass=_exact_mass, evict=_exact_evict)
