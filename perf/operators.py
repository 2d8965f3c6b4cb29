"""Measured cases of the serving operators around the shared K/V cache.

A prompt or a drafted token goes through five of them: the per-head norms of
its query and key with the position rotation, written into the paged cache
(hs2_qk_norm_rope); causal attention over a batch of packed prompts
(hs2_varlen_attn); attention of a tree of drafted tokens over the paged cache
(hs2_tree_attn); the attention weight that each cached token collects
(hs2_cache_weights); and the eviction of the tokens that collected least
(hs2_cache_evict).

With `own` false, `run` computes each in its plain form (elementary torch
operations in 32 bits, angles in 64, rounded once at the end); with `own` true
it makes the calls a user makes.  `exact` evaluates the definitions in 64 bits.
"""
import math
import random

import torch

own = False

D = 128          # head dimension of every layout here
E4M3_MAX = 448.0
SCALE = 1.0 / math.sqrt(D)


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step of a batch: 32 new tokens, latency counts
        dict(name="rope_decode_32", op="rope", n=32, Hq=32, Hkv=8, cache="bf16", page=64, weights=True,
             interleaved=False, far=131072),
        # a prompt chunk of a long context written to an 8-bit cache
        dict(name="rope_chunk_32768_e4m3", op="rope", n=32768, Hq=64, Hkv=8, cache="e4m3", page=64, weights=True,
             interleaved=False, far=1048576),
        # a handful of short prompts, one of them a single token
        dict(name="varlen_short", op="varlen", seqs=7, shortest=1, longest=333, Hq=4, Hkv=1, prefix=0, lens=5),
        # an ordinary serving batch: prompts from tens to thousands of tokens
        dict(name="varlen_mixed", op="varlen", seqs=32, shortest=20, longest=4096, Hq=32, Hkv=8, prefix=0, lens=2),
        # long prompts, each continued after a prefix whose keys are there already
        dict(name="varlen_long_prefix", op="varlen", seqs=2, shortest=12001, longest=16384, Hq=64, Hkv=8, prefix=2048,
             lens=3),
        # plain decode of one sequence: the smallest call
        dict(name="tree_one_token", op="tree", seqs=1, longest=2048, shortest=2048, draft=1, tree=False, Hq=4, Hkv=1,
             cache="bf16", page=16, lens=4),
        # drafted trees of up to 16 tokens for a batch of ordinary contexts
        dict(name="tree_batch", op="tree", seqs=16, longest=8192, shortest=300, draft=16, tree=True, Hq=32, Hkv=8,
             cache="bf16", page=64, lens=5),
        # the same over long contexts in an 8-bit cache
        dict(name="tree_long_e4m3", op="tree", seqs=4, longest=131072, shortest=30000, draft=16, tree=True, Hq=64,
             Hkv=8, cache="e4m3", page=64, lens=6),
        # weights collected from the accepted tokens of a decode step
        dict(name="weights_batch", op="weights", seqs=16, longest=8192, shortest=300, draft=16, tree=True, Hq=32,
             Hkv=8, cache="bf16", page=32, lens=7),
        # weights of an observation window at the end of a long prompt
        dict(name="weights_long_e4m3", op="weights", seqs=2, longest=131072, shortest=90000, draft=32, tree=False,
             Hq=64, Hkv=8, cache="e4m3", page=128, lens=8),
        # a batch cut back to the 1024 + 128 tokens that the sparse layers use
        dict(name="evict_batch", op="evict", seqs=16, longest=8192, shortest=600, Hkv=8, keep=1152, recent=128,
             cache="bf16", page=64, lens=9),
        # a long 8-bit cache cut to a sixteenth
        dict(name="evict_long_e4m3", op="evict", seqs=2, longest=131072, shortest=120001, Hkv=8, keep=8192, recent=128,
             cache="e4m3", page=64, lens=10),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "varlen", "tree", "weights", "evict"))
    Hq, Hkv = rng.choice(((4, 1), (32, 8), (64, 8), (32, 4), (8, 2), (16, 8)))
    cache, page, lens = rng.choice(("bf16", "e4m3")), rng.choice((16, 32, 64, 128)), rng.randrange(1000)
    if op == "rope":
        return dict(op=op, n=_log_int(rng, 1, 32768), Hq=Hq, Hkv=Hkv, cache=cache, page=page,
                    weights=rng.random() < 0.8, interleaved=rng.random() < 0.4, far=_log_int(rng, 2048, 1 << 20))
    if op == "varlen":
        longest = _log_int(rng, 40, 12000)
        seqs = _log_int(rng, 1, max(1, min(48, 60000 // longest)))
        if seqs * longest * longest * Hq > 2.5e10:
            seqs = max(1, int(2.5e10 / (longest * longest * Hq)))
        return dict(op=op, seqs=seqs, shortest=_log_int(rng, 1, longest), longest=longest, Hq=Hq, Hkv=Hkv,
                    prefix=rng.choice((0, 0, _log_int(rng, 1, 2000))), lens=lens)
    longest = _log_int(rng, 200, 131072)
    seqs = _log_int(rng, 1, max(1, min(32, 262144 // longest)))
    shortest = _log_int(rng, 1, longest)
    if op == "evict":
        keep = _log_int(rng, 64, min(16384, max(65, longest)))
        return dict(op=op, seqs=seqs, longest=longest, shortest=shortest, Hkv=Hkv, keep=keep,
                    recent=rng.randrange(0, min(257, keep + 1)), cache=cache, page=page, lens=lens)
    return dict(op=op, seqs=seqs, longest=longest, shortest=shortest, draft=_log_int(rng, 1, 32),
                tree=rng.random() < 0.6, Hq=Hq, Hkv=Hkv, cache=cache, page=page, lens=lens)


def _lengths(c):
    """The sequences' lengths: between shortest and longest, spread over the logarithm; the first is the longest."""
    r = random.Random(7919 * c["lens"] + c["seqs"])
    return [c["longest"]] + [_log_int(r, min(c["shortest"], c["longest"]), c["longest"]) for _ in range(c["seqs"] - 1)]


def _drafts(c):
    """Drafted tokens of each sequence, 1 .. draft; the first has the most, and a large batch has one with none."""
    r = random.Random(104729 * c["lens"] + c["seqs"])
    n = [c["draft"]] + [r.randint(max(1, c["draft"] // 2), c["draft"]) for _ in range(c["seqs"] - 1)]
    if c["seqs"] >= 8:
        n[3] = 0
    return n


def work(c):
    """Bytes and operations of one pass that no form of it can do without."""
    row = 2 * D if c.get("cache", "bf16") == "bf16" else D + 4
    if c["op"] == "rope":
        rows_in = c["n"] * (c["Hq"] + 2 * c["Hkv"])
        return {"bytes": 2 * D * rows_in + c["n"] * (2 * D * c["Hq"] + 2 * row * c["Hkv"] + 8) + 4 * D + 4 * D,
                "flops": 8 * D * c["n"] * (c["Hq"] + c["Hkv"])}
    lens = _lengths(c)
    if c["op"] == "varlen":
        pairs = sum(n * (n + 1) // 2 + n * c["prefix"] for n in lens)
        nq, nk = sum(lens), sum(lens) + c["prefix"] * len(lens)
        return {"bytes": 2 * D * (2 * nq * c["Hq"] + 2 * nk * c["Hkv"]) + 4 * nq * c["Hq"],
                "flops": 4 * D * c["Hq"] * pairs}
    if c["op"] == "evict":
        kept = [min(n, c["keep"]) for n in lens]
        moved = sum(k for n, k in zip(lens, kept) if n > c["keep"])
        return {"bytes": c["Hkv"] * (sum(4 * n for n in lens if n > c["keep"]) + moved * (4 * row + 4) + 4 * c["keep"] *
                                     len(lens)), "flops": c["Hkv"] * sum(lens)}
    t = _drafts(c)
    keys = sum(n + k for n, k in zip(lens, t) if k)
    pairs = sum((n + k) * k for n, k in zip(lens, t))
    q = 2 * D * c["Hq"] * sum(t)
    if c["op"] == "tree":
        return {"bytes": 2 * row * c["Hkv"] * keys + 2 * q + (4 * c["Hq"] + 8) * sum(t), "flops": 4 * D * c["Hq"] * pairs}
    return {"bytes": (row + 8) * c["Hkv"] * keys + q + (4 * c["Hq"] + 8) * sum(t), "flops": 2 * D * c["Hq"] * pairs}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _quantize(x):
    """fp32 rows -> (e4m3 values, fp32 scales): scale = amax / 448, 1 for a row of zeros."""
    amax = x.abs().amax(-1)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, E4M3_MAX), torch.ones_like(amax))
    return (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _pool(c, tokens, g):
    """A K and a V pool of `tokens` rows, in the cache's type."""
    out = {}
    for name in ("k", "v"):
        x = torch.randn((tokens, c["Hkv"], D), generator=g, device="cuda", dtype=torch.bfloat16)
        if c["cache"] == "bf16":
            out[name], out[name + "_scale"] = x, None
        else:
            parts = [_quantize(p.float()) for p in x.split(1 << 17)]
            out[name] = torch.cat([p[0].view(torch.uint8) for p in parts])
            out[name + "_scale"] = torch.cat([p[1] for p in parts])
    return out


def _table(c, lens, g):
    """Each sequence's pages, drawn from the pool in random order; one page more than the longest needs."""
    width = -(-max(lens) // c["page"]) + 1
    n_pages = width * c["seqs"] + 3
    order = torch.randperm(n_pages, generator=g, device="cuda")[: width * c["seqs"]]
    return n_pages, order.view(c["seqs"], width).to(torch.int32)


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _tree_masks(c, t, seed):
    """One 64-bit mask per drafted token: itself and its ancestors in a random tree."""
    r, masks = random.Random(seed), []
    for n in t:
        rows = []
        for i in range(n):
            parent = r.randrange(-1, i)
            rows.append((1 << i) | (rows[parent] if parent >= 0 else 0))
        masks += rows
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device="cuda")


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    if c["op"] == "rope":
        n, pages = c["n"], -(-c["n"] // c["page"]) + 2
        s["qkv"] = rnd(n, c["Hq"] + 2 * c["Hkv"], D)
        s["wq"] = s["wk"] = None
        if c["weights"]:
            s["wq"], s["wk"] = 1 + 0.2 * rnd(D), 1 + 0.2 * rnd(D)
        s["inv_freq"] = 1e6 ** (-torch.arange(0, D // 2, device="cuda", dtype=torch.float64) / (D // 2))
        s["pos"] = torch.randint(0, c["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
        s["slots"] = torch.randperm(pages * c["page"], generator=g, device="cuda")[:n].to(torch.int32)
        s["q_out"] = torch.zeros((n, c["Hq"], D), device="cuda", dtype=torch.bfloat16)
        dt = torch.bfloat16 if c["cache"] == "bf16" else torch.uint8
        for name in ("k", "v"):
            s[name] = torch.zeros((pages * c["page"], c["Hkv"], D), device="cuda", dtype=dt)
            s[name + "_scale"] = None if dt == torch.bfloat16 else torch.ones((pages * c["page"], c["Hkv"]), device="cuda")
        return s
    lens = _lengths(c)
    if c["op"] == "varlen":
        s["cu_q"], s["cu_k"] = _cu(lens), _cu([n + c["prefix"] for n in lens])
        nq, nk = sum(lens), sum(lens) + c["prefix"] * len(lens)
        s["q"], s["k"], s["v"] = rnd(nq, c["Hq"], D) * 1.5, rnd(nk, c["Hkv"], D), rnd(nk, c["Hkv"], D)
        s["o"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros((c["Hq"], nq), device="cuda")
        return s
    t = _drafts(c) if c["op"] != "evict" else [0] * c["seqs"]
    n_pages, s["table"] = _table(c, [n + k for n, k in zip(lens, t)], g)
    s.update(_pool(c, n_pages * c["page"], g))
    s["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    width = s["table"].shape[1] * c["page"]
    if c["op"] == "evict":
        # collected weight: a few tokens take most of it, many took almost none
        s["acc"] = torch.rand((c["seqs"], c["Hkv"], width), generator=g, device="cuda").pow(8)
        s["acc_out"] = torch.zeros_like(s["acc"])
        s["idx"] = torch.zeros((c["seqs"], c["Hkv"], c["keep"]), dtype=torch.int32, device="cuda")
        s["new_len"] = torch.zeros(c["seqs"], dtype=torch.int32, device="cuda")
        return s
    s["cu"] = _cu(t)
    s["q"] = rnd(sum(t), c["Hq"], D) * 1.5
    s["mask"] = _tree_masks(c, t, seed) if c["tree"] else None
    if c["op"] == "tree":
        s["o"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros((c["Hq"], sum(t)), device="cuda")
        return s
    # the log-sum that the attention returned for these queries, and which drafted tokens were accepted
    s["lse"] = torch.zeros((c["Hq"], sum(t)), device="cuda")
    s["lse"].copy_(_plain_tree(s)[1])
    s["count"] = (torch.rand(sum(t), generator=g, device="cuda") < 0.7).to(torch.uint8)
    s["acc"] = torch.zeros((c["seqs"], c["Hkv"], width), device="cuda")
    return s


# ------------------------------------------------------------ plain forms --

def _plain_rope(s):
    c, qkv = s["c"], s["qkv"]
    Hq, Hkv = c["Hq"], c["Hkv"]
    x = qkv[:, : Hq + Hkv].float()
    if s["wq"] is not None:
        w = torch.cat([s["wq"].float().expand(Hq, D), s["wk"].float().expand(Hkv, D)])
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    angle = s["pos"].double()[:, None] * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if c["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        x = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : D // 2], x[..., D // 2:]
        x = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    s["q_out"].copy_(x[:, :Hq])
    slots = s["slots"].long()
    for name, rows in (("k", x[:, Hq:]), ("v", qkv[:, Hq + Hkv:].float())):
        if c["cache"] == "bf16":
            s[name][slots] = rows.to(torch.bfloat16)
        else:
            codes, scale = _quantize(rows)
            s[name][slots] = codes.view(torch.uint8)
            s[name + "_scale"][slots] = scale


def _softmax_pv(scores, v):
    """Rows of scores (-inf where masked) times v, and the rows' log-sum; a row of -inf alone gives zeros and -inf."""
    m = scores.amax(-1, keepdim=True)
    p = (scores - m.clamp_min(-3e38)).exp()
    l = p.sum(-1, keepdim=True)
    return (p @ v) / l.clamp_min(1e-30), (m + l.log()).squeeze(-1)


def _plain_varlen(s):
    c, B, G = s["c"], s["c"]["seqs"], s["c"]["Hq"] // s["c"]["Hkv"]
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    top = c["longest"]
    tk = torch.arange(top + c["prefix"], device="cuda")
    at = (ck[:-1, None] + tk).clamp_max(s["k"].shape[0] - 1)
    k, v = (s[x][at].float().permute(0, 2, 3, 1) if x == "k" else s[x][at].float().permute(0, 2, 1, 3) for x in "kv")
    q_of = torch.repeat_interleave(torch.arange(B, device="cuda"), nq, output_size=s["q"].shape[0])
    t_of = torch.arange(s["q"].shape[0], device="cuda") - cq[q_of]
    step = max(1, int(1.5e9 / (B * c["Hq"] * (top + c["prefix"]))))
    q = torch.zeros((B, top, c["Hq"], D), device="cuda")
    q[q_of, t_of] = s["q"].float() * SCALE
    o, lse = torch.empty_like(q), torch.empty((B, top, c["Hq"]), device="cuda")
    for lo in range(0, top, step):  # a piece of the queries at a time, as the scores of all would not fit
        rows = torch.arange(lo, min(top, lo + step), device="cuda")
        n = rows.numel()
        qq = q[:, lo:lo + n].view(B, n, c["Hkv"], G, D).permute(0, 2, 3, 1, 4).reshape(B, c["Hkv"], G * n, D)
        sc = (qq @ k).view(B, c["Hkv"], G, n, -1)
        seen = tk[None, None] <= rows[None, :, None] + (nk - nq)[:, None, None]
        sc = sc.masked_fill_(~seen[:, None, None], -math.inf)
        oo, ll = _softmax_pv(sc.view(B, c["Hkv"], G * n, -1), v)
        o[:, lo:lo + n] = oo.view(B, c["Hkv"], G, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, c["Hq"], D)
        lse[:, lo:lo + n] = ll.view(B, c["Hkv"], G, n).permute(0, 3, 1, 2).reshape(B, n, c["Hq"])
    s["o"].copy_(o[q_of, t_of])
    s["lse"].copy_(lse[q_of, t_of].T)


def _rows_of(s, n):
    """Rows of the pool that hold positions 0 .. n-1 of every sequence."""
    pos = torch.arange(n, device="cuda")
    return s["table"].long()[:, pos // s["c"]["page"]] * s["c"]["page"] + pos % s["c"]["page"]


def _cached(s, name, rows):
    x = s[name][rows]
    if s["c"]["cache"] == "bf16":
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * s[name + "_scale"][rows][..., None]


def _drafted(s):
    """Padded queries [B][Hkv][T * G][d] times 1/sqrt(d), which keys each sees [B][T][keys], and where each lies."""
    c, B, T = s["c"], s["c"]["seqs"], s["c"]["draft"]
    cu, ctx = s["cu"].long(), s["len"].long()
    t_of = cu[1:] - cu[:-1]
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), t_of, output_size=s["q"].shape[0])
    t = torch.arange(s["q"].shape[0], device="cuda") - cu[b]
    q = torch.zeros((B, T, c["Hq"], D), device="cuda")
    q[b, t] = s["q"].float() * SCALE
    q = q.view(B, T, c["Hkv"], -1, D).permute(0, 2, 1, 3, 4).reshape(B, c["Hkv"], -1, D)
    mask = torch.zeros((B, T), dtype=torch.int64, device="cuda")
    mask[b, t] = s["mask"] if s["mask"] is not None else (2 << t) - 1
    j = torch.arange(c["longest"] + T, device="cuda")[None] - ctx[:, None]  # drafted index of each key, < 0: context
    seen = (j < 0)[:, None] | ((j < t_of[:, None])[:, None] & ((mask[:, :, None] >> j.clamp(0, 63)[:, None]) & 1).bool())
    return q, seen & (torch.arange(T, device="cuda")[None] < t_of[:, None])[..., None], b, t


def _plain_tree(s):
    c, B, T = s["c"], s["c"]["seqs"], s["c"]["draft"]
    q, seen, b, t = _drafted(s)
    rows = _rows_of(s, c["longest"] + T)
    sc = q @ _cached(s, "k", rows).permute(0, 2, 3, 1)
    sc = sc.view(B, c["Hkv"], T, -1, sc.shape[-1]).masked_fill_(~seen[:, None, :, None], -math.inf).view(sc.shape)
    o, lse = _softmax_pv(sc, _cached(s, "v", rows).permute(0, 2, 1, 3))
    o = o.view(B, c["Hkv"], T, -1, D).permute(0, 2, 1, 3, 4).reshape(B, T, c["Hq"], D)
    lse = lse.view(B, c["Hkv"], T, -1).permute(0, 2, 1, 3).reshape(B, T, c["Hq"])
    return o[b, t], lse[b, t].T


def _plain_weights(s):
    c, B, T = s["c"], s["c"]["seqs"], s["c"]["draft"]
    q, seen, b, t = _drafted(s)
    counted = torch.zeros((B, T), dtype=torch.bool, device="cuda")
    counted[b, t] = s["count"].bool()
    lse = torch.zeros((B, T, c["Hq"]), device="cuda")
    lse[b, t] = s["lse"].T
    lse = lse.view(B, T, c["Hkv"], -1).permute(0, 2, 1, 3).reshape(B, c["Hkv"], -1, 1)
    sc = q @ _cached(s, "k", _rows_of(s, c["longest"] + T)).permute(0, 2, 3, 1)
    p = (sc - lse).exp().view(B, c["Hkv"], T, -1, sc.shape[-1])
    p = p.masked_fill_(~(seen & counted[..., None])[:, None, :, None], 0.0)
    s["acc"][..., : sc.shape[-1]] += p.sum((2, 3))


def _plain_evict(s):
    c, n = s["c"], s["len"].long()[:, None, None]
    keep, recent = c["keep"], c["recent"]
    j = torch.arange(c["longest"], device="cuda")
    acc = s["acc"][..., : c["longest"]]
    rank = acc.masked_fill(j >= n - recent, -math.inf).sort(dim=-1, descending=True, stable=True).indices
    i = torch.arange(keep, device="cuda")
    old = torch.full((1,), 1 << 30, device="cuda")
    best = torch.where(i < keep - recent, torch.nn.functional.pad(rank, (0, max(0, keep - c["longest"])))[..., :keep], old)
    src = torch.where(i < keep - recent, best, n - keep + i).sort(-1).values
    short = n <= keep  # nothing to evict: every token stays where it is
    src = torch.where(short, torch.where(i < n, i, -1), src)
    s["idx"].copy_(src)
    s["new_len"].copy_(s["len"].clamp_max(keep))
    # entries past a short sequence's end move its first token onto itself
    src, dst = torch.where(src < 0, 0, src), torch.where(short & (i >= n), 0, i)
    page = c["page"]
    table = s["table"].long()[:, None].expand(-1, c["Hkv"], -1)
    row = lambda p: table.gather(-1, p // page) * page + p % page  # noqa: E731
    src_row, dst_row = row(src), row(dst.expand_as(src))
    head = torch.arange(c["Hkv"], device="cuda")[None, :, None]
    for name in ("k", "v", "k_scale", "v_scale"):
        if s[name] is not None:
            s[name][dst_row, head] = s[name][src_row, head]
    s["acc_out"][..., : c["longest"]].masked_fill_(j < n, 0.0)
    s["acc_out"].scatter_(-1, dst.expand_as(src).contiguous(), s["acc"].gather(-1, src))


# -------------------------------------------------------------------- run --

def _values(s, name):
    return s[name] if s["c"]["cache"] == "bf16" else s[name].view(torch.float8_e4m3fn)


def _own_run(s):
    """The library's calls.  What a program keeps between steps (handles, workspace) is made on the first."""
    from token_level_sparse_causal_b200 import hs2

    c = s["c"]
    if c["op"] == "varlen":
        if "plan" not in s:
            s["plan"] = hs2.make_varlen(s["q"], s["k"], c["seqs"])
        hs2.hs2_varlen_attn(s["plan"], s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["o"], s["lse"])
        return
    if "cache" not in s:
        s["cache"] = hs2.make_cache(s["k"], s["v"], s.get("table"), c["page"], s["k_scale"], s["v_scale"])
    if c["op"] == "rope":
        q, k, v = s["qkv"].split((c["Hq"], c["Hkv"], c["Hkv"]), 1)
        hs2.hs2_qk_norm_rope(s["cache"], q, k, v, s["wq"], s["wk"], 1e-6, s["inv_freq"], s["pos"], s["slots"],
                             s["q_out"], interleaved=c["interleaved"])
        return
    if c["op"] == "evict":
        hs2.hs2_cache_evict(s["cache"], s["len"], s["acc"], c["keep"], c["recent"], s["idx"], s["new_len"],
                            s["acc_out"])
        return
    if "draft" not in s:
        s["draft"] = hs2.make_draft(s["q"], s["cu"], s["len"], s["mask"], c["draft"])
        if c["op"] == "tree":
            s["ws"] = torch.empty(hs2.tree_attn_workspace_bytes(s["cache"], s["draft"]), dtype=torch.uint8, device="cuda")
    if c["op"] == "tree":
        hs2.hs2_tree_attn(s["cache"], s["draft"], s["q"], s["o"], s["lse"], s["ws"])
    else:
        hs2.hs2_cache_weights(s["cache"], s["draft"], s["q"], s["lse"], s["count"], s["acc"])


def run(state):
    s, op = state, state["c"]["op"]
    if own:
        _own_run(s)
    elif op == "tree":
        o, lse = _plain_tree(s)
        s["o"].copy_(o)
        s["lse"].copy_(lse)
    else:
        {"rope": _plain_rope, "varlen": _plain_varlen, "weights": _plain_weights, "evict": _plain_evict}[op](s)
    if op == "rope":
        return {"q": s["q_out"], "k": _values(s, "k"), "v": _values(s, "v"), "k_scale": s["k_scale"],
                "v_scale": s["v_scale"]}
    if op in ("varlen", "tree"):
        return {"o": s["o"], "lse": s["lse"]}
    if op == "weights":
        return {"acc": s["acc"]}
    return {"idx": s["idx"], "new_len": s["new_len"], "acc": s["acc_out"], "k": _values(s, "k"), "v": _values(s, "v"),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ------------------------------------------------------------------ exact --

def _decode64(s, name, rows):
    x = s[name].index_select(0, rows)
    if s["c"]["cache"] == "bf16":
        return x.double()
    return x.view(torch.float8_e4m3fn).double() * s[name + "_scale"].index_select(0, rows).double().unsqueeze(-1)


def _exact_rope(s):
    c = s["c"]
    n, half, freq = c["n"], D // 2, s["inv_freq"]
    out = {}
    turn = torch.polar(torch.ones((n, half), dtype=torch.float64, device="cuda"), s["pos"].double().outer(freq))
    for name, lo, hi, w in (("q", 0, c["Hq"], s["wq"]), ("k", c["Hq"], c["Hq"] + c["Hkv"], s["wk"])):
        x = s["qkv"][:, lo:hi].double()
        if w is not None:
            x = x / (torch.linalg.vector_norm(x, dim=-1, keepdim=True).pow(2) / D + 1e-6).sqrt() * w.double()
        z = torch.complex(x[..., 0::2], x[..., 1::2]) if c["interleaved"] else torch.complex(x[..., :half], x[..., half:])
        z = z * turn[:, None]
        out[name] = torch.stack((z.real, z.imag), -1).flatten(-2) if c["interleaved"] else torch.cat((z.real, z.imag), -1)
    out["v"] = s["qkv"][:, c["Hq"] + c["Hkv"]:].double()
    res = {"q": out["q"], "k_scale": None, "v_scale": None}
    for name in ("k", "v"):
        pool = torch.zeros(s[name].shape, dtype=torch.float64, device="cuda")
        if c["cache"] == "bf16":
            pool[s["slots"].long()] = out[name]
        else:
            top = out[name].abs().amax(-1) / E4M3_MAX
            top = torch.where(top == 0, torch.ones_like(top), top)
            scale = torch.ones(pool.shape[:2], dtype=torch.float64, device="cuda")
            scale[s["slots"].long()] = top
            pool[s["slots"].long()] = out[name] / top[..., None]
            res[name + "_scale"] = scale
        res[name] = pool
    return res


def _attend64(q, k, v, hidden):
    """One KV head: q [n][G][d], k, v [m][d], hidden [n][m] -> outputs and log-sums in 64 bits."""
    sc = torch.einsum("ngd,md->gnm", q, k) / math.sqrt(D)
    sc.masked_fill_(hidden, -math.inf)
    lse = sc.logsumexp(-1)
    p = torch.exp(sc - lse.nan_to_num(neginf=0.0)[..., None])
    return torch.einsum("gnm,md->ngd", p, v), lse


def _exact_varlen(s):
    c, G = s["c"], s["c"]["Hq"] // s["c"]["Hkv"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty((c["Hq"], s["q"].shape[0]), dtype=torch.float64, device="cuda")
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(c["seqs"]):
        nk, off = ck[b + 1] - ck[b], (ck[b + 1] - ck[b]) - (cq[b + 1] - cq[b])
        piece = max(1, int(2e8 / (G * nk)))
        for h in range(c["Hkv"]):
            k, v = s["k"][ck[b]:ck[b + 1], h].double(), s["v"][ck[b]:ck[b + 1], h].double()
            for i in range(cq[b], cq[b + 1], piece):
                e = min(cq[b + 1], i + piece)
                last = torch.arange(i - cq[b], e - cq[b], device="cuda") + off
                hidden = torch.arange(nk, device="cuda")[None] > last[:, None]
                hs = slice(h * G, h * G + G)
                o[i:e, hs], lse[hs, i:e] = _attend64(s["q"][i:e, hs].double(), k, v, hidden)
    return {"o": o, "lse": lse}


def _each_sequence(s):
    """(sequence, its drafted rows, rows of the pool, hidden keys [t][keys]) one after another."""
    cu, lens = s["cu"].tolist(), s["len"].tolist()
    for b in range(s["c"]["seqs"]):
        lo, hi = cu[b], cu[b + 1]
        if lo == hi:
            continue
        m = lens[b] + hi - lo
        pages = s["table"][b].long()
        rows = (pages[:, None] * s["c"]["page"] + torch.arange(s["c"]["page"], device="cuda")).flatten()[:m]
        hidden = torch.zeros((hi - lo, m), dtype=torch.bool)
        for i in range(hi - lo):
            bits = (2 << i) - 1 if s["mask"] is None else int(s["mask"][lo + i]) & ((1 << 64) - 1)
            for j in range(hi - lo):
                hidden[i, lens[b] + j] = not bits >> j & 1
        yield b, lo, hi, rows, hidden.cuda()


def _exact_tree(s):
    c, G = s["c"], s["c"]["Hq"] // s["c"]["Hkv"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty((c["Hq"], s["q"].shape[0]), dtype=torch.float64, device="cuda")
    for b, lo, hi, rows, hidden in _each_sequence(s):
        k, v = _decode64(s, "k", rows), _decode64(s, "v", rows)
        for h in range(c["Hkv"]):
            hs = slice(h * G, h * G + G)
            o[lo:hi, hs], lse[hs, lo:hi] = _attend64(s["q"][lo:hi, hs].double(), k[:, h], v[:, h], hidden)
    return {"o": o, "lse": lse}


def _exact_weights(s):
    c, G = s["c"], s["c"]["Hq"] // s["c"]["Hkv"]
    acc = s["acc"].double()
    for b, lo, hi, rows, hidden in _each_sequence(s):
        k, counted = _decode64(s, "k", rows), s["count"][lo:hi].bool()
        for h in range(c["Hkv"]):
            sc = torch.einsum("ngd,md->ngm", s["q"][lo:hi, h * G:h * G + G].double(), k[:, h]) / math.sqrt(D)
            p = torch.exp(sc - s["lse"][h * G:h * G + G, lo:hi].double().T[..., None])
            acc[b, h, : rows.numel()] += p.masked_fill(hidden[:, None], 0.0)[counted].sum((0, 1))
    return {"acc": acc}


def _exact_evict(s):
    """Values only move here: whatever is kept is kept bit for bit."""
    c, lens, page = s["c"], s["len"].tolist(), s["c"]["page"]
    res = {x: None if s[x] is None else s[x].clone() for x in ("k", "v", "k_scale", "v_scale")}
    res["acc"] = s["acc_out"].clone()
    idx = torch.full_like(s["idx"], -1)
    for b, n in enumerate(lens):
        rows = (s["table"][b].long()[:, None] * page + torch.arange(page, device="cuda")).flatten()
        for h in range(c["Hkv"]):
            if n <= c["keep"]:
                idx[b, h, :n] = torch.arange(n, device="cuda")
                res["acc"][b, h, :n] = s["acc"][b, h, :n]
                continue
            weight = s["acc"][b, h, : n - c["recent"]].double().cpu().numpy()
            order = (-weight).argsort(kind="stable")[: c["keep"] - c["recent"]]
            kept = torch.tensor(sorted(order.tolist()) + list(range(n - c["recent"], n)), device="cuda")
            idx[b, h] = kept
            for x in ("k", "v", "k_scale", "v_scale"):
                if res[x] is not None:
                    res[x][rows[: c["keep"]], h] = s[x][rows[kept], h]
            res["acc"][b, h, : c["keep"]] = s["acc"][b, h, kept]
    wide = lambda x: None if res[x] is None else (res[x].view(torch.float8_e4m3fn) if res[x].dtype == torch.uint8 else res[x]).double()  # noqa: E731,E501
    return {"idx": idx, "new_len": torch.tensor([min(n, c["keep"]) for n in lens], dtype=torch.int32, device="cuda"),
            "acc": res["acc"].double(), "k": wide("k"), "v": wide("v"), "k_scale": wide("k_scale"),
            "v_scale": wide("v_scale")}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "varlen": _exact_varlen, "tree": _exact_tree, "weights": _exact_weights,
            "evict": _exact_evict}[case["op"]](s)
