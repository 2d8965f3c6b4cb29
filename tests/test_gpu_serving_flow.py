"""The serving operators one after another, as a program uses them: prompts
are rotated into a paged cache and attended to, drafted trees are rotated
behind them, attended to and partly accepted, the cache is cut back to the
tokens that collected most weight, and decoding goes on over what is left.
Every step is checked against the fp64 oracle on the values that the step
before left in the cache, with the bounds of the operators' own tests."""
import numpy as np
import pytest
import torch

from oracle import hs2_oracle as orc
from oracle import serving as so
from tests import gpu_harness as H
from tests.serving_cases import check_lse, check_o, f64, random_tree
from token_level_sparse_causal_b200 import hs2, inputs

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    H.ensure_built()
    hs2.hs2_debug_set(H.WAIT_LIMIT_NS, 0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("kv8", [False, True])
def test_prompt_draft_accept_evict_decode(kv8):
    Hq, Hkv, page, keep, recent = 8, 2, 32, 96, 24
    G = Hq // Hkv
    prompt, T = [150, 97, 203], [6, 1, 9]
    B, max_pages = len(prompt), 9
    g = torch.Generator().manual_seed(21)
    rng = np.random.default_rng(21)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)
    wq, wk = 1 + 0.2 * rnd(128), 1 + 0.2 * rnd(128)
    freq = torch.from_numpy(1e4 ** (-np.arange(64) / 64)).to(DEV)
    n_pages = B * max_pages
    table = torch.randperm(n_pages, generator=g).view(B, max_pages).to(torch.int32)
    dt = torch.uint8 if kv8 else torch.bfloat16
    pools = [torch.zeros((n_pages * page, Hkv, 128), dtype=dt, device=DEV) for _ in range(2)]
    scales = [torch.ones((n_pages * page, Hkv), device=DEV) if kv8 else None for _ in range(2)]
    cache = hs2.make_cache(*pools, table.to(DEV), page, *scales)
    acc = torch.zeros((B, Hkv, max_pages * page), device=DEV)

    def slots(starts, counts):
        return i32(np.concatenate([so.rows_of(table[b].numpy(), page, s + n)[s:] for b, (s, n) in
                                   enumerate(zip(starts, counts))] or [[]]).astype(np.int32))

    def cached():
        if kv8:
            return [orc.dequantize(inputs.as_u8(p), s.cpu().numpy()) for p, s in zip(pools, scales)]
        return [f64(p) for p in pools]

    # ---- the prompts: rotated into the cache and, packed, into a cache of their own that the prefill reads
    n = sum(prompt)
    cu = np.concatenate([[0], np.cumsum(prompt)])
    x = rnd(n, Hq + 2 * Hkv, 128)
    q, k, v = x.split((Hq, Hkv, Hkv), 1)
    pos = i32(np.concatenate([np.arange(m) for m in prompt]))
    packed = [torch.zeros((-(-n // 64) * 64, Hkv, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    flat = hs2.make_cache(*packed, None, 64)
    qr, q2 = torch.empty((n, Hq, 128), dtype=torch.bfloat16, device=DEV), None
    hs2.hs2_qk_norm_rope(flat, q, k, v, wq, wk, 1e-6, freq, pos, None, qr)
    q2 = torch.empty_like(qr)
    hs2.hs2_qk_norm_rope(cache, q, k, v, wq, wk, 1e-6, freq, pos, slots([0] * B, prompt), q2)
    o, lse = torch.empty_like(qr), torch.empty((Hq, n), device=DEV)
    kp, vp = packed[0][:n], packed[1][:n]
    hs2.hs2_varlen_attn(hs2.make_varlen(qr, kp, B), qr, kp, vp, i32(cu), None, o, lse)
    hs2.hs2_sync()
    assert torch.equal(qr.view(torch.int16), q2.view(torch.int16))
    ref, rl = so.varlen_attn(f64(qr), f64(kp), f64(vp), cu, cu)
    spread, _ = so.varlen_attn(f64(qr), f64(kp), np.abs(f64(vp)), cu, cu)
    check_o(f64(o), ref, spread, "prompts")
    check_lse(lse.double().cpu().numpy(), rl, "prompts")

    # ---- an observation window: the last 8 prompt tokens as chains over the cache collect weight
    def attend(q, cu_d, ctx, masks, what):
        draft = hs2.make_draft(q, i32(cu_d), i32(ctx), masks, max(1, int(np.diff(cu_d).max())))
        ws = torch.empty(hs2.tree_attn_workspace_bytes(cache, draft), dtype=torch.uint8, device=DEV)
        o, lse = torch.empty_like(q), torch.empty((Hq, q.shape[0]), device=DEV)
        hs2.hs2_tree_attn(cache, draft, q, o, lse, ws)
        hs2.hs2_sync()
        kk, vv = cached()
        m = None if masks is None else masks.cpu().numpy().view(np.uint64)
        args = (table.numpy(), page, ctx, cu_d, m)
        ref, rl = so.tree_attn(f64(q), kk, vv, *args)
        spread, _ = so.tree_attn(f64(q), kk, np.abs(vv), *args)
        check_o(f64(o), ref, spread, what)
        check_lse(lse.double().cpu().numpy(), rl, what)
        return draft, o, lse, args

    def collect(draft, q, lse, args, counted, what):
        before = acc.double().cpu().numpy()
        hs2.hs2_cache_weights(cache, draft, q, lse, counted, acc)
        hs2.hs2_sync()
        want = so.cache_weights(f64(q), cached()[0], *args, lse.double().cpu().numpy(),
                                None if counted is None else counted.cpu().numpy(), before)
        assert (np.abs(acc.double().cpu().numpy() - want) <= 3e-4 * (want - before) + 2.0 ** -22 * want).all(), what

    win = np.concatenate([np.arange(c - 8, c) for c in cu[1:]])
    qw = qr[torch.from_numpy(win).to(DEV)].contiguous()
    draft, ow, lsew, args = attend(qw, [0, 8, 16, 24], [m - 8 for m in prompt], None, "window")
    if not kv8:  # the same rows of the prefill, by the other kernel: each within its bound of one reference
        lim = 2 * (2.0 ** -8 * (np.abs(ref) + spread) + 2.0 ** -12 * spread)
        assert (np.abs(f64(ow) - f64(o)[win]) <= lim[win]).all()
    collect(draft, qw, lsew, args, None, "window")

    # ---- drafted trees behind the prompts
    nt = sum(T)
    cu_d = np.concatenate([[0], np.cumsum(T)])
    masks = torch.from_numpy(np.array([m for t in T for m in random_tree(t, rng)], dtype=np.uint64).view(np.int64)).to(DEV)
    depth = [bin(int(m) & (2 ** 64 - 1)).count("1") - 1 for m in masks.tolist()]
    x = rnd(nt, Hq + 2 * Hkv, 128)
    q, k, v = x.split((Hq, Hkv, Hkv), 1)
    qd = torch.empty((nt, Hq, 128), dtype=torch.bfloat16, device=DEV)
    tpos = i32([prompt[b] + depth[cu_d[b] + i] for b in range(B) for i in range(T[b])])
    hs2.hs2_qk_norm_rope(cache, q, k, v, wq, wk, 1e-6, freq, tpos, slots(prompt, T), qd)
    draft, od, lsed, args = attend(qd, cu_d, prompt, masks, "trees")
    counted = torch.from_numpy((rng.random(nt) < 0.5).astype(np.uint8)).to(DEV)
    collect(draft, qd, lsed, args, counted, "trees")

    # ---- one drafted token is accepted; the cache is cut back to 96 tokens a head
    lens = [m + 1 for m in prompt]
    before, acc0 = [p.clone() for p in pools], acc.cpu().numpy().copy()
    s_before = [None if s is None else s.clone() for s in scales]
    idx, new_len = torch.empty((B, Hkv, keep), dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)
    hs2.hs2_cache_evict(cache, i32(lens), acc, keep, recent, idx, new_len, acc)
    hs2.hs2_sync()
    assert new_len.tolist() == [min(m, keep) for m in lens]
    for b in range(B):
        rows = so.rows_of(table[b].numpy(), page, lens[b])
        for h in range(Hkv):
            kept = so.kept_positions(acc0[b, h], lens[b], keep, recent)
            assert idx[b, h, :len(kept)].tolist() == kept
            for p, old in list(zip(pools, before)) + [(s, o2) for s, o2 in zip(scales, s_before) if s is not None]:
                assert torch.equal(p[rows[:len(kept)], h], old[rows[kept], h])

    # ---- decoding goes on over what is left, at the positions the tokens really have
    x = rnd(B, Hq + 2 * Hkv, 128)
    q, k, v = x.split((Hq, Hkv, Hkv), 1)
    q1 = torch.empty((B, Hq, 128), dtype=torch.bfloat16, device=DEV)
    left = new_len.tolist()
    hs2.hs2_qk_norm_rope(cache, q, k, v, wq, wk, 1e-6, freq, i32(lens), slots(left, [1] * B), q1)
    attend(q1, list(range(B + 1)), left, None, "after the cut")


@pytest.mark.parametrize("kv8", [False, True])
def test_a_captured_decode_step_equals_eager_ones(kv8):
    """Rotation, attention and weights of one token a sequence as one graph, replayed over advancing lengths: bit for
    bit what the calls give one by one, on another stream and over pools of their own."""
    Hq, Hkv, page, max_pages, steps = 16, 2, 64, 8, 6
    lens = [0, 1, 62, 127, 300]
    B = len(lens)
    g = torch.Generator().manual_seed(22)
    table = torch.randperm(B * max_pages, generator=g).view(B, max_pages).to(torch.int32)
    freq = torch.from_numpy(1e4 ** (-np.arange(64) / 64)).to(DEV)
    shape = (B * max_pages * page, Hkv, 128)
    start = [torch.randn(shape, generator=g).to(torch.bfloat16) for _ in range(2)]
    rows = torch.randn((steps, B, Hq + 2 * Hkv, 128), generator=g).to(torch.bfloat16).to(DEV)

    def state():
        s = dict(ks=None, vs=None)
        if kv8:
            (s["k"], s["ks"]), (s["v"], s["vs"]) = ([t.to(DEV) for t in inputs.quantize_e4m3(x)] for x in start)
        else:
            s["k"], s["v"] = (x.to(DEV) for x in start)
        s["cache"] = hs2.make_cache(s["k"], s["v"], table.to(DEV), page, s["ks"], s["vs"])
        s["acc"] = torch.zeros((B, Hkv, max_pages * page), device=DEV)
        s["x"] = torch.zeros((B, Hq + 2 * Hkv, 128), dtype=torch.bfloat16, device=DEV)
        s["q"], s["o"] = (torch.zeros((B, Hq, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        s["lse"] = torch.zeros((Hq, B), device=DEV)
        s["ctx"], s["slots"] = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
        s["draft"] = hs2.make_draft(s["q"], torch.arange(B + 1, dtype=torch.int32, device=DEV), s["ctx"], None, 1)
        s["ws"] = torch.empty(hs2.tree_attn_workspace_bytes(s["cache"], s["draft"]), dtype=torch.uint8, device=DEV)
        return s

    def set_step(s, i):
        at = [n + i for n in lens]
        s["x"].copy_(rows[i])
        s["ctx"].copy_(torch.tensor(at, dtype=torch.int32))
        s["slots"].copy_(torch.tensor([int(table[b, n // page]) * page + n % page for b, n in enumerate(at)],
                                      dtype=torch.int32))

    def step(s, stream=None):
        q, k, v = s["x"].split((Hq, Hkv, Hkv), 1)
        hs2.hs2_qk_norm_rope(s["cache"], q, k, v, None, None, 0.0, freq, s["ctx"], s["slots"], s["q"], stream=stream)
        hs2.hs2_tree_attn(s["cache"], s["draft"], s["q"], s["o"], s["lse"], s["ws"], stream)
        hs2.hs2_cache_weights(s["cache"], s["draft"], s["q"], s["lse"], None, s["acc"], stream)

    eager, captured = state(), state()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    side = torch.cuda.Stream()
    for i in range(steps):
        set_step(captured, i)
        set_step(eager, i)
        torch.cuda.synchronize()
        graph.replay()
        step(eager, side)
        torch.cuda.synchronize()
        hs2.hs2_sync()
        for n in ("q", "o", "lse", "acc", "k", "v", "ks", "vs"):
            if eager[n] is not None:
                assert torch.equal(eager[n].view(torch.uint8), captured[n].view(torch.uint8)), (i, n)
    total = captured["acc"].sum(-1).cpu()
    assert torch.allclose(total, torch.full((B, Hkv), steps * Hq / Hkv), rtol=3e-4)  # a row's weights sum to one
