"""Paged caches and drafted batches for the serving tests: inputs on the CPU,
their fp64 values for the oracle, and their copies on the device."""
import numpy as np
import torch

from oracle import hs2_oracle as orc
from oracle import serving as so
from token_level_sparse_causal_b200 import hs2, inputs


def f64(t):
    return orc.decode_bf16(inputs.as_u16(t))


def random_tree(t, rng):
    rows = []
    for i in range(t):
        parent = int(rng.integers(-1, i)) if i else -1
        rows.append((1 << i) | (rows[parent] if parent >= 0 else 0))
    return rows


class Paged:
    """A paged cache with context lengths `ctx` and drafted counts `drafts`.
    Positions behind each sequence (and unused pages) hold `behind`."""

    def __init__(self, ctx, drafts, Hq, Hkv, kv8=False, page=64, tree=True, seed=0, behind=float("nan"), q_scale=1.5):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.ctx, self.t, self.Hq, self.Hkv, self.page, self.kv8 = list(ctx), list(drafts), Hq, Hkv, page, kv8
        lens = [c + t for c, t in zip(ctx, drafts)]
        B = len(lens)
        self.max_pages = max(1, -(-max(lens) // page)) + 1
        n_pages = self.max_pages * B + 2
        self.table = torch.randperm(n_pages, generator=g)[:self.max_pages * B].view(B, self.max_pages).to(torch.int32)
        shape = (n_pages * page, Hkv, 128)
        k, v = (torch.randn(shape, generator=g).to(torch.bfloat16) for _ in range(2))
        live = np.zeros(shape[0], bool)
        for b, n in enumerate(lens):
            live[so.rows_of(self.table[b], page, n)] = True
        dead = torch.from_numpy(~live)
        self.ks = self.vs = None
        if kv8:
            (k, self.ks), (v, self.vs) = (inputs.quantize_e4m3(x) for x in (k, v))
            if np.isnan(behind):
                k[dead] = 0x7F
                v[dead] = 0x7F
            self.k64, self.v64 = (orc.dequantize(inputs.as_u8(x), s.numpy()) for x, s in ((k, self.ks), (v, self.vs)))
        else:
            k[dead] = behind
            v[dead] = behind
            self.k64, self.v64 = f64(k), f64(v)
        self.k, self.v = k, v
        self.cu = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int64)
        self.n_tok = int(self.cu[-1])
        self.q = (torch.randn((self.n_tok, Hq, 128), generator=g) * q_scale).to(torch.bfloat16)
        self.masks = None
        if tree:
            self.masks = np.array([m for t in drafts for m in random_tree(t, rng)], dtype=np.uint64)

    def device(self, dev):
        self.d = d = {n: None if getattr(self, n) is None else getattr(self, n).to(dev)
                      for n in ("k", "v", "ks", "vs", "table", "q")}
        d["cu"] = torch.tensor(self.cu, dtype=torch.int32, device=dev)
        d["ctx"] = torch.tensor(self.ctx, dtype=torch.int32, device=dev)
        d["mask"] = None if self.masks is None else torch.from_numpy(self.masks.view(np.int64)).to(dev)
        self.cache = hs2.make_cache(d["k"], d["v"], d["table"], self.page, d["ks"], d["vs"])
        self.draft = hs2.make_draft(d["q"], d["cu"], d["ctx"], d["mask"], max(1, max(self.t)))
        self.ws = torch.empty(hs2.tree_attn_workspace_bytes(self.cache, self.draft), dtype=torch.uint8, device=dev)
        return self

    def oracle(self):
        a = (self.table.numpy(), self.page, self.ctx, self.cu, self.masks)
        o, lse = so.tree_attn(f64(self.q), self.k64, self.v64, *a)
        spread, _ = so.tree_attn(f64(self.q), self.k64, np.abs(self.v64), *a)
        return o, lse, spread


def check_o(got, ref, spread, what=""):
    """|o - ref| <= 2^-8 |o| (the result's rounding) + 2^-8 sum w |v| (the rounding of each weight before the
    product) + 2^-12 sum w |v| (fp32 scores and sums): every term is a bound, none is an average."""
    lim = 2.0 ** -8 * (np.abs(ref) + spread) + 2.0 ** -12 * spread + 1e-30
    bad = ~(np.abs(got - ref) <= lim)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / lim):.2f} x bound"


def check_lse(got, ref, what=""):
    """A score is a sum of 128 fp32 products whose magnitudes add up to about 16 after the scale: 128 roundings of
    2^-23 of that are 2.4e-4; the sum of exponentials and its logarithm add 2^-20 relative."""
    assert np.array_equal(np.isneginf(got), np.isneginf(ref)), what
    live = ~np.isneginf(ref)
    err = np.abs(got[live] - ref[live])
    assert (err <= 2.5e-4 + 2.0 ** -20 * np.abs(ref[live])).all(), f"{what}: {err.max()}"
