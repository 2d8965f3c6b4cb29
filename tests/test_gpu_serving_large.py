"""The serving operators over pools whose byte and element offsets pass 32
bits: the same tokens in a small pool and at the far end of a large one have to
give the same results, bit for bit."""
import numpy as np
import pytest
import torch

from tests import gpu_harness as H
from tests.serving_cases import Paged
from token_level_sparse_causal_b200 import hs2

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    H.ensure_built()
    hs2.hs2_debug_set(H.WAIT_LIMIT_NS, 0)


def _bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("kv8", [False, True])
def test_far_pages_hold_what_near_ones_do(kv8):
    page, Hkv = 64, 2
    c = Paged([700, 61], [3, 5], 8, Hkv, kv8, page, True, seed=20).device(DEV)
    n_small = c.k.shape[0] // page
    tokens = (2 ** 32 + 2 ** 28) // (Hkv * 128 * (1 if kv8 else 2)) // page * page  # 4.25 GiB a pool
    n_big = tokens // page
    where = torch.arange(n_small) * 7 + n_big - 7 * n_small
    where[::3] = torch.arange(n_small)[::3]  # a third of the pages stays at the near end
    rows = (where[:, None] * page + torch.arange(page)).flatten().to(DEV)

    def spread(t):
        if t is None:
            return None
        big = torch.empty((tokens,) + t.shape[1:], dtype=t.dtype, device=DEV)
        big[rows] = t
        return big

    big = {n: spread(c.d[n]) for n in ("k", "v", "ks", "vs")}
    table = where[c.table.long()].to(torch.int32).to(DEV)
    caches = [c.cache, hs2.make_cache(big["k"], big["v"], table, page, big["ks"], big["vs"])]

    got = []
    for cache, to in ((caches[0], None), (caches[1], rows)):
        x = torch.randn((8, 12, 128), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
        q, k, v = x.split((8, Hkv, Hkv), 1)
        near = torch.tensor([5, 64 * (n_small - 1), 64 * 2 + 1, -1, 64 * 4, 64 * 5 + 63, 9, 64 * 7 + 31])
        keep_live = {int(r) for b, n in enumerate((703, 66)) for r in
                     (c.table[b, torch.arange(n) // page].long() * page + torch.arange(n) % page)}
        near = torch.tensor([s if s < 0 or s not in keep_live else -1 for s in near.tolist()])
        slots = near.to(DEV) if to is None else torch.where(near.to(DEV) < 0, -1, to[near.clamp_min(0).to(DEV)])
        freq = torch.from_numpy(1e4 ** (-np.arange(64) / 64)).to(DEV)
        pos = torch.arange(8, dtype=torch.int32, device=DEV) * 1000
        qr = torch.empty_like(c.d["q"])
        hs2.hs2_qk_norm_rope(cache, q, k, v, None, None, 0.0, freq, pos, slots.to(torch.int32), qr)
        o, lse = torch.empty_like(qr), torch.empty((8, 8), device=DEV)
        hs2.hs2_tree_attn(cache, c.draft, c.d["q"], o, lse, c.ws)
        acc = torch.zeros((2, Hkv, c.max_pages * page), device=DEV)
        hs2.hs2_cache_weights(cache, c.draft, c.d["q"], lse, None, acc)
        weights = acc.clone()
        idx, new_len = torch.empty((2, Hkv, 200), dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
        lens = torch.tensor([703, 66], dtype=torch.int32, device=DEV)
        hs2.hs2_cache_evict(cache, lens, acc, 200, 50, idx, new_len, acc)
        hs2.hs2_sync()
        pools = [t if to is None else t[to] for t in ((c.d if to is None else big)[n] for n in ("k", "v", "ks", "vs"))
                 if t is not None]
        got.append([qr, o, lse, weights, idx, new_len, acc] + [t.clone() for t in pools])
    for a, b in zip(*got):
        assert torch.equal(_bits(a), _bits(b))
    assert (got[0][3] > 0).any() and got[0][5].tolist() == [200, 66]
