"""hs2_cache_evict (through the C ABI) against the oracle's stable ranking.
Values only move, so every comparison is exact."""
import numpy as np
import pytest
import torch

from oracle import serving as so
from tests import gpu_harness as H
from token_level_sparse_causal_b200 import hs2

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    H.ensure_built()
    hs2.hs2_debug_set(H.WAIT_LIMIT_NS, 0)


def _case(lens, Hkv, kv8, page, seed, width=None, values="rand"):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    need = -(-max(max(lens), 1) // page)
    max_pages = need + 1 if width is None else -(-width // page)
    n_pages = max_pages * B + 3
    table = torch.randperm(n_pages, generator=g)[:max_pages * B].view(B, max_pages).to(torch.int32)
    shape = (n_pages * page, Hkv, 128)
    if kv8:
        k, v = (torch.randint(0, 256, shape, generator=g, dtype=torch.uint8) for _ in range(2))
        ks, vs = torch.rand(shape[:2], generator=g), torch.rand(shape[:2], generator=g)
    else:
        k, v = (torch.randn(shape, generator=g).to(torch.bfloat16) for _ in range(2))
        ks = vs = None
    acc = torch.rand((B, Hkv, max_pages * page), generator=g)
    if values == "ties":
        acc = (acc * 4).floor() / 4
    elif values == "equal":
        acc = torch.ones_like(acc)
    elif values == "wild":
        acc = (acc - 0.5) * torch.exp(60 * torch.rand(acc.shape, generator=g) - 40)
        acc[..., ::7] = -0.0
        acc[..., 1::7] = 0.0
    return dict(k=k, v=v, ks=ks, vs=vs, table=table, acc=acc, lens=torch.tensor(lens, dtype=torch.int32), page=page)


def _run(x, keep, recent, in_place_acc=False, stream=None):
    d = {n: None if x[n] is None else x[n].clone().to(DEV) for n in ("k", "v", "ks", "vs", "table", "acc", "lens")}
    B, Hkv = x["acc"].shape[:2]
    d["cache"] = hs2.make_cache(d["k"], d["v"], d["table"], x["page"], d["ks"], d["vs"])
    d["idx"], d["ib"] = H.guarded((B, Hkv, keep), torch.int32, DEV, fill=-9)
    d["new_len"] = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    d["acc_out"] = d["acc"] if in_place_acc else torch.full_like(d["acc"], -5.0)
    hs2.hs2_cache_evict(d["cache"], d["lens"], d["acc"], keep, recent, d["idx"], d["new_len"], d["acc_out"], stream)
    return d


def _check(x, d, keep, recent, in_place_acc=False):
    B, Hkv, width = x["acc"].shape
    want = {n: None if x[n] is None else x[n].clone() for n in ("k", "v", "ks", "vs")}
    want_acc = x["acc"].clone() if in_place_acc else torch.full_like(x["acc"], -5.0)
    idx = torch.full((B, Hkv, keep), -1, dtype=torch.int32)
    for b, n in enumerate(x["lens"].tolist()):
        for g in range(Hkv):
            kept = so.kept_positions(x["acc"][b, g].numpy(), n, keep, recent)
            idx[b, g, :len(kept)] = torch.tensor(kept, dtype=torch.int32)
            want_acc[b, g, :n] = 0
            want_acc[b, g, :len(kept)] = x["acc"][b, g, kept]
            src = torch.from_numpy(so.rows_of(x["table"][b], x["page"], n)[kept]) if kept else torch.zeros(0).long()
            dst = torch.from_numpy(so.rows_of(x["table"][b], x["page"], len(kept)))
            for p in ("k", "v", "ks", "vs"):
                if want[p] is not None:
                    want[p][dst, g] = x[p][src, g]
    assert torch.equal(d["idx"].cpu(), idx)
    assert torch.equal(d["new_len"].cpu(), x["lens"].clamp_max(keep))
    assert torch.equal(d["acc_out"].cpu(), want_acc)
    for p in ("k", "v", "ks", "vs"):
        if want[p] is not None:
            assert torch.equal(d[p].cpu().view(torch.uint8), want[p].view(torch.uint8)), p
    assert H.guards_intact(d["ib"])


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("lens,Hkv,page,keep,recent", [
    ([200], 1, 16, 40, 8), ([1, 0, 33, 32], 2, 32, 32, 0), ([300, 77, 500], 3, 64, 76, 76), ([2000, 1999], 2, 128, 1, 1),
    ([2000], 2, 16, 1999, 100), ([700], 1, 64, 1, 0),
])
def test_matches_oracle(lens, Hkv, page, keep, recent, kv8):
    x = _case(lens, Hkv, kv8, page, seed=len(lens) + keep)
    d = _run(x, keep, recent)
    hs2.hs2_sync()
    _check(x, d, keep, recent)


@pytest.mark.parametrize("B,Hkv", [(2, 8), (5, 5), (10, 4), (9, 8), (10, 12)])
def test_clusters_of_every_size(B, Hkv):
    """16 to 120 rows get clusters of 6 down to 1 CTAs."""
    rng = np.random.default_rng(B)
    x = _case([2500] + [int(n) for n in rng.integers(100, 2500, B - 1)], Hkv, bool(B & 1), 32, seed=B, values="ties")
    d = _run(x, 400, 33)
    hs2.hs2_sync()
    _check(x, d, 400, 33)


@pytest.mark.parametrize("kv8", [False, True])
def test_more_rows_than_sms(kv8):
    """Above one row an SM a CTA has fewer threads: 160 rows, every length from none to some hundreds."""
    rng = np.random.default_rng(8)
    x = _case([int(n) for n in rng.integers(0, 400, 40)], 4, kv8, 16, seed=8, values="ties")
    d = _run(x, 150, 20)
    hs2.hs2_sync()
    _check(x, d, 150, 20)


@pytest.mark.parametrize("values", ["ties", "equal", "wild"])
@pytest.mark.parametrize("n,keep,recent", [(4099, 1000, 64), (9000, 4500, 0)])
def test_ties_signs_and_ranges(values, n, keep, recent):
    x = _case([n, 3], 2, False, 64, seed=3, values=values)
    d = _run(x, keep, recent, in_place_acc=True)
    hs2.hs2_sync()
    _check(x, d, keep, recent, in_place_acc=True)


def test_rows_too_long_for_shared_memory():
    """Above 8 x 40960 positions the keys are read from global memory in every pass."""
    n = 8 * 40960 + 999
    x = _case([n], 1, True, 128, seed=4, values="ties")
    d = _run(x, 5000, 128)
    hs2.hs2_sync()
    _check(x, d, 5000, 128)


def test_bad_length_and_bad_page_are_reported():
    x = _case([100, 90], 1, False, 16, seed=5)
    for bad in (-1, x["acc"].shape[2] + 1):
        y = dict(x, lens=torch.tensor([100, bad], dtype=torch.int32))
        d = _run(y, 20, 4)
        with pytest.raises(hs2.Hs2Error) as e:
            hs2.hs2_sync()
        assert e.value.code == hs2.HS2_ERR_INDEX
        assert (d["idx"][1] == -9).all() and d["new_len"].tolist() == [20, -9] and (d["acc_out"][1] == -5).all()
        rows = so.rows_of(x["table"][1], 16, 90)
        assert torch.equal(d["k"].cpu()[rows], x["k"][rows])
    for page_id in (-1, x["k"].shape[0] // 16):
        y = dict(x, table=x["table"].clone())
        y["table"][0, 3] = page_id
        d = _run(y, 20, 4)
        with pytest.raises(hs2.Hs2Error) as e:
            hs2.hs2_sync()
        assert e.value.code == hs2.HS2_ERR_INDEX
        kept = so.kept_positions(x["acc"][0, 0].numpy(), 100, 20, 4)
        assert d["idx"][0, 0].tolist() == kept          # the list does not depend on the pages
        rows = so.rows_of(x["table"][0], 16, 20)
        for i, p in enumerate(kept):
            if p // 16 != 3 and i // 16 != 3:
                assert torch.equal(d["k"].cpu()[rows[i]], x["k"][int(x["table"][0, p // 16]) * 16 + p % 16])
    hs2.hs2_sync()


def test_other_stream_and_graph_replay():
    x = _case([900, 40], 2, False, 64, seed=6)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        d = _run(x, 100, 16, stream=st)
    hs2.hs2_sync(st)
    _check(x, d, 100, 16)
    d = _run(x, 100, 16)                       # warm: buffers for the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hs2.hs2_cache_evict(d["cache"], d["lens"], d["acc"], 100, 16, d["idx"], d["new_len"], d["acc_out"])
    y = _case([900, 40], 2, False, 64, seed=7)
    for n in ("k", "v", "acc", "table"):
        d[n].copy_(y[n])
    d["acc_out"].fill_(-5.0)
    g.replay()
    hs2.hs2_sync()
    _check(y, d, 100, 16)


def test_acc_out_not_wanted():
    x = _case([500, 10], 2, True, 64, seed=9)
    d = {n: None if x[n] is None else x[n].clone().to(DEV) for n in ("k", "v", "ks", "vs", "table", "acc", "lens")}
    cache = hs2.make_cache(d["k"], d["v"], d["table"], 64, d["ks"], d["vs"])
    idx = torch.empty(2, 2, 60, dtype=torch.int32, device=DEV)
    new_len = torch.empty(2, dtype=torch.int32, device=DEV)
    hs2.hs2_cache_evict(cache, d["lens"], d["acc"], 60, 8, idx, new_len)
    hs2.hs2_sync()
    assert torch.equal(d["acc"].cpu(), x["acc"]) and new_len.tolist() == [60, 10]
    for g in range(2):
        assert idx[0, g].tolist() == so.kept_positions(x["acc"][0, g].numpy(), 500, 60, 8)
