"""hs2_cache_weights (through the C ABI) with rows that are not finite, against
the fp64 oracle: a counted row's NaN reaches the weights of every key that the
row sees, a row that is left out reaches none.  Finite weights keep the bound
of test_gpu_tree_attn.py (3e-4 relative)."""
import numpy as np
import pytest
import torch

from oracle import serving as so
from tests import gpu_harness as H
from tests.serving_cases import Paged, f64
from token_level_sparse_causal_b200 import hs2

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    H.ensure_built()
    hs2.hs2_debug_set(H.WAIT_LIMIT_NS, 0)


def _collect(c, lse, counted=None):
    """acc (from zeros) of the kernel and of the oracle."""
    acc, ab = H.guarded((len(c.ctx), c.Hkv, c.max_pages * c.page), torch.float32, DEV)
    cnt = None if counted is None else torch.from_numpy(counted).to(DEV)
    hs2.hs2_cache_weights(c.cache, c.draft, c.d["q"], torch.from_numpy(lse).float().to(DEV), cnt, acc)
    hs2.hs2_sync()
    assert H.guards_intact(ab)
    with np.errstate(invalid="ignore", over="ignore"):
        ref = so.cache_weights(f64(c.q), c.k64, c.table.numpy(), c.page, c.ctx, c.cu, c.masks,
                               lse.astype(np.float32).astype(np.float64), counted, np.zeros(acc.shape))
    return acc.double().cpu().numpy(), ref


def _close(got, ref):
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert (np.abs(got[ok] - ref[ok]) <= 3e-4 * ref[ok]).all()


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("Hq,drafts", [(1, 64), (2, 40), (8, 12)])
def test_a_counted_row_that_is_not_finite_reaches_its_keys(Hq, drafts, kv8):
    """In every column of a chunk of 32, by its log-sum and by its query."""
    c = Paged([300, 41], [drafts, 2], Hq, 1, kv8, 64, True, seed=50)
    _, rl, _ = c.oracle()
    c.device(DEV)
    for column in range(34):
        t, h = divmod(column, Hq)
        lse = rl.copy()
        lse[h, t] = np.nan
        got, ref = _collect(c, lse)
        assert np.isnan(ref[0, 0, :300]).all() and not np.isnan(ref[1]).any()
        _close(got, ref)
    for column in range(32):
        t, h = divmod(column, Hq)
        q = c.q.clone()
        c.q[t, h, 7] = float("nan")
        c.d["q"].copy_(c.q)
        _close(*_collect(c, rl))
        c.q = q


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("Hq,drafts", [(1, 64), (2, 5), (8, 12), (16, 33)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_row_that_is_left_out_reaches_no_key(bad, Hq, drafts, kv8):
    """By counted = 0 (its log-sum is NaN then, or finite), or by a log-sum of -inf."""
    c = Paged([300, 41], [drafts, 2], Hq, 1, kv8, 64, True, seed=51)
    _, rl, _ = c.oracle()
    out = [1, drafts - 2]
    for t in out:
        c.q[t, :, 7] = bad
        c.q[t, :, 8] = -bad
    c.device(DEV)
    counted = np.ones(c.n_tok, np.uint8)
    counted[out] = 0
    for lse_of_out in (rl[:, out], np.nan, np.inf):
        lse = rl.copy()
        lse[:, out] = lse_of_out
        got, ref = _collect(c, lse, counted)
        assert np.isfinite(ref).all()
        _close(got, ref)
    lse = rl.copy()
    lse[:, out] = -np.inf
    got, ref = _collect(c, lse)
    assert np.isfinite(ref).all()
    _close(got, ref)


def _outlier(kv8, Hq, drafts, large, small, seed):
    """Queries with one large dimension among small ones, and keys that are small where the queries are large (so
    that the scores stay ordinary ones while the small dimensions decide)."""
    c = Paged([600, 41], [drafts, 2], Hq, 1, kv8, 64, True, seed=seed)
    c.q = (c.q.float() * (small / 1.5)).to(torch.bfloat16)
    c.q[:, :, 7] = large
    if kv8:
        from token_level_sparse_causal_b200 import inputs
        from oracle import hs2_oracle as orc
        k = torch.from_numpy(c.k64).clone()
        k[:, :, 7] *= 2.0 ** -6
        c.k, c.ks = inputs.quantize_e4m3(k.float().nan_to_num().to(torch.bfloat16))
        c.k64 = orc.dequantize(inputs.as_u8(c.k), c.ks.numpy())
    else:
        c.k[:, :, 7] *= 2.0 ** -6
        c.k64 = f64(c.k)
    return c


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("large,small", [(64.0, 0.12), (300.0, 1.5), (1e6, 1.0)])
@pytest.mark.parametrize("Hq,drafts", [(1, 20), (8, 4), (8, 32)])
def test_a_large_dimension_costs_the_small_ones_nothing(Hq, drafts, large, small, kv8):
    """Scores are fp32 sums: 128 roundings of 2^-23 of the products' magnitudes, for a score s beside them 8
    roundings of 2^-24 of |s| and |lse| (scales, the argument, the stored log-sum); an exponential and the sum of
    weights add 2^-17 relative (the polynomial 2.6e-6, ex2 and 64 rows' sums less).  A weight below 2^-125 counts as
    2^-125 (the polynomial's smallest) or as zero, so a position is off by up to 2^-125 a row on top."""
    c = _outlier(kv8, Hq, drafts, large, small, seed=52 + drafts)
    _, rl, _ = c.oracle()
    c.device(DEV)
    lse = torch.zeros((Hq, c.n_tok), device=DEV)
    o = torch.empty_like(c.d["q"])
    hs2.hs2_tree_attn(c.cache, c.draft, c.d["q"], o, lse, c.ws)
    hs2.hs2_sync()
    got_l = lse.double().cpu().numpy()
    got, ref = _collect(c, rl)
    q64 = f64(c.q)
    lim = np.zeros(ref.shape)
    lim_l = np.zeros(rl.shape)
    for b, ctx in enumerate(c.ctx):
        t = c.t[b]
        at = so.rows_of(c.table[b].numpy(), c.page, ctx + t)
        seen = so.draft_seen(ctx, c.masks[c.cu[b]:c.cu[b + 1]], t)
        k = c.k64[at, 0]
        for i in range(t):
            r = c.cu[b] + i
            for h in range(Hq):
                s = k @ q64[r, h] / np.sqrt(128)
                err = 128 * 2.0 ** -23 * (np.abs(k) @ np.abs(q64[r, h])) / np.sqrt(128) \
                    + 8 * 2.0 ** -24 * (np.abs(s) + abs(rl[h, r]))
                p = np.where(seen[i], np.exp(s - rl[h, r]), 0.0)
                lim[b, 0, :ctx + t] += p * (np.expm1(err) + 2.0 ** -17) + 2.0 ** -125
                lim_l[h, r] = (p * err).sum() + 2.0 ** -17
    assert (np.abs(got - ref) <= lim).all(), np.nanmax(np.abs(got - ref) / np.maximum(lim, 1e-300))
    assert (np.abs(got_l - rl) <= lim_l).all(), np.max(np.abs(got_l - rl) / lim_l)
