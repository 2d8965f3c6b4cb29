"""hs2_tree_attn and hs2_cache_weights (through the C ABI) against the fp64
oracle; the bounds of outputs are derived in serving_cases.  A collected
weight is exp(s - lse): an fp32 score (2.5e-4 absolute at most, see check_lse)
and 2^-20 for the exponential and the sum, so 3e-4 relative."""
import numpy as np
import pytest
import torch

from oracle import serving as so
from tests import gpu_harness as H
from tests.serving_cases import Paged, check_lse, check_o, f64
from token_level_sparse_causal_b200 import hs2

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    H.ensure_built()
    hs2.hs2_debug_set(H.WAIT_LIMIT_NS, 0)


def _attend(c, stream=None, with_lse=True):
    o, ob = H.guarded((c.n_tok, c.Hq, 128), torch.bfloat16, DEV, fill=5.0)
    lse, lb = H.guarded((c.Hq, c.n_tok), torch.float32, DEV, fill=5.0)
    hs2.hs2_tree_attn(c.cache, c.draft, c.d["q"], o, lse if with_lse else None, c.ws, stream)
    return o, lse, (ob, lb)


def _check(c, o, lse, guards=()):
    hs2.hs2_sync()
    ref, rl, spread = c.oracle()
    check_o(f64(o), ref, spread)
    check_lse(lse.double().cpu().numpy(), rl)
    assert all(H.guards_intact(b) for b in guards)
    return rl


def _weights(c, lse_ref, counted=None, stride=None, seed=0):
    stride = stride or c.max_pages * c.page
    g = torch.Generator().manual_seed(seed)
    acc0 = torch.rand((len(c.ctx), c.Hkv, stride), generator=g)
    acc, ab = H.guarded(tuple(acc0.shape), torch.float32, DEV)
    acc.copy_(acc0)
    lse = torch.from_numpy(lse_ref).float().to(DEV)
    cnt = None if counted is None else torch.from_numpy(counted).to(DEV)
    hs2.hs2_cache_weights(c.cache, c.draft, c.d["q"], lse, cnt, acc)
    hs2.hs2_sync()
    assert H.guards_intact(ab)
    ref = so.cache_weights(f64(c.q), c.k64, c.table.numpy(), c.page, c.ctx, c.cu, c.masks,
                           lse.double().cpu().numpy(), counted, acc0.double().numpy())
    got = acc.double().cpu().numpy()
    gained = ref - acc0.double().numpy()
    assert (np.abs(got - ref) <= 3e-4 * gained + 2.0 ** -23 * ref).all()
    for b, (n, t) in enumerate(zip(c.ctx, c.t)):
        behind = slice((n + t) if t else 0, None)
        assert np.array_equal(got[b, :, behind], acc0.double().numpy()[b, :, behind])


CASES = [
    # ctx, drafts, Hq, Hkv, page, tree
    ([1], [1], 4, 1, 16, False),
    ([0], [1], 1, 1, 64, False),                           # nothing but itself
    ([127, 128, 129, 5], [1, 1, 1, 1], 8, 2, 64, False),   # plain decoding around a tile's border
    ([300, 0, 77], [5, 3, 7], 8, 1, 16, True),
    ([1000, 64, 200], [16, 0, 9], 16, 2, 128, True),       # a sequence without drafted tokens
    ([250, 120], [64, 33], 8, 4, 32, True),                # drafted keys over a tile's border
    ([500], [64], 16, 1, 64, False),                       # eight tiles of rows
    ([90, 3], [20, 11], 3, 1, 64, True),                   # 42 tokens of 3 heads a tile
    ([4000], [2], 5, 5, 64, True),
    ([700, 30], [32, 20], 2, 1, 64, True),                 # 64 rows: two blocks of a tile
    ([600, 129], [10, 2], 9, 3, 64, True),                 # 30 of 32 rows
    ([260], [21], 3, 1, 16, True),                         # 63 of 64 rows
]


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("ctx,drafts,Hq,Hkv,page,tree", CASES)
def test_matches_oracle(ctx, drafts, Hq, Hkv, page, tree, kv8):
    c = Paged(ctx, drafts, Hq, Hkv, kv8, page, tree, seed=sum(ctx) + Hq).device(DEV)
    o, lse, gb = _attend(c)
    rl = _check(c, o, lse, gb)
    rng = np.random.default_rng(1)
    _weights(c, rl)
    _weights(c, rl, counted=(rng.random(c.n_tok) < 0.6).astype(np.uint8))


@pytest.mark.parametrize("kv8", [False, True])
def test_masks_that_leave_rows_empty_and_bits_behind_the_drafts(kv8):
    c = Paged([0, 140, 0], [4, 6, 1], 8, 2, kv8, 32, True, seed=2)
    c.masks[:4] = [0, 0b0010, 0, 0b0101]
    c.masks[4:10] |= np.uint64(0xFFFFFFFFFFFFFFC0)   # bits of tokens that are not there
    c.masks[10] = 0
    c.device(DEV)
    o, lse, gb = _attend(c)
    rl = _check(c, o, lse, gb)
    assert (o[0] == 0).all() and torch.isneginf(lse[:, 0]).all() and (o[10] == 0).all()
    _weights(c, rl)


def test_many_sequences_of_many_lengths():
    rng = np.random.default_rng(3)
    ctx = [int(x) for x in np.exp(rng.uniform(0, np.log(3000), 60))]
    drafts = [int(x) for x in rng.integers(0, 6, 60)]
    for kv8 in (False, True):
        c = Paged(ctx, drafts, 8, 2, kv8, 16, True, seed=4).device(DEV)
        o, lse, gb = _attend(c)
        rl = _check(c, o, lse, gb)
        _weights(c, rl)


def test_4096_sequences():
    c = Paged([i % 3 for i in range(4096)], [1] * 4096, 2, 1, False, 16, False, seed=5).device(DEV)
    o, lse, gb = _attend(c)
    rl = _check(c, o, lse, gb)
    _weights(c, rl)


@pytest.mark.parametrize("drafts", [1, 4, 7])
def test_many_short_e4m3_sequences(drafts):
    """Units of one to three key tiles, several to a CTA: each role is a unit or more ahead of the next."""
    rng = np.random.default_rng(drafts)
    ctx = [int(x) for x in rng.choice([0, 1, 100, 124, 127, 128, 200, 255, 300], 150)]
    c = Paged(ctx, [drafts] * 150, 16, 2, True, 16, drafts > 1, seed=30 + drafts).device(DEV)
    for _ in range(3):
        o, lse, gb = _attend(c)
        rl = _check(c, o, lse, gb)
    _weights(c, rl)


def test_scales_of_any_size():
    """e4m3 caches whose scales are far from one: V around 1e-6 and 1e4, K that makes the same scores."""
    for f in (1e-6, 1e4):
        c = Paged([700, 90], [4, 2], 8, 1, True, 64, True, seed=6)
        c.vs = c.vs * f
        c.v64 = c.v64 * f
        c.device(DEV)
        o, lse, _ = _attend(c)
        hs2.hs2_sync()
        from oracle import hs2_oracle as orc
        from token_level_sparse_causal_b200 import inputs
        c.v64 = orc.dequantize(inputs.as_u8(c.v), c.vs.numpy())
        ref, _, spread = c.oracle()
        check_o(f64(o), ref, spread)


def test_large_queries_and_sharp_rows():
    """Scores in the hundreds: one key takes all the weight, the others underflow."""
    c = Paged([513, 40], [3, 8], 8, 2, False, 64, True, seed=7, q_scale=60.0).device(DEV)
    o, lse, gb = _attend(c)
    hs2.hs2_sync()
    ref, rl, spread = c.oracle()
    # scores are 40 times those of check_lse's count, and so are their errors; a weight is off by as much
    err = 40 * 2.5e-4
    got = lse.double().cpu().numpy()
    assert (np.abs(got - rl) <= err + 2.0 ** -20 * np.abs(rl)).all()
    lim = 2.0 ** -8 * (np.abs(ref) + spread) + 2 * err * spread + 1e-30
    assert (np.abs(f64(o) - ref) <= lim).all()


def test_strided_pools_and_queries():
    c = Paged([130, 61], [3, 5], 8, 2, False, 64, True, seed=8).device(DEV)
    both = torch.empty(c.k.shape[0], 4, 128, dtype=torch.bfloat16, device=DEV)   # K and V heads side by side
    both[:, :2], both[:, 2:] = c.d["k"], c.d["v"]
    wide = torch.full((c.n_tok, 12, 128), 5.0, dtype=torch.bfloat16, device=DEV)
    wide[:, :8] = c.d["q"]
    q = wide[:, :8]
    cache = hs2.make_cache(both[:, :2], both[:, 2:], c.d["table"], 64)
    draft = hs2.make_draft(q, c.d["cu"], c.d["ctx"], c.d["mask"], 5)
    wide_o = torch.full_like(wide, 5.0)
    lse = torch.empty((8, c.n_tok), device=DEV)
    hs2.hs2_tree_attn(cache, draft, q, wide_o[:, :8], lse, c.ws)
    _check(c, wide_o[:, :8], lse)
    assert (wide_o[:, 8:] == 5).all()


def test_rows_outside_the_sequences_are_left_alone():
    c = Paged([130, 61], [3, 5], 8, 2, False, 64, False, seed=9).device(DEV)
    q = torch.full((c.n_tok + 4, 8, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    q[2:-2] = c.d["q"]
    o, lse = torch.full_like(q, 5.0), torch.full((8, c.n_tok + 4), 5.0, device=DEV)
    draft = hs2.make_draft(q, c.d["cu"] + 2, c.d["ctx"], None, 5)
    hs2.hs2_tree_attn(c.cache, draft, q, o, lse, c.ws)
    hs2.hs2_sync()
    ref, rl, spread = c.oracle()
    check_o(f64(o[2:-2]), ref, spread)
    for edge in (slice(0, 2), slice(-2, None)):
        assert (o[edge] == 5).all() and (lse[:, edge] == 5).all()


def test_without_lse_and_an_e4m3_cache_with_strides():
    c = Paged([300, 41], [3, 5], 8, 2, True, 64, True, seed=16).device(DEV)
    both = torch.zeros(c.k.shape[0], 4, 144, dtype=torch.uint8, device=DEV)   # codes of K and V side by side, padded
    both[:, :2, :128], both[:, 2:, :128] = c.d["k"], c.d["v"]
    cache = hs2.make_cache(both[:, :2, :128], both[:, 2:, :128], c.d["table"], 64, c.d["ks"], c.d["vs"])
    o = torch.full_like(c.d["q"], 5.0)
    hs2.hs2_tree_attn(cache, c.draft, c.d["q"], o, None, c.ws)
    hs2.hs2_sync()
    ref, rl, spread = c.oracle()
    check_o(f64(o), ref, spread)
    acc = torch.zeros((2, 2, c.max_pages * 64), device=DEV)
    hs2.hs2_cache_weights(cache, c.draft, c.d["q"], torch.from_numpy(rl).float().to(DEV), None, acc)
    hs2.hs2_sync()
    assert torch.allclose(acc.sum(-1).double().cpu(), torch.tensor([[12.0, 12.0], [20.0, 20.0]], dtype=torch.float64),
                          rtol=3e-4)                                   # every row of a group sums to one


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("drafts", [3, 20])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(bad, drafts, kv8):
    c = Paged([300, 41], [drafts, 2], 8, 2, kv8, 64, True, seed=40)
    ref, rl, spread = c.oracle()
    c.q[1, 5, 7] = bad
    c.device(DEV)
    o, lse, gb = _attend(c)
    hs2.hs2_sync()
    got, keep = f64(o), np.ones(ref.shape[:2], bool)
    keep[1, 5] = False
    assert np.isnan(got[1, 5]).all() and torch.isnan(lse[5, 1])
    check_o(got[keep], ref[keep], spread[keep])


def test_rows_of_very_different_size():
    """Each query row has a scale of its own: large and small rows, zeros, numbers far below their row's largest."""
    c = Paged([260, 77], [3, 4], 8, 2, True, 64, True, seed=41)
    f = torch.tensor([2.0 ** -100, 2.0 ** -20, 1e-3, 1.0, 3.0, 0.0, 0.5])
    c.q = (c.q.float() * f[:, None, None]).to(torch.bfloat16)
    c.q[3, :, ::2] *= 2.0 ** -12
    c.device(DEV)
    o, lse, gb = _attend(c)
    rl = _check(c, o, lse, gb)
    _weights(c, rl)


def test_more_drafts_than_said_are_reported():
    c = Paged([130, 61], [3, 5], 8, 2, False, 64, True, seed=17).device(DEV)
    ref, rl, spread = c.oracle()
    c.draft = hs2.make_draft(c.d["q"], c.d["cu"], c.d["ctx"], c.d["mask"], 4)
    o, lse, gb = _attend(c)
    with pytest.raises(hs2.Hs2Error) as e:
        hs2.hs2_sync()
    assert e.value.code == hs2.HS2_ERR_INDEX
    check_o(f64(o)[:3], ref[:3], spread[:3])
    assert (o[3:] == 5).all()


def test_sequences_that_share_pages():
    """A common prefix lies in the cache once: two sequences name its pages."""
    c = Paged([256, 256], [2, 3], 8, 2, False, 64, True, seed=18)
    c.table[1, :4] = c.table[0, :4]
    c.device(DEV)
    o, lse, gb = _attend(c)
    rl = _check(c, o, lse, gb)
    _weights(c, rl)


def test_bad_sequences_and_pages_are_reported():
    c = Paged([130, 61, 40], [3, 5, 2], 8, 2, False, 64, True, seed=10).device(DEV)
    ref, rl, spread = c.oracle()
    good_ctx = c.d["ctx"].clone()
    for bad in (-1, c.max_pages * 64 - 4, 2 ** 31 - 1):
        c.d["ctx"][1] = bad
        o, lse, gb = _attend(c)
        acc = torch.zeros((3, 2, c.max_pages * 64), device=DEV)
        with pytest.raises(hs2.Hs2Error) as e:
            hs2.hs2_sync()
        assert e.value.code == hs2.HS2_ERR_INDEX
        hs2.hs2_cache_weights(c.cache, c.draft, c.d["q"], torch.from_numpy(rl).float().to(DEV), None, acc)
        with pytest.raises(hs2.Hs2Error) as e:
            hs2.hs2_sync()
        assert e.value.code == hs2.HS2_ERR_INDEX
        assert (o[3:8] == 5).all() and (acc[1] == 0).all(), "the bad sequence is skipped"
        keep = [0, 1, 2, 8, 9]
        check_o(f64(o)[keep], ref[keep], spread[keep])
        assert (acc[0, :, :133] > 0).all()
    c.d["ctx"].copy_(good_ctx)
    for bad in (-1, c.k.shape[0] // 64):
        table = c.d["table"].clone()
        c.d["table"][0, 0] = bad
        o, lse, gb = _attend(c)
        with pytest.raises(hs2.Hs2Error) as e:
            hs2.hs2_sync()
        assert e.value.code == hs2.HS2_ERR_INDEX
        check_o(f64(o)[3:], ref[3:], spread[3:])
        c.d["table"].copy_(table)
    o, lse, gb = _attend(c)
    _check(c, o, lse, gb)


@pytest.mark.parametrize("kv8", [False, True])
def test_an_acc_shorter_than_a_sequence_is_reported(kv8):
    c = Paged([130, 61, 98], [3, 5, 2], 8, 2, kv8, 64, True, seed=19).device(DEV)
    ref, rl, spread = c.oracle()
    lse = torch.from_numpy(rl).float().to(DEV)
    room = torch.full((3 * 2 * 100 + 256,), 7.0, device=DEV)  # 133 tokens of sequence 0 do not fit, 66 and 100 do
    acc = room[:600].view(3, 2, 100)
    acc.zero_()
    hs2.hs2_cache_weights(c.cache, c.draft, c.d["q"], lse, None, acc)
    with pytest.raises(hs2.Hs2Error) as e:
        hs2.hs2_sync()
    assert e.value.code == hs2.HS2_ERR_INDEX
    assert (room[600:] == 7).all() and (acc[0] == 0).all()
    full = torch.zeros((3, 2, c.max_pages * 64), device=DEV)
    hs2.hs2_cache_weights(c.cache, c.draft, c.d["q"], lse, None, full)
    hs2.hs2_sync()
    assert torch.equal(acc[1:], full[1:, :, :100]) and (full[0, :, :133] > 0).all()


def test_streams_graphs_and_repeats():
    c = Paged([900, 61, 400], [3, 5, 2], 16, 2, False, 64, True, seed=11).device(DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        o, lse, gb = _attend(c, stream=st)
    hs2.hs2_sync(st)
    _check(c, o, lse, gb)
    o2, lse2 = torch.full_like(o, 5.0), torch.full_like(lse, 5.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hs2.hs2_tree_attn(c.cache, c.draft, c.d["q"], o2, lse2, c.ws)
    g.replay()
    hs2.hs2_sync()
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse, lse2)
    # other lengths: the graph reads them from the device
    c.ctx = [200, 300, 959 - 64]
    c.d["ctx"].copy_(torch.tensor(c.ctx, dtype=torch.int32))
    for pool, name in ((c.k, "k"), (c.v, "v")):
        pool.copy_(torch.randn(pool.shape, generator=torch.Generator().manual_seed(12)).to(torch.bfloat16))
        c.d[name].copy_(pool)
    c.k64, c.v64 = f64(c.k), f64(c.v)
    g.replay()
    _check(c, o2, lse2)


def test_two_calls_at_once_with_their_own_workspaces():
    cs = [Paged([2000 + 100 * i, 50], [4, 3], 8, 2, bool(i), 64, True, seed=13 + i).device(DEV) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs = [_attend(c, stream=s) for c, s in zip(cs, streams)]
    for s in streams:
        hs2.hs2_sync(s)
    for c, (o, lse, gb) in zip(cs, outs):
        _check(c, o, lse, gb)


@pytest.mark.parametrize("kv8", [False, True])
def test_a_lost_load_times_out(kv8):
    c = Paged([900, 61], [3, 5], 8, 2, kv8, 64, True, seed=15).device(DEV)
    hs2.hs2_debug_set(20_000_000, hs2.DEBUG_SKIP_LOADS)
    try:
        _attend(c)
        with pytest.raises(hs2.Hs2Error) as e:
            hs2.hs2_sync()
        assert e.value.code == hs2.HS2_ERR_TIMEOUT
        hs2.hs2_cache_weights(c.cache, c.draft, c.d["q"], torch.zeros((8, 8), device=DEV), None,
                              torch.zeros((2, 2, c.max_pages * 64), device=DEV))
        with pytest.raises(hs2.Hs2Error) as e:
            hs2.hs2_sync()
        assert e.value.code == hs2.HS2_ERR_TIMEOUT
    finally:
        hs2.hs2_debug_set(H.WAIT_LIMIT_NS, 0)
    o, lse, gb = _attend(c)
    _check(c, o, lse, gb)


def test_every_e4m3_code_is_converted_exactly():
    """256 sequences of one drafted token each, so its weight is one: o is the value row, exactly, and lse the score.
    Sequence b's value row runs through all codes from b on; its key row is code b everywhere and its query a one
    in one dimension.  The two NaN codes stay NaN."""
    import math
    from oracle import hs2_oracle as orc
    codes = torch.arange(256)
    v = ((codes[:, None] + codes[None, :128]) % 256).to(torch.uint8)
    pool = lambda rows: torch.zeros(256 * 16, 1, 128, dtype=torch.uint8).index_copy_(
        0, 16 * codes, rows.view(256, 1, 128)).to(DEV)
    k = codes.to(torch.uint8).view(256, 1).expand(256, 128).contiguous()
    q = torch.zeros(256, 1, 128, dtype=torch.bfloat16)
    q[codes, 0, codes % 128] = 1
    one = torch.ones(256 * 16, 1, device=DEV)
    cache = hs2.make_cache(pool(k), pool(v), codes.to(torch.int32).view(256, 1).to(DEV), 16, one, one)
    q = q.to(DEV)
    draft = hs2.make_draft(q, torch.arange(257, dtype=torch.int32, device=DEV),
                           torch.zeros(256, dtype=torch.int32, device=DEV), None, 1)
    o, lse = torch.empty_like(q), torch.empty(1, 256, device=DEV)
    ws = torch.empty(hs2.tree_attn_workspace_bytes(cache, draft), dtype=torch.uint8, device=DEV)
    hs2.hs2_tree_attn(cache, draft, q, o, lse, ws)
    hs2.hs2_sync()
    value = orc.decode_e4m3(np.arange(256, dtype=np.uint8))
    finite = np.isfinite(value)
    assert (~finite).sum() == 2
    good = [b for b in range(256) if finite[b]]      # a NaN score leaves no weight to speak of
    assert np.array_equal(f64(o[good, 0]), value[v.numpy()[good]], equal_nan=True)
    # a key of one code adds up 127 zeros and itself: the score is that value times 1/sqrt(128), rounded
    got = lse[0].double().cpu().numpy()
    assert np.isnan(got[~finite]).all() and torch.isnan(o.cpu()[~finite]).all()
    assert (np.abs(got[good] - value[good] / math.sqrt(128)) <= 2.0 ** -20 * np.abs(value[good])).all()
