"""hs2_varlen_attn (through the C ABI) against the fp64 oracle; the bounds are
derived in serving_cases.check_o / check_lse."""
import numpy as np
import pytest
import torch

from oracle import serving as so
from tests import gpu_harness as H
from tests.serving_cases import check_lse, check_o, f64
from token_level_sparse_causal_b200 import hs2

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    H.ensure_built()
    hs2.hs2_debug_set(H.WAIT_LIMIT_NS, 0)


def _cu(lens, start=0):
    return [start] + [start + int(x) for x in np.cumsum(lens)]


def _inputs(cu_q, cu_k, Hq, Hkv, seed, pad=3, behind=float("nan")):
    """Packed rows with `pad` tokens of `behind` after the last (and before a late first) sequence."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for cu, h in ((cu_q, Hq), (cu_k, Hkv), (cu_k, Hkv)):
        x = (torch.randn((cu[-1] + pad, h, 128), generator=g) * (1.5 if h == Hq else 1)).to(torch.bfloat16)
        x[cu[-1]:] = behind
        x[:cu[0]] = behind
        out.append(x)
    return out


def _run(q, k, v, cu_q, cu_k, stream=None, with_lse=True):
    qd, kd, vd = (x if x.is_cuda else x.to(DEV) for x in (q, k, v))
    o, ob = H.guarded(tuple(q.shape), torch.bfloat16, DEV, fill=5.0)
    lse, lb = H.guarded((q.shape[1], q.shape[0]), torch.float32, DEV, fill=5.0)
    t = lambda c: None if c is None else torch.tensor(c, dtype=torch.int32, device=DEV)
    shape = hs2.Hs2Varlen(len(cu_q) - 1, q.shape[0], k.shape[0], q.shape[1], k.shape[1], 128, *hs2._strides(o),
                          *hs2._strides(kd))
    hs2.hs2_varlen_attn(shape, qd, kd, vd, t(cu_q), t(cu_k), o, lse if with_lse else None, stream)
    return o, lse, (ob, lb)


def _check(q, k, v, cu_q, cu_k, o, lse, guards=(), seqs=None):
    cu_k = cu_q if cu_k is None else cu_k
    hs2.hs2_sync()
    got, gl = f64(o), lse.double().cpu().numpy()
    q64, k64, v64 = (np.nan_to_num(f64(x)) for x in (q, k, v))
    ref, rl = so.varlen_attn(q64, k64, v64, cu_q, cu_k)
    spread, _ = so.varlen_attn(q64, k64, np.abs(v64), cu_q, cu_k)
    s = slice(cu_q[0], cu_q[-1])
    check_o(got[s], ref[s], spread[s])
    check_lse(gl[:, s], rl[:, s])
    for outside in (slice(0, cu_q[0]), slice(cu_q[-1], None)):
        assert (got[outside] == 5).all() and (gl[:, outside] == 5).all(), "rows of no sequence are left alone"
    assert all(H.guards_intact(b) for b in guards)


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (2, 2), (6, 2), (16, 1), (5, 1), (8, 1)])
@pytest.mark.parametrize("lens", [[1], [130], [0, 1, 2, 0, 31, 64, 65, 0], [127, 128, 129], [300, 7, 0, 150]])
def test_matches_oracle(Hq, Hkv, lens):
    cu = _cu(lens)
    q, k, v = _inputs(cu, cu, Hq, Hkv, seed=sum(lens) + Hq)
    o, lse, gb = _run(q, k, v, cu, None)
    _check(q, k, v, cu, None, o, lse, gb)


@pytest.mark.parametrize("nq,nk", [
    ([1, 1, 1], [128, 129, 1]),          # a single new token after a prefix
    ([17, 40, 3], [200, 40, 515]),       # chunks after prefixes
    ([50, 20, 9], [30, 0, 9]),           # rows that see no key
    ([300], [1]), ([5, 0, 6], [0, 4, 0]),
])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (3, 1)])
def test_other_key_lengths(nq, nk, Hq, Hkv):
    cu_q, cu_k = _cu(nq, start=2), _cu(nk, start=1)
    q, k, v = _inputs(cu_q, cu_k, Hq, Hkv, seed=sum(nk))
    o, lse, gb = _run(q, k, v, cu_q, cu_k)
    _check(q, k, v, cu_q, cu_k, o, lse, gb)


def test_no_keys_at_all():
    cu = [0, 4, 9]
    q = torch.randn(9, 4, 128).to(torch.bfloat16)
    k = torch.zeros(0, 2, 128, dtype=torch.bfloat16)
    o, lse, gb = _run(q, k, k, cu, [0, 0, 0])
    hs2.hs2_sync()
    assert (o == 0).all() and torch.isneginf(lse).all() and all(H.guards_intact(b) for b in gb)


def test_many_sequences_in_every_order():
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 20, 700)]
    lens[5], lens[699] = 400, 333
    cu = _cu(lens)
    q, k, v = _inputs(cu, cu, 4, 1, seed=9)
    o, lse, gb = _run(q, k, v, cu, None)
    _check(q, k, v, cu, None, o, lse, gb)


def test_4096_sequences():
    lens = [1] * 4096
    cu = _cu(lens)
    q, k, v = _inputs(cu, cu, 2, 1, seed=10)
    o, lse, gb = _run(q, k, v, cu, None)
    hs2.hs2_sync()
    # one key: its weight is one, so o is v
    assert torch.equal(o[:4096].cpu(), v[:4096].expand(-1, 2, -1)) and all(H.guards_intact(b) for b in gb)


def test_strided_views_of_one_projection():
    lens, Hq, Hkv = [70, 133], 8, 2
    cu = _cu(lens)
    x = torch.randn(203, Hq + 2 * Hkv, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    q, k, v = x.split((Hq, Hkv, Hkv), 1)
    o_all = torch.full_like(x, 5.0)
    o = o_all[:, :Hq]
    lse = torch.full((Hq, 203), 5.0, device=DEV)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    hs2.hs2_varlen_attn(hs2.make_varlen(q, k, 2), q, k, v, c, None, o, lse)
    _check(q, k, v, cu, None, o, lse)
    assert (o_all[:, Hq:] == 5).all()


def test_without_lse():
    cu = _cu([40, 200])
    q, k, v = _inputs(cu, cu, 4, 2, seed=11)
    o, lse, gb = _run(q, k, v, cu, None, with_lse=False)
    o2, _, _ = _run(q, k, v, cu, None)
    hs2.hs2_sync()
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and (lse == 5).all()
    assert all(H.guards_intact(b) for b in gb)


def test_single_and_paired_tiles_agree():
    """The same prompt alone (single tiles, as SMs are free) and among many (pairs): bit for bit the same."""
    rng = np.random.default_rng(12)
    lens = [500] + [int(x) for x in rng.integers(100, 400, 60)]
    cu = _cu(lens)
    q, k, v = _inputs(cu, cu, 32, 8, seed=12)
    o, lse, gb = _run(q, k, v, cu, None)
    o1, lse1, _ = _run(q[:500].contiguous(), k[:500].contiguous(), v[:500].contiguous(), [0, 500], None)
    hs2.hs2_sync()
    assert torch.equal(o[:500].view(torch.int16), o1.view(torch.int16)) and torch.equal(lse[:, :500], lse1)


def test_long_prompt_equals_kernel_1():
    """One sequence of a multiple of 64: the same attention as hs2_attn_fwd up to the weights' rounding."""
    L, Hq, Hkv = 8192, 8, 2
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.randn((L, h, 128), generator=g, device=DEV, dtype=torch.bfloat16) for h in (Hq, Hkv, Hkv))
    o, lse, _ = _run(q, k, v, [0, L], None)
    s = hs2.make_shape(q, k)
    o2, lse2 = torch.empty_like(q), torch.empty((Hq, L), device=DEV)
    hs2.hs2_attn_fwd(s, q, k, v, None, None, o2, lse2)
    hs2.hs2_sync()
    assert (o.float() - o2.float()).abs().max() <= 2 * H.O_MAX
    assert (lse - lse2).abs().max() <= 5e-4


def test_bad_lengths_are_reported_and_write_nothing():
    q, k, v = _inputs([0, 50], [0, 50], 4, 1, seed=4, pad=0, behind=0.0)
    for cu in ([0, 30, 20, 50], [-1, 10, 20, 50], [0, 10, 20, 51]):
        o, lse, gb = _run(q, k, v, cu, None)
        with pytest.raises(hs2.Hs2Error) as e:
            hs2.hs2_sync()
        assert e.value.code == hs2.HS2_ERR_INDEX
        assert (o == 5).all() and (lse == 5).all()
    hs2.hs2_sync()


def test_stream_graph_and_repeat():
    cu = _cu([90, 257, 4])
    q, k, v = (x.to(DEV) for x in _inputs(cu, cu, 8, 2, seed=5))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        o, lse, gb = _run(q, k, v, cu, None, stream=st)
    hs2.hs2_sync(st)
    _check(q, k, v, cu, None, o, lse, gb)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    shape = hs2.make_varlen(q, k, 3)
    o2, l2 = torch.full_like(q, 5.0), torch.full_like(lse, 5.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs2.hs2_varlen_attn(shape, q, k, v, c, None, o2, l2)
    # other lengths of the same total: the graph reads them from the device
    cu = _cu([300, 1, 50])
    c.copy_(torch.tensor(cu, dtype=torch.int32))
    graph.replay()
    _check(q, k, v, cu, None, o2, l2)
    o3 = o2.clone()
    graph.replay()
    hs2.hs2_sync()
    assert torch.equal(o3.view(torch.int16), o2.view(torch.int16))


def test_a_lost_load_times_out():
    cu = _cu([200, 40])
    q, k, v = _inputs(cu, cu, 4, 1, seed=6)
    hs2.hs2_debug_set(20_000_000, hs2.DEBUG_SKIP_LOADS)
    try:
        _run(q, k, v, cu, None)
        with pytest.raises(hs2.Hs2Error) as e:
            hs2.hs2_sync()
        assert e.value.code == hs2.HS2_ERR_TIMEOUT
    finally:
        hs2.hs2_debug_set(H.WAIT_LIMIT_NS, 0)
    o, lse, gb = _run(q, k, v, cu, None)
    _check(q, k, v, cu, None, o, lse, gb)
