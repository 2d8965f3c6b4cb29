"""hs2_qk_norm_rope (through the C ABI) against the fp64 oracle.

Tolerances, counted before the first run.  A bf16 result is one rounding of
the fp32 value: 2^-8 relative.  An e4m3 code is one rounding of x / scale:
2^-4 relative, or half the subnormal step (2^-10) of a code.  The fp32 value
itself: the norm is a sum of 128 squares, a square root and two products
(about 2^-20 relative, 12 roundings of 2^-24), the angle is off by one fp32
rounding of a turn in [-1/2, 1/2] (2 pi 2^-25 < 2^-22 rad) plus two units of
the sine and cosine, so a rotated value is within 2^-19 of its pair's length.
"""
import numpy as np
import pytest
import torch

from oracle import hs2_oracle as orc
from oracle import serving as so
from tests import gpu_harness as H
from token_level_sparse_causal_b200 import hs2, inputs

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    H.ensure_built()
    hs2.hs2_debug_set(H.WAIT_LIMIT_NS, 0)


def f64(t):
    return orc.decode_bf16(inputs.as_u16(t))


def _case(n, Hq, Hkv, kv8, rot, norm, seed=0, page=16, far=1 << 20):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
    pages = (n + page - 1) // page + 2
    x = dict(qkv=rnd(n, Hq + 2 * Hkv, 128).to(DEV), wq=None, wk=None, pages=pages, page=page)
    if norm:
        x["wq"], x["wk"] = (1 + 0.3 * rnd(128).float()).to(torch.bfloat16).to(DEV), rnd(128).to(DEV)
    x["freq"] = torch.from_numpy(1e6 ** (-np.arange(rot // 2) / (rot // 2))).to(DEV)
    x["pos"] = torch.randint(0, far, (n,), generator=g, dtype=torch.int32).to(DEV)
    x["slots"] = torch.randperm(pages * page, generator=g)[:n].to(torch.int32).to(DEV)
    dt = torch.uint8 if kv8 else torch.bfloat16
    x["k"], x["kb"] = H.guarded((pages * page, Hkv, 128), dt, DEV) if not kv8 else (torch.zeros((pages * page, Hkv, 128), dtype=dt, device=DEV), None)
    x["v"], x["vb"] = H.guarded((pages * page, Hkv, 128), dt, DEV) if not kv8 else (torch.zeros((pages * page, Hkv, 128), dtype=dt, device=DEV), None)
    sc = lambda: torch.full((pages * page, Hkv), 3.0, device=DEV) if kv8 else None
    x["ks"], x["vs"] = sc(), sc()
    x["cache"] = hs2.make_cache(x["k"], x["v"], None, page, x["ks"], x["vs"])
    x["q_out"], x["qb"] = H.guarded((n, Hq, 128), torch.bfloat16, DEV)
    return x


def _check(x, Hq, Hkv, rot, interleaved, eps=1e-6, q_out=None):
    qkv, pos, freq = f64(x["qkv"]), x["pos"].tolist(), x["freq"].cpu().numpy()
    w = lambda t: None if t is None else f64(t)
    ref_q = so.norm_rope(qkv[:, :Hq], pos, freq, w(x["wq"]), eps, interleaved)
    ref_k = so.norm_rope(qkv[:, Hq:Hq + Hkv], pos, freq, w(x["wk"]), eps, interleaved)
    ref_v = qkv[:, Hq + Hkv:]
    slack = lambda r: 2.0 ** -19 * np.abs(r).max(-1, keepdims=True) * np.sqrt(2)
    got_q = f64(x["q_out"] if q_out is None else q_out)
    assert (np.abs(got_q - ref_q) <= 2.0 ** -8 * np.abs(ref_q) + slack(ref_q)).all()
    slots = None if x["slots"] is None else x["slots"].cpu().numpy()
    at = np.arange(len(pos)) if slots is None else slots
    live = at >= 0
    for pool, sc, ref in ((x["k"], x["ks"], ref_k), (x["v"], x["vs"], ref_v)):
        if sc is None:
            got = f64(pool)[at[live]]
            lim = 2.0 ** -8 * np.abs(ref[live]) + slack(ref[live])
            if pool is x["v"]:
                lim = 0 * lim  # values are copied
        else:
            s = sc.cpu().numpy().astype(np.float64)[at[live]]
            amax = np.abs(ref[live]).max(-1)
            assert (np.abs(s - amax / 448) <= 2.0 ** -18 * amax / 448).all()
            got = orc.decode_e4m3(inputs.as_u8(pool))[at[live]] * s[..., None]
            lim = 2.0 ** -4 * np.abs(ref[live]) + 2.0 ** -10 * s[..., None] + slack(ref[live])
        assert (np.abs(got - ref[live]) <= lim).all()
        rest = np.ones(pool.shape[0], bool)
        rest[at[live]] = False
        assert (pool.cpu()[torch.from_numpy(rest)] == 0).all(), "slots of no row are left alone"
        if sc is not None:
            assert (sc.cpu()[torch.from_numpy(rest)] == 3.0).all()
    for b in ("qb", "kb", "vb"):
        if x[b] is not None:
            assert H.guards_intact(x[b])


def _run(x, Hq, Hkv, interleaved=False, eps=1e-6, q_out=None, stream=None):
    q, k, v = x["qkv"].split((Hq, Hkv, Hkv), 1)
    hs2.hs2_qk_norm_rope(x["cache"], q, k, v, x["wq"], x["wk"], eps, x["freq"], x["pos"], x["slots"],
                         x["q_out"] if q_out is None else q_out, interleaved, stream)


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,Hq,Hkv,rot,norm", [
    (1, 4, 1, 128, True), (3, 1, 1, 128, False), (17, 8, 2, 64, True), (50, 5, 5, 96, True), (33, 32, 8, 16, False),
])
def test_matches_oracle(n, Hq, Hkv, rot, norm, interleaved, kv8):
    x = _case(n, Hq, Hkv, kv8, rot, norm, seed=n)
    _run(x, Hq, Hkv, interleaved)
    hs2.hs2_sync()
    _check(x, Hq, Hkv, rot, interleaved)


@pytest.mark.parametrize("kv8", [False, True])
def test_many_tokens_per_cta(kv8):
    """From 16 tokens per SM on a CTA takes eight tokens; the last has fewer."""
    n = 148 * 32 + 3
    x = _case(n, 2, 1, kv8, 128, True, seed=5)
    _run(x, 2, 1)
    hs2.hs2_sync()
    keep = np.r_[0:64, n - 70:n]
    y = dict(x)
    y.update(qkv=x["qkv"][keep], pos=x["pos"][keep], q_out=x["q_out"][keep], slots=x["slots"][keep], qb=None)
    sub = np.setdiff1d(np.arange(n), keep)
    for p in ("k", "v"):
        y[p] = x[p].clone()
        y[p][x["slots"][sub].long()] = 0
    for p in ("ks", "vs"):
        if kv8:
            y[p] = x[p].clone()
            y[p][x["slots"][sub].long()] = 3.0
    _check(y, 2, 1, 128, False)


def test_no_slots_skipped_rows_and_in_place():
    x = _case(9, 4, 2, False, 128, True, seed=6)
    x["slots"] = None
    _run(x, 4, 2)
    hs2.hs2_sync()
    _check(x, 4, 2, 128, False)
    x = _case(9, 4, 2, True, 128, True, seed=7)
    x["slots"][2:5] = -1
    saved = x["qkv"].clone()
    q = x["qkv"][:, :4]
    _run(x, 4, 2, q_out=q)          # in place on the projection's rows
    hs2.hs2_sync()
    q_new = q.clone()
    assert torch.equal(x["qkv"][:, 4:], saved[:, 4:])
    x["qkv"] = saved
    _check(x, 4, 2, 128, False, q_out=q_new)


def test_zero_rows_and_far_positions():
    x = _case(4, 2, 1, True, 128, True, seed=8)
    x["qkv"].zero_()
    _run(x, 2, 1)
    hs2.hs2_sync()
    at = x["slots"].long()
    assert (x["q_out"] == 0).all() and (x["k"][at] & 127 == 0).all() and (x["ks"][at] == 1).all()
    x = _case(4, 2, 1, False, 128, True, seed=9)
    x["pos"] = torch.tensor([0, 2 ** 24 + 1, 2 ** 31 - 1, -7], dtype=torch.int32, device=DEV)
    _run(x, 2, 1)
    hs2.hs2_sync()
    _check(x, 2, 1, 128, False)


def test_bad_slot_is_reported_and_skipped():
    x = _case(5, 2, 1, False, 128, True, seed=10)
    good = x["slots"].clone()
    x["slots"][1] = x["pages"] * x["page"]
    x["slots"][3] = -2
    _run(x, 2, 1)
    with pytest.raises(hs2.Hs2Error) as e:
        hs2.hs2_sync()
    assert e.value.code == hs2.HS2_ERR_INDEX
    x["slots"] = good
    x["slots"][1] = -1
    x["slots"][3] = -1
    _check(x, 2, 1, 128, False)
    hs2.hs2_sync()


def test_other_stream_and_graph():
    x = _case(7, 4, 1, False, 128, True, seed=11)
    st = torch.cuda.Stream()
    _run(x, 4, 1, stream=st)
    hs2.hs2_sync(st)
    _check(x, 4, 1, 128, False)
    x["q_out"].zero_()
    x["k"].zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run(x, 4, 1)
    x["qkv"].copy_(torch.randn_like(x["qkv"].float()).to(torch.bfloat16))
    g.replay()
    torch.cuda.synchronize()
    _check(x, 4, 1, 128, False)


def test_the_written_cache_is_the_one_quantize_kv_writes():
    """Value rows of an e4m3 cache get the scales and codes of hs2_quantize_kv."""
    x = _case(24, 2, 2, True, 128, False, seed=12)
    x["slots"] = None
    _run(x, 2, 2)
    v = x["qkv"][:, 4:].contiguous()
    codes, scale = torch.empty(v.shape, dtype=torch.uint8, device=DEV), torch.empty((24, 2), device=DEV)
    hs2.hs2_quantize_kv(v, codes, scale)
    hs2.hs2_sync()
    assert torch.equal(x["v"][:24], codes) and torch.equal(x["vs"][:24], scale)
