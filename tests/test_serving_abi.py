"""Refusals of the serving calls, on the CPU: every call below fails a
host-side check (fake addresses are never dereferenced or launched on)."""
import ctypes

import pytest
import torch

from token_level_sparse_causal_b200 import build, hs2

P = 0x10000        # aligned fake address
MIS = 0x10008      # misaligned for 16-byte accesses
INV, UNS, WSP = hs2.HS2_ERR_INVALID_ARG, hs2.HS2_ERR_UNSUPPORTED, hs2.HS2_ERR_WORKSPACE
ST = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return hs2.lib()


def vp(x):
    return ctypes.c_void_p(x)


def cache(**kw):
    base = dict(Hkv=2, d=128, kv_dtype=0, page=64, n_pages=10, n_seqs=3, max_pages=4, reserved=0, tok_stride=256,
                head_stride=128, k=P, v=P, k_scale=None, v_scale=None, page_table=P)
    base.update(kw)
    return hs2.Hs2Cache(**base)


BAD_CACHES = [
    (dict(d=64), UNS), (dict(page=48), UNS), (dict(page=256), UNS), (dict(page=0), UNS), (dict(Hkv=0), INV),
    (dict(Hkv=257, tok_stride=257 * 128), UNS), (dict(n_pages=0), INV), (dict(n_pages=1 << 25), UNS),
    (dict(kv_dtype=2), INV), (dict(kv_dtype=1), INV), (dict(kv_dtype=1, k_scale=P), INV),
    (dict(kv_dtype=1, k_scale=P + 2, v_scale=P), UNS), (dict(kv_dtype=1, k_scale=P, v_scale=P, tok_stride=264), UNS),
    (dict(k=None), INV), (dict(v=None), INV), (dict(k=MIS), UNS), (dict(tok_stride=128), UNS),
    (dict(tok_stride=260), UNS), (dict(head_stride=64), UNS), (dict(head_stride=-128), INV), (dict(reserved=1), INV),
]
BAD_TABLES = [(dict(page_table=None), INV), (dict(n_seqs=0), INV), (dict(n_seqs=4097), UNS), (dict(max_pages=0), INV),
              (dict(max_pages=1 << 25), UNS), (dict(page_table=P + 2), UNS)]


def rope_call(lib, c, rope=None, q=P, k=P, v=P, wq=P, wk=P, freq=P, pos=P, slots=P, out=P + 64, **kw):
    base = dict(n=4, Hq=8, rot=128, interleaved=0, eps=1e-6, reserved=0, q_tok_stride=12 * 128, q_head_stride=128,
                kv_tok_stride=12 * 128, kv_head_stride=128, out_tok_stride=8 * 128, out_head_stride=128)
    base.update(kw)
    r = hs2.Hs2Rope(**base)
    return lib.hs2_qk_norm_rope(ctypes.byref(c), ctypes.byref(r), vp(q), vp(k), vp(v), vp(wq), vp(wk), vp(freq),
                                vp(pos), vp(slots), vp(out), ST)


def evict_call(lib, c, lens=P, acc=P, acc_out=P + 64, stride=256, keep=32, recent=8, idx=P, new=P + 64):
    return lib.hs2_cache_evict(ctypes.byref(c), vp(lens), vp(acc), vp(acc_out), stride, keep, recent, vp(idx), vp(new),
                               ST)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches(lib, kw, code):
    assert rope_call(lib, cache(**kw)) == code
    assert evict_call(lib, cache(**kw)) == code


@pytest.mark.parametrize("kw,code", BAD_TABLES)
def test_bad_tables(lib, kw, code):
    assert evict_call(lib, cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), INV), (dict(Hq=0), INV), (dict(rot=0), INV), (dict(rot=144), INV), (dict(rot=24), UNS),
    (dict(interleaved=2), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(reserved=5), INV),
    (dict(q_tok_stride=7 * 128), UNS), (dict(q_head_stride=100), UNS), (dict(out_tok_stride=8 * 128 + 4), UNS),
    (dict(kv_tok_stride=0), INV), (dict(kv_head_stride=64), UNS), (dict(q=None), INV), (dict(k=None), INV),
    (dict(v=None), INV), (dict(freq=None), INV), (dict(pos=None), INV), (dict(out=None), INV), (dict(wq=None), INV),
    (dict(wk=None), INV), (dict(q=MIS), UNS), (dict(out=MIS), UNS), (dict(freq=P + 4), UNS), (dict(slots=P + 2), UNS),
    (dict(wq=P + 1), UNS), (dict(out=P), INV),   # in place with other strides
])
def test_bad_rotations(lib, kw, code):
    assert rope_call(lib, cache(), **kw) == code


def test_no_tokens_is_no_work(lib):
    assert rope_call(lib, cache(), n=0) == hs2.HS2_OK


@pytest.mark.parametrize("kw,code", [
    (dict(lens=None), INV), (dict(acc=None), INV), (dict(idx=None), INV), (dict(new=None), INV), (dict(new=P), INV),
    (dict(keep=0), INV), (dict(recent=-1), INV), (dict(recent=33), INV), (dict(stride=0), INV), (dict(stride=254), INV),
    (dict(keep=(1 << 24) + 1), UNS), (dict(acc=MIS), UNS), (dict(acc_out=MIS), UNS), (dict(idx=P + 2), UNS),
])
def test_bad_evictions(lib, kw, code):
    assert evict_call(lib, cache(), **kw) == code


def test_python_checks_name_the_argument():
    k = torch.zeros(128, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="page"):
        hs2.make_cache(k, k, None, 48)
    with pytest.raises(ValueError, match="^v:"):
        hs2.make_cache(k, k[:64], None, 64)
    with pytest.raises(ValueError, match="page_table"):
        hs2.make_cache(k, k, torch.zeros(2, 2), 64)
    with pytest.raises(ValueError, match="scale"):
        hs2.make_cache(k.to(torch.uint8), k.to(torch.uint8), None, 64)
    c = hs2.make_cache(k, k, torch.zeros(2, 2, dtype=torch.int32), 64)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="acc"):
        hs2.hs2_cache_evict(c, i, torch.zeros(2, 3, 128), 4, 1, torch.zeros(2, 2, 4, dtype=torch.int32), i.clone())
    with pytest.raises(ValueError, match="CUDA"):
        hs2.hs2_cache_evict(c, i, torch.zeros(2, 2, 128), 4, 1, torch.zeros(2, 2, 4, dtype=torch.int32), i.clone())
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="positions"):
        hs2.hs2_qk_norm_rope(c, x, x, x, None, None, 0.0, torch.zeros(64, dtype=torch.float64),
                             torch.zeros(4), None, x.clone())
