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


def draft(**kw):
    base = dict(n_tok=6, max_draft=4, Hq=8, reserved=0, q_tok_stride=1024, q_head_stride=128, cu_draft=P, ctx_len=P,
                mask=P)
    base.update(kw)
    return hs2.Hs2Draft(**base)


def tree_call(lib, c, d=None, q=P, o=P + 64, lse=P, ws=P, wsb=1 << 30):
    return lib.hs2_tree_attn(ctypes.byref(c), ctypes.byref(d or draft()), vp(q), vp(o), vp(lse), vp(ws), wsb, ST)


def weights_call(lib, c, d=None, q=P, lse=P, counted=P, acc=P, stride=256):
    return lib.hs2_cache_weights(ctypes.byref(c), ctypes.byref(d or draft()), vp(q), vp(lse), vp(counted), vp(acc),
                                 stride, ST)


def varlen_call(lib, q=P, k=P, v=P, cu_q=P, cu_k=P, o=P + 64, lse=P, **kw):
    base = dict(n_seqs=3, total_q=100, total_k=100, Hq=8, Hkv=2, d=128, q_tok_stride=1024, q_head_stride=128,
                kv_tok_stride=256, kv_head_stride=128)
    base.update(kw)
    s = hs2.Hs2Varlen(**base)
    return lib.hs2_varlen_attn(ctypes.byref(s), vp(q), vp(k), vp(v), vp(cu_q), vp(cu_k), vp(o), vp(lse), ST)


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches(lib, kw, code):
    n = ctypes.c_size_t(0)
    for call in (rope_call, evict_call, tree_call, weights_call):
        assert call(lib, cache(**kw)) == code
    assert lib.hs2_tree_attn_workspace(ctypes.byref(cache(**kw)), ctypes.byref(draft()), ctypes.byref(n)) == code


@pytest.mark.parametrize("kw,code", BAD_TABLES)
def test_bad_tables(lib, kw, code):
    for call in (evict_call, tree_call, weights_call):
        assert call(lib, cache(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n_tok=-1), INV), (dict(max_draft=0), INV), (dict(max_draft=65), INV), (dict(Hq=7), INV), (dict(Hq=0), INV),
    (dict(Hq=34, q_tok_stride=34 * 128), UNS), (dict(reserved=1), INV), (dict(cu_draft=None), INV),
    (dict(ctx_len=None), INV), (dict(q_tok_stride=1000), UNS), (dict(q_tok_stride=512), UNS),
    (dict(q_head_stride=0), INV), (dict(cu_draft=P + 2), UNS), (dict(ctx_len=P + 1), UNS), (dict(mask=P + 4), UNS),
])
def test_bad_drafts(lib, kw, code):
    n = ctypes.c_size_t(0)
    assert tree_call(lib, cache(), draft(**kw)) == code
    assert weights_call(lib, cache(), draft(**kw)) == code
    assert lib.hs2_tree_attn_workspace(ctypes.byref(cache()), ctypes.byref(draft(**kw)), ctypes.byref(n)) == code


def test_tree_attn_arguments(lib):
    n = ctypes.c_size_t(0)
    c, d = ctypes.byref(cache()), ctypes.byref(draft())
    assert lib.hs2_tree_attn_workspace(c, d, ctypes.byref(n)) == hs2.HS2_OK and n.value > 0
    assert lib.hs2_tree_attn_workspace(c, d, None) == INV
    for kw, code in ((dict(q=None), INV), (dict(o=None), INV), (dict(ws=None), INV), (dict(wsb=n.value - 1), WSP),
                     (dict(q=MIS), UNS), (dict(o=MIS), UNS), (dict(ws=MIS), UNS), (dict(lse=P + 2), UNS)):
        assert tree_call(lib, cache(), **kw) == code
    assert tree_call(lib, cache(), draft(n_tok=0), q=None, o=None, ws=None) == hs2.HS2_OK


def test_cache_weights_arguments(lib):
    for kw, code in ((dict(q=None), INV), (dict(lse=None), INV), (dict(acc=None), INV), (dict(stride=0), INV),
                     (dict(stride=255), INV), (dict(q=MIS), UNS), (dict(acc=MIS), UNS), (dict(lse=P + 2), UNS)):
        assert weights_call(lib, cache(), **kw) == code
    assert weights_call(lib, cache(), draft(n_tok=0), q=None, lse=None, acc=None) == hs2.HS2_OK


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), INV), (dict(n_seqs=4097), UNS), (dict(total_q=-1), INV), (dict(total_k=-1), INV),
    (dict(Hq=9), INV), (dict(Hkv=0), INV), (dict(Hq=34, q_tok_stride=34 * 128), UNS), (dict(d=64), UNS),
    (dict(q_tok_stride=1004), UNS), (dict(q_tok_stride=512), UNS), (dict(kv_head_stride=64), UNS),
    (dict(kv_tok_stride=-256), INV), (dict(cu_q=None), INV), (dict(q=None), INV), (dict(k=None), INV),
    (dict(v=None), INV), (dict(o=None), INV), (dict(q=MIS), UNS), (dict(k=MIS), UNS), (dict(o=MIS), UNS),
    (dict(lse=P + 1), UNS), (dict(cu_q=P + 2), UNS), (dict(cu_k=P + 2), UNS),
    (dict(total_q=(1 << 31) - 1, Hq=2048, Hkv=128, q_tok_stride=2048 * 128, kv_tok_stride=128 * 128), UNS),
])
def test_bad_packed_prompts(lib, kw, code):
    assert varlen_call(lib, **kw) == code


def test_no_queries_is_no_work(lib):
    assert varlen_call(lib, total_q=0, q=None, o=None) == hs2.HS2_OK


def test_a_failing_tensor_map_launches_nothing(lib):
    """The host-side fault injection of hs2_debug_set covers every call that encodes a descriptor."""
    assert lib.hs2_debug_set(2_000_000_000, hs2.DEBUG_FAIL_TMAP) == hs2.HS2_OK
    try:
        before = hs2.hs2_launch_count()
        for rc in (tree_call(lib, cache()), weights_call(lib, cache()), varlen_call(lib)):
            assert rc == hs2.HS2_ERR_CUDA
        assert hs2.hs2_launch_count() == before
    finally:
        lib.hs2_debug_set(2_000_000_000, 0)


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


def test_evictions_whose_outputs_overlap_inputs(lib):
    far = P + (1 << 20)
    assert evict_call(lib, cache(), lens=P, new=P, acc_out=far) == INV
    assert evict_call(lib, cache(), lens=P + 4, new=P, acc_out=far) == INV
    assert evict_call(lib, cache(), lens=P, new=P + 4, acc_out=far) == INV
    assert evict_call(lib, cache(), acc=P + 1024, acc_out=P) == INV
    assert evict_call(lib, cache(), acc=P, acc_out=P + 1024) == INV


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
