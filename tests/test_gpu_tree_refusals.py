"""Arguments on the device that hs2_tree_attn and hs2_cache_weights refuse as a
whole: they are reported, and nothing is written."""
import pytest
import torch

from tests import gpu_harness as H
from tests.serving_cases import Paged, check_o, f64
from token_level_sparse_causal_b200 import hs2

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    H.ensure_built()
    hs2.hs2_debug_set(H.WAIT_LIMIT_NS, 0)


def _writes_nothing(c):
    o, ob = H.guarded((c.n_tok, c.Hq, 128), torch.bfloat16, DEV, fill=5.0)
    lse, lb = H.guarded((c.Hq, c.n_tok), torch.float32, DEV, fill=5.0)
    acc, ab = H.guarded((len(c.ctx), c.Hkv, c.max_pages * c.page), torch.float32, DEV, fill=5.0)
    for call in (lambda: hs2.hs2_tree_attn(c.cache, c.draft, c.d["q"], o, lse, c.ws),
                 lambda: hs2.hs2_cache_weights(c.cache, c.draft, c.d["q"], torch.zeros_like(lse), None, acc)):
        call()
        with pytest.raises(hs2.Hs2Error) as e:
            hs2.hs2_sync()
        assert e.value.code == hs2.HS2_ERR_INDEX
    assert (o == 5).all() and (lse == 5).all() and (acc == 5).all()
    assert all(H.guards_intact(b) for b in (ob, lb, ab))


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("cu", [
    [0, 6, 3, 8, 10], [-1, 2, 4, 8, 10], [0, 2, 4, 8, 11], [0, 12, 3, 4, 10], [0, 3, 2 ** 31 - 1, 9, 10],
    [0, 3, -2 ** 31, 9, 10], [10, 8, 6, 4, 2],
])
def test_a_cu_draft_that_is_no_split_of_the_rows(cu, kv8):
    c = Paged([130, 61, 40, 7], [3, 5, 0, 2], 8, 2, kv8, 64, True, seed=70).device(DEV)
    ref, rl, spread = c.oracle()
    good = c.d["cu"].clone()
    c.d["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
    _writes_nothing(c)
    c.d["cu"].copy_(good)
    o = torch.empty_like(c.d["q"])
    hs2.hs2_tree_attn(c.cache, c.draft, c.d["q"], o, None, c.ws)
    hs2.hs2_sync()
    check_o(f64(o), ref, spread)


def test_one_bad_entry_behind_the_first_32_sequences():
    c = Paged([i % 200 for i in range(100)], [1] * 100, 4, 1, False, 16, False, seed=71).device(DEV)
    c.d["cu"][70] = 68
    _writes_nothing(c)


def test_more_work_than_a_call_takes():
    """4096 sequences of 2^20 - 1 tokens (one page, named over and over) and a drafted one, for 64 heads: 2^31 tiles,
    and three more a unit."""
    B, H_, pages = 4096, 64, 1 << 13
    k = torch.zeros((128, H_, 128), dtype=torch.bfloat16, device=DEV)
    cache = hs2.make_cache(k, k, torch.zeros((B, pages), dtype=torch.int32, device=DEV), 128)
    q = torch.zeros((B, H_, 128), dtype=torch.bfloat16, device=DEV)
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    draft = hs2.make_draft(q, cu, torch.full((B,), 128 * pages - 1, dtype=torch.int32, device=DEV), None, 1)
    assert B * H_ * (pages + 3) == 2 ** 31 + 3 * 2 ** 18
    o = torch.full_like(q, 5.0)
    lse = torch.full((H_, B), 5.0, device=DEV)
    ws = torch.empty(hs2.tree_attn_workspace_bytes(cache, draft), dtype=torch.uint8, device=DEV)
    hs2.hs2_tree_attn(cache, draft, q, o, lse, ws)
    with pytest.raises(hs2.Hs2Error) as e:
        hs2.hs2_sync()
    assert e.value.code == hs2.HS2_ERR_INDEX
    assert (o == 5).all() and (lse == 5).all()
