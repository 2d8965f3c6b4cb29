"""hs2_varlen_attn where one CTA does many items of unlike shape one after the
other: items of one tile and of two, with long and short key ranges, and with
none at all, so that its warps are items apart."""
import numpy as np
import pytest
import torch

from tests import gpu_harness as H
from tests.serving_cases import f64
from tests.test_gpu_varlen import _check, _cu, _inputs, _run
from token_level_sparse_causal_b200 import hs2

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    H.ensure_built()
    hs2.hs2_debug_set(H.WAIT_LIMIT_NS, 0)


def _lens(kind, n, rng):
    if kind == "one token, long prefix":
        return [1] * n, [int(x) for x in rng.integers(1, 700, n)]
    if kind == "no keys between others":
        nq = [int(x) for x in rng.integers(1, 9, n)]
        return nq, [0 if i % 3 else m + int(rng.integers(0, 300)) for i, m in enumerate(nq)]
    if kind == "one tile and two":
        nq = [int(rng.choice([1, 9, 17])) for _ in range(n)]
        return nq, [m + int(rng.choice([0, 130, 400])) for m in nq]
    nq = [int(x) for x in rng.integers(1, 40, n)]     # rows that see no key, at the front of a prompt
    return nq, [max(0, m - int(rng.integers(0, 40))) for m in nq]


@pytest.mark.parametrize("kind", ["one token, long prefix", "no keys between others", "one tile and two",
                                  "fewer keys than rows"])
def test_many_items_a_cta(kind):
    rng = np.random.default_rng(len(kind))
    nq, nk = _lens(kind, 260, rng)
    cu_q, cu_k = _cu(nq), _cu(nk)
    q, k, v = _inputs(cu_q, cu_k, 32, 2, seed=60)
    for _ in range(3):
        o, lse, gb = _run(q, k, v, cu_q, cu_k)
        hs2.hs2_sync()
    _check(q, k, v, cu_q, cu_k, o, lse, gb)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(bad):
    cu = _cu([70, 200, 3])
    q, k, v = _inputs(cu, cu, 8, 2, seed=61, pad=0)
    o, lse, _ = _run(q, k, v, cu, None)
    hs2.hs2_sync()
    q[100, 5, 7] = bad
    o2, lse2, gb = _run(q, k, v, cu, None)
    hs2.hs2_sync()
    got, ref = f64(o2), f64(o)
    assert np.isnan(got[100, 5]).all() and torch.isnan(lse2[5, 100])
    got[100, 5], lse2[5, 100] = ref[100, 5], lse[5, 100]
    assert np.array_equal(got, ref) and torch.equal(lse, lse2) and all(H.guards_intact(b) for b in gb)
