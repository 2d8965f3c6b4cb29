"""hs2_qk_norm_rope with a warp per token (many tokens): every layout with more
heads than a warp takes in a step, so that each of its loops over heads goes
round again.  Bounds as in test_gpu_norm_rope.py."""
import numpy as np
import pytest
import torch

from tests import gpu_harness as H
from tests.test_gpu_norm_rope import _case, _check, _run
from token_level_sparse_causal_b200 import hs2

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    H.ensure_built()
    hs2.hs2_debug_set(H.WAIT_LIMIT_NS, 0)


def _some_rows(x, keep):
    """The case cut to `keep` of its rows: the others' slots as they were before the call."""
    y = dict(x)
    y.update({n: x[n][keep] for n in ("qkv", "pos", "q_out", "slots")}, qb=None)
    rest = np.setdiff1d(np.arange(len(x["pos"])), keep)
    at = x["slots"][rest].long()
    for n, before in (("k", 0), ("v", 0), ("ks", 3.0), ("vs", 3.0)):
        if x[n] is not None:
            y[n] = x[n].clone()
            y[n][at] = before
    return y


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hkv,rot,norm", [(20, 10, 128, True), (17, 17, 64, True), (33, 3, 96, False),
                                             (9, 9, 16, True), (1, 1, 128, False)])
def test_many_tokens_of_many_heads(Hq, Hkv, rot, norm, interleaved, kv8):
    n = 148 * 16 + 5
    x = _case(n, Hq, Hkv, kv8, rot, norm, seed=Hq)
    x["slots"][3] = -1                      # a row without a cache write among the others
    _run(x, Hq, Hkv, interleaved)
    hs2.hs2_sync()
    for b in ("qb", "kb", "vb"):
        assert x[b] is None or H.guards_intact(x[b])
    keep = np.r_[0:24, n - 21:n]
    y = _some_rows(x, keep)
    _check(y, Hq, Hkv, rot, interleaved)
