"""The serving calls on streams beside one another.  All inputs and outputs are
made and filled before the first launch, and live until the streams are done, so
that nothing but the calls themselves can write to them."""
import numpy as np
import pytest
import torch

from tests import gpu_harness as H
from tests.serving_cases import Paged, check_lse, check_o, f64
from tests.test_gpu_norm_rope import _case, _check, _run
from tests.test_gpu_varlen import _cu, _inputs
from token_level_sparse_causal_b200 import hs2

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    H.ensure_built()
    hs2.hs2_debug_set(H.WAIT_LIMIT_NS, 0)


def _outputs(c, n):
    out = []
    for _ in range(n):
        o, ob = H.guarded((c.n_tok, c.Hq, 128), torch.bfloat16, DEV, fill=5.0)
        lse, lb = H.guarded((c.Hq, c.n_tok), torch.float32, DEV, fill=5.0)
        out.append((o, lse, ob, lb))
    return out


def _equal(a, b):
    return torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a,
                       b.view(torch.int16) if b.dtype == torch.bfloat16 else b)


@pytest.mark.parametrize("drafts", [[1, 1], [4, 3], [17, 3]])
def test_attention_on_two_streams(drafts):
    """A bf16 and an e4m3 cache, each with its own workspace; every repeat gives the same bits."""
    cs = [Paged([2000 + 100 * i, 50], drafts, 8, 2, bool(i), 64, True, seed=80 + i).device(DEV) for i in range(2)]
    outs = [_outputs(c, 6) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for i in range(6):
        for c, s, out in zip(cs, streams, outs):
            hs2.hs2_tree_attn(c.cache, c.draft, c.d["q"], out[i][0], out[i][1], c.ws, s)
    for s in streams:
        hs2.hs2_sync(s)
    for c, out in zip(cs, outs):
        ref, rl, spread = c.oracle()
        check_o(f64(out[0][0]), ref, spread)
        check_lse(out[0][1].double().cpu().numpy(), rl)
        for o, lse, ob, lb in out:
            assert _equal(o, out[0][0]) and _equal(lse, out[0][1]) and H.guards_intact(ob) and H.guards_intact(lb)


def test_rotation_on_another_stream():
    for kv8 in (False, True):
        x = _case(7, 4, 1, kv8, 128, True, seed=82)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        _run(x, 4, 1, stream=s)
        hs2.hs2_sync(s)
        _check(x, 4, 1, 128, False)


def test_every_call_beside_itself_in_graphs():
    """Two graphs of a rotation, packed prompts, an attention and its weights, on their own data, replayed together
    and again; the second replay's outputs are the first's, and the weights have grown by as much."""
    graphs, streams, keep, grown = [], [], [], []
    for i in range(2):
        x = _case(9, 4, 2, bool(i), 128, True, seed=84 + i)
        c = Paged([700, 90], [5, 3], 8, 2, bool(i), 64, True, seed=86 + i).device(DEV)
        cu = _cu([70, 33, 150])
        q, k, v = (t.to(DEV) for t in _inputs(cu, cu, 8, 2, seed=88 + i))
        cd = torch.tensor(cu, dtype=torch.int32, device=DEV)
        vo, vl = torch.zeros_like(q), torch.zeros((8, q.shape[0]), device=DEV)
        (o, lse, ob, lb), = _outputs(c, 1)
        acc = torch.zeros((2, 2, c.max_pages * 64), device=DEV)
        shape = hs2.make_varlen(q, k, 3)
        torch.cuda.synchronize()
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            _run(x, 4, 2)
            hs2.hs2_varlen_attn(shape, q, k, v, cd, None, vo, vl)
            hs2.hs2_tree_attn(c.cache, c.draft, c.d["q"], o, lse, c.ws)
            hs2.hs2_cache_weights(c.cache, c.draft, c.d["q"], lse, None, acc)
        graphs.append(g)
        streams.append(s)
        keep.append((x, c, q, k, v, cd, vo, vl, o, lse, ob, lb, acc, shape))
    torch.cuda.synchronize()
    first = None
    for _ in range(2):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        for s in streams:
            hs2.hs2_sync(s)
        now = [[t.clone() for t in (x["q_out"], vo, vl, o, lse)] for x, c, q, k, v, cd, vo, vl, o, lse, *_ in keep]
        grown.append([t[-2].clone() for t in keep])
        if first:
            assert all(_equal(a, b) for f, n in zip(first, now) for a, b in zip(f, n))
        first = now
    for once, twice in zip(*grown):
        assert (once > 0).any() and torch.equal(twice, once + once)
    for x, c, q, k, v, cd, vo, vl, o, lse, ob, lb, acc, shape in keep:
        _check(x, 4, 2, 128, False)
        ref, rl, spread = c.oracle()
        check_o(f64(o), ref, spread)
        check_lse(lse.double().cpu().numpy(), rl)
        assert np.isfinite(f64(vo[:253])).all() and H.guards_intact(ob) and H.guards_intact(lb)
