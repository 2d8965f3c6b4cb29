"""Pins of the serving oracle (oracle/serving.py) to something other than
itself: torch's attention with explicit masks, complex rotation, hand-made
cases, brute force."""
import numpy as np
import pytest
import torch

from oracle import serving as so


def _rnd(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_complex_multiplication(interleaved):
    x, pos = _rnd(0, 3, 2, 8), [0, 5, 1 << 20]
    freq = np.array([1.0, 0.1, 0.01, 1e-3])
    y = so.norm_rope(x, pos, freq, interleaved=interleaved)
    z = x[..., 0::2] + 1j * x[..., 1::2] if interleaved else x[..., :4] + 1j * x[..., 4:]
    w = z * np.exp(1j * np.outer(pos, freq))[:, None]
    got = y[..., 0::2] + 1j * y[..., 1::2] if interleaved else y[..., :4] + 1j * y[..., 4:]
    assert np.allclose(got, w, rtol=0, atol=1e-9)
    assert np.array_equal(y[0], x[0])


def test_norm_and_partial_rotation():
    x, w = _rnd(1, 2, 1, 16), 1 + 0.1 * _rnd(2, 16)
    y = so.norm_rope(x, [3, 4], np.array([0.5, 0.25]), w, 1e-5)
    t = torch.nn.functional.rms_norm(torch.from_numpy(x), (16,), torch.from_numpy(w), 1e-5).numpy()
    assert np.allclose(y[..., 4:], t[..., 4:], atol=1e-12)          # not rotated
    assert np.allclose((y ** 2).sum(-1), (t ** 2).sum(-1), atol=1e-12)  # a rotation keeps the length
    assert not np.allclose(y[..., :4], t[..., :4])


def test_varlen_against_sdpa():
    cu_q, cu_k = [0, 3, 3, 10], [0, 5, 7, 11]
    q, k, v = _rnd(3, 12, 4, 16), _rnd(4, 11, 2, 16), _rnd(5, 11, 2, 16)
    o, lse = so.varlen_attn(q, k, v, cu_q, cu_k)
    assert np.isnan(o[10:]).all() and np.isnan(lse[:, 10:]).all()
    for b in (0, 2):
        qs, ks = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        m = torch.ones(nq, nk, dtype=torch.bool).tril(nk - nq)
        t = lambda x, s: torch.from_numpy(x[s]).permute(1, 0, 2)[None]
        ref = torch.nn.functional.scaled_dot_product_attention(t(q, qs), t(k, ks), t(v, ks), attn_mask=m,
                                                               enable_gqa=True)[0].permute(1, 0, 2).numpy()
        live = m.any(1).numpy()
        assert np.allclose(o[qs][live], ref[live], atol=1e-12)
        assert (o[qs][~live] == 0).all() and (lse[:, qs][:, ~live] == -np.inf).all()
    assert (~torch.ones(7, 4, dtype=torch.bool).tril(-3).any(1)).sum() == 3  # the last sequence has rows without a key


def test_tree_chain_equals_causal_and_branches_do_not_mix():
    page, ctx, t = 4, 6, 3
    table = np.array([[5, 2, 0]])
    k, v, q = _rnd(6, 24, 1, 8), _rnd(7, 24, 1, 8), _rnd(8, t, 2, 8)
    at = so.rows_of(table[0], page, ctx + t)
    assert list(at) == [20, 21, 22, 23, 8, 9, 10, 11, 0]
    chain, _ = so.tree_attn(q, k, v, table, page, [ctx], [0, t], None)
    ref, _ = so.varlen_attn(q, k[at], v[at], [0, t], [0, ctx + t])
    assert np.allclose(chain, ref, atol=1e-13)
    # token 2 is a sibling of token 1: changing token 1's key must not move it
    masks = np.array([0b001, 0b011, 0b101], dtype=np.uint64)
    a, _ = so.tree_attn(q, k, v, table, page, [ctx], [0, t], masks)
    k2 = k.copy()
    k2[at[ctx + 1]] += 1
    b, _ = so.tree_attn(q, k2, v, table, page, [ctx], [0, t], masks)
    assert np.array_equal(a[2], b[2]) and not np.allclose(a[1], b[1])
    z, l = so.tree_attn(q, k, v, table, page, [0], [0, t], np.zeros(t, np.uint64))
    assert (z == 0).all() and (l == -np.inf).all()


def test_weights_sum_to_the_counted_rows():
    page, table = 4, np.array([[1, 3, 2]])
    k, v, q = _rnd(9, 16, 2, 8), _rnd(10, 16, 2, 8), _rnd(11, 3, 4, 8)
    args = (table, page, [7], [0, 3], None)
    _, lse = so.tree_attn(q, k, v, *args)
    acc = so.cache_weights(q, k, *args, lse, np.array([1, 0, 1]), np.zeros((1, 2, 12)))
    assert np.allclose(acc.sum(-1), 2 * 2)       # two counted rows, two heads a group, each sums to one
    assert acc[0, 0, 8] > 0 and acc[0, 0, 9] > 0 and (acc[..., 10:] == 0).all()


@pytest.mark.parametrize("n,keep,recent", [(9, 4, 2), (9, 4, 0), (9, 4, 4), (5, 5, 1), (3, 8, 2), (0, 2, 1)])
def test_kept_positions_brute_force(n, keep, recent):
    acc = np.array([1.0, 3.0, 1.0, 0.0, 3.0, 1.0, 2.0, 9.0, 9.0])[:n]
    got = so.kept_positions(acc, n, keep, recent)
    if n <= keep:
        assert got == list(range(n))
        return
    assert got[keep - recent:] == list(range(n - recent, n)) and got == sorted(set(got)) and len(got) == keep
    chosen, rest = got[:keep - recent], [j for j in range(n - recent) if j not in got]
    for c in chosen:
        for r in rest:
            assert acc[c] > acc[r] or (acc[c] == acc[r] and c < r)
