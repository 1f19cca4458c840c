"""Pins of oracle/decoder_ops_oracle.py (CPU, fp64): gradients against central differences and against
torch's autograd of the same formula, closed forms, and attention against one dense masked softmax."""
import numpy as np
import pytest
import torch

from oracle import decoder_ops_oracle as oo
from oracle import decoder_oracle as do

RNG = np.random.default_rng(7)


def _pos(L, far=0):
    return np.stack([np.arange(L) + far, np.arange(L) // 2 + far, np.arange(L) % 3 + far])


def test_norm_without_rotation_is_rms_norm():
    x, w = RNG.normal(size=(3, 2, 16)), RNG.normal(size=16)
    y = oo.norm_rope(x, w, np.zeros((3, 3)), (2, 3, 3))
    ref = torch.nn.functional.rms_norm(torch.from_numpy(x), (16,), torch.from_numpy(w), eps=1e-6).numpy()
    np.testing.assert_allclose(y, ref, rtol=1e-12)


def test_norm_keeps_the_rotated_norm():
    x = RNG.normal(size=(5, 3, 16))
    y = oo.norm_rope(x, None, _pos(5, 100000), (2, 3, 3), eps=1e-12)
    np.testing.assert_allclose((y ** 2).mean(-1), 1.0, rtol=1e-9)


@pytest.mark.parametrize("far", [0, 90000])
def test_norm_gradient_against_differences(far):
    x, w, dy = RNG.normal(size=(4, 2, 16)), RNG.normal(size=16), RNG.normal(size=(4, 2, 16))
    pos, sec = _pos(4, far), (2, 3, 3)
    dx, dw = oo.norm_rope_grad(dy, x, w, pos, sec)
    f = lambda x_, w_: (dy * oo.norm_rope(x_, w_, pos, sec)).sum()   # noqa: E731
    h = 1e-6
    for i in [(0, 0, 0), (1, 1, 7), (2, 0, 8), (3, 1, 15)]:
        e = np.zeros_like(x)
        e[i] = h
        np.testing.assert_allclose(dx[i], (f(x + e, w) - f(x - e, w)) / (2 * h), rtol=1e-6, atol=1e-8)
    for i in (0, 5, 15):
        e = np.zeros_like(w)
        e[i] = h
        np.testing.assert_allclose(dw[i], (f(x, w + e) - f(x, w - e)) / (2 * h), rtol=1e-6, atol=1e-8)


def test_embed_rows_reduce_to_the_scatter_at_scale_one():
    ids = np.array([1, do.IMAGE_TOKEN_ID, 3, do.VIDEO_TOKEN_ID, 1])
    table, vis = RNG.normal(size=(5, 8)), RNG.normal(size=(2, 8))
    np.testing.assert_array_equal(oo.embed_rows(ids, table, vis, 1.0), do.scatter_tokens(ids, table, vis))
    two = oo.embed_rows(ids, table, vis, 2.0)
    np.testing.assert_array_equal(two[[0, 2, 4]], 2 * table[[1, 3, 1]])
    np.testing.assert_array_equal(two[[1, 3]], vis)


def test_embed_gradient_is_the_transpose():
    ids = np.array([1, do.IMAGE_TOKEN_ID, 3, do.VIDEO_TOKEN_ID, 1, 1])
    table, vis, d = RNG.normal(size=(5, 8)), RNG.normal(size=(2, 8)), RNG.normal(size=(6, 8))
    dt, dv = oo.embed_rows_grad(ids, d, 5, 1.5)
    # the map is linear: <d, rows(table, vision)> = <d_table, table> + <d_vision, vision>
    np.testing.assert_allclose((d * oo.embed_rows(ids, table, vis, 1.5)).sum(), (dt * table).sum() + (dv * vis).sum())
    assert (dt[[0, 2, 4]] == 0).all()


@pytest.mark.parametrize("causal", [True, False])
def test_prefix_attention_is_one_masked_softmax(causal):
    B, H, Hk, D, Lp, cap = 3, 4, 2, 8, 5, 6
    n_q, lens = np.array([2, 1, 4]), np.array([4, 6, 3])      # the last: queries without a visible own key
    cu = np.concatenate([[0], np.cumsum(n_q)])
    q = RNG.normal(size=(cu[-1], H, D))
    pk, pv = RNG.normal(size=(2, Lp, Hk, D))
    k, v = RNG.normal(size=(2, B, cap, Hk, D))
    out, lse = oo.prefix_attention(q, pk, pv, k, v, lens, cu, 0.3, causal)
    for b in range(B):
        keys = np.concatenate([pk, k[b]]).repeat(H // Hk, 1)
        vals = np.concatenate([pv, v[b]]).repeat(H // Hk, 1)
        s = np.einsum("qhd,nhd->hqn", q[cu[b]:cu[b + 1]], keys) * 0.3
        i, j = np.arange(cap), np.arange(n_q[b])[:, None]
        seen = (i < lens[b]) & ((i <= lens[b] - n_q[b] + j) | (not causal))
        s = np.where(np.concatenate([np.ones((n_q[b], Lp), bool), seen], 1)[None], s, -np.inf)
        t = torch.from_numpy(s)
        np.testing.assert_allclose(out[cu[b]:cu[b + 1]],
                                   np.einsum("hqn,nhd->qhd", torch.softmax(t, -1).numpy(), vals), rtol=1e-10)
        np.testing.assert_allclose(lse[cu[b]:cu[b + 1]], torch.logsumexp(t, -1).numpy().T, rtol=1e-10)


def test_prefix_attention_rows_without_keys():
    q = RNG.normal(size=(3, 2, 8))
    k = RNG.normal(size=(1, 4, 2, 8))
    out, lse = oo.prefix_attention(q, None, None, k, k, [1], [0, 3], 1.0)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all()      # only the last query sees the one key
    np.testing.assert_allclose(out[2], k[0, 0])
