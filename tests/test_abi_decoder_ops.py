"""The decoder-side entry points with types, gradients and workspaces refuse bad arguments on the host,
before any CUDA call, and size their workspaces without a device."""
import ctypes
import os

import numpy as np
import pytest
import torch

P = ctypes.c_void_p(0x10000)
OFF = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def nv():
    from resolution_vit_vision_b200 import build as b
    if not os.path.exists(b.LIB):
        b.build()
    from resolution_vit_vision_b200 import native
    native.lib()
    return native


def _sec(*v):
    return (ctypes.c_int32 * 3)(*v)


def _norm(nv, **kw):
    a = dict(q=P, qs=3584, qo=P, qos=3584, H=28, k=P, ks=512, ko=P, kos=512, Hk=4, D=128, dt=0, qw=P, kw=P, eps=1e-6,
             pos=P, L=4, theta=1e6, sec=_sec(16, 24, 24))
    a.update(kw)
    return nv.lib().mrope_norm_apply(a["q"], a["qs"], a["qo"], a["qos"], a["H"], a["k"], a["ks"], a["ko"], a["kos"],
                                     a["Hk"], a["D"], a["dt"], a["qw"], a["kw"], a["eps"], a["pos"], a["L"], a["theta"],
                                     a["sec"], None)


@pytest.mark.parametrize("bad, code", [
    (dict(q=None), "ARG"), (dict(ko=None), "ARG"), (dict(pos=None), "ARG"), (dict(sec=_sec(16, 24, 23)), "ARG"),
    (dict(sec=_sec(-8, 48, 24)), "ARG"), (dict(sec=_sec(2 ** 31 - 1, 2 ** 31 - 1, 66)), "ARG"), (dict(D=120), "ARG"),
    (dict(D=272), "ARG"), (dict(dt=3), "ARG"), (dict(eps=0.0), "ARG"), (dict(eps=float("nan")), "ARG"),
    (dict(theta=1.0), "ARG"), (dict(L=-1), "ARG"), (dict(H=-1), "ARG"), (dict(H=513), "ARG"), (dict(qs=3583), "ARG"),
    (dict(H=2 ** 30, D=16), "ARG"), (dict(qos=4608), "ARG"),              # in place with another stride
    (dict(qs=3588, qo=ctypes.c_void_p(0x20000)), "ALIGN"), (dict(q=OFF), "ALIGN"), (dict(qw=OFF), "ALIGN")])
def test_norm_refusals(nv, bad, code):
    assert _norm(nv, **bad) == getattr(nv, "VIT_ERR_" + code)


def test_norm_nothing_to_do(nv):
    assert _norm(nv, L=0) == nv.VIT_OK


def _norm_grad(nv, **kw):
    a = dict(x=P, xs=512, H=4, D=128, dt=0, dqw=P, ws=P, bytes=1 << 30, L=4)
    a.update(kw)
    return nv.lib().mrope_norm_grad(a["x"], a["xs"], a["x"], a["xs"], a["x"], a["xs"], a["H"], None, 0, None, 0, None,
                                    0, 0, a["D"], a["dt"], None, None, a["dqw"], None, 1e-6, P, a["L"], 1e6,
                                    _sec(16, 24, 24), a["ws"], a["bytes"], None)


def test_norm_grad_refusals(nv):
    need = nv.lib().mrope_norm_grad_workspace(128)
    assert need > 0 and nv.lib().mrope_norm_grad_workspace(8) == 0
    assert _norm_grad(nv, bytes=need - 1) == nv.VIT_ERR_ARG
    assert _norm_grad(nv, ws=None) == nv.VIT_ERR_ARG
    assert _norm_grad(nv, ws=OFF) == nv.VIT_ERR_ALIGN
    assert _norm_grad(nv, x=None) == nv.VIT_ERR_ARG
    assert _norm_grad(nv, dt=7) == nv.VIT_ERR_ARG
    assert _norm_grad(nv, xs=516) == nv.VIT_ERR_ALIGN


def test_embed_refusals(nv):
    def call(L=10, table=P, dt=0, vocab=100, dim=64, scale=2.0, vis=P, n=2, out=P, ids=P):
        return nv.lib().embed_vision_tokens(ids, L, table, dt, vocab, dim, scale, vis, n, out, None, None)
    assert call(dim=12) == nv.VIT_ERR_ARG and call(dim=65544) == nv.VIT_ERR_ARG
    assert call(L=(1 << 18) + 1) == nv.VIT_ERR_ARG and call(L=-1) == nv.VIT_ERR_ARG
    assert call(vocab=0) == nv.VIT_ERR_ARG and call(vocab=(1 << 30) + 1) == nv.VIT_ERR_ARG
    assert call(dt=3) == nv.VIT_ERR_ARG and call(scale=float("inf")) == nv.VIT_ERR_ARG
    assert call(vis=None) == nv.VIT_ERR_ARG and call(ids=None) == nv.VIT_ERR_ARG and call(n=-1) == nv.VIT_ERR_ARG
    assert call(table=OFF) == nv.VIT_ERR_ALIGN and call(out=OFF) == nv.VIT_ERR_ALIGN
    assert call(L=0, n=0, ids=None, table=None, out=None, vis=None) == nv.VIT_OK


def test_embed_grad_refusals(nv):
    lib = nv.lib()
    need = lib.embed_vision_tokens_grad_workspace(10, 100, 64)
    assert need > 0
    for bad in ((-1, 100, 64), ((1 << 18) + 1, 100, 64), (10, 0, 64), (10, 100, 60), (10, (1 << 30) + 1, 64)):
        assert lib.embed_vision_tokens_grad_workspace(*bad) == 0

    def call(L=10, ids=P, d=P, dt=0, vocab=100, dim=64, scale=1.0, table=P, tdt=0, vis=P, n=2, ws=P, size=need):
        return lib.embed_vision_tokens_grad(ids, L, d, dt, vocab, dim, scale, table, tdt, 0, vis, n, ws, size, None, None)
    assert call(size=need - 1) == nv.VIT_ERR_ARG and call(ws=None) == nv.VIT_ERR_ARG
    assert call(ws=OFF) == nv.VIT_ERR_ALIGN and call(table=OFF) == nv.VIT_ERR_ALIGN and call(d=OFF) == nv.VIT_ERR_ALIGN
    assert call(dt=0, tdt=1) == nv.VIT_ERR_ARG and call(dt=2, tdt=0) == nv.VIT_ERR_ARG and call(dt=5, tdt=5) == nv.VIT_ERR_ARG
    assert call(vis=None) == nv.VIT_ERR_ARG and call(ids=None) == nv.VIT_ERR_ARG and call(table=None) == nv.VIT_ERR_ARG
    assert call(scale=float("nan")) == nv.VIT_ERR_ARG and call(dim=20) == nv.VIT_ERR_ARG


def _desc(nv, **kw):
    d = nv.PrefixAttentionDesc()
    a = dict(dtype=0, n_heads=28, n_kv_heads=4, head_dim=128, scale=0.1, causal=1, q=P.value, q_stride=3584, out=P.value,
             out_stride=3584, lse=None, total_q=6, max_q=2, cu_q=None, n_seq=3, prefix_k=P.value, prefix_v=P.value,
             prefix_len=10, prefix_k_token=512, prefix_k_head=128, prefix_v_token=512, prefix_v_head=128, k=P.value,
             v=P.value, k_seq=4096, k_token=512, k_head=128, v_seq=4096, v_token=512, v_head=128, lens=P.value, max_len=8)
    a.update(kw)
    for n, v in a.items():
        setattr(d, n, v)
    return d


@pytest.mark.parametrize("bad, code", [
    (dict(dtype=2), "ARG"), (dict(head_dim=136), "ARG"), (dict(head_dim=12), "ARG"), (dict(head_dim=0), "ARG"),
    (dict(n_heads=27), "ARG"), (dict(n_kv_heads=0), "ARG"), (dict(n_heads=129 * 4), "ARG"),
    (dict(scale=float("inf")), "ARG"), (dict(scale=0.0), "ARG"), (dict(scale=-0.1), "ARG"), (dict(n_seq=0), "ARG"), (dict(max_q=0), "ARG"), (dict(total_q=7), "ARG"),
    (dict(total_q=-1), "ARG"), (dict(prefix_len=-1), "ARG"), (dict(prefix_k=None), "ARG"), (dict(v=None), "ARG"),
    (dict(lens=None), "ARG"), (dict(k=None, v=None, lens=None), "ARG"), (dict(q=None), "ARG"), (dict(out=None), "ARG"),
    (dict(q_stride=3576), "ARG"), (dict(k_token=0), "ARG"), (dict(k_seq=0), "ARG"), (dict(k_seq=-4096), "ARG"),
    (dict(prefix_v_head=64), "ARG"), (dict(n_seq=65537, total_q=65537, max_q=1), "LIMIT"),
    (dict(prefix_len=(1 << 30) + 1), "LIMIT"), (dict(max_len=(1 << 30) + 1), "LIMIT"),
    (dict(total_q=1 << 27, cu_q=P.value), "LIMIT"), (dict(q=OFF.value), "ALIGN"), (dict(prefix_k=OFF.value), "ALIGN"),
    (dict(v=OFF.value), "ALIGN"), (dict(out_stride=3588), "ALIGN"), (dict(k_token=516), "ALIGN")])
def test_prefix_attention_refusals(nv, bad, code):
    d = _desc(nv, **bad)
    assert nv.lib().prefix_attention_workspace(ctypes.byref(d)) == 0
    assert nv.lib().prefix_attention(ctypes.byref(d), P, 1 << 40, None, None) == getattr(nv, "VIT_ERR_" + code)


def test_prefix_attention_row_numbers_fit(nv):
    # an item's rows are numbered in 32 bits up to a tile behind the last: no row may come near 2^31
    one = dict(n_heads=8, n_kv_heads=1, head_dim=8, q_stride=64, out_stride=64, cu_q=P.value, n_seq=1, k=None, v=None,
               lens=None, max_len=0, max_q=1)
    most = ((1 << 31) - 1024) // 8
    for bad in (dict(total_q=most + 1), dict(total_q=6, max_q=most + 1), dict(total_q=6, n_seq=64, max_q=most // 64 + 1)):
        d = _desc(nv, **{**one, **bad})
        assert nv.lib().prefix_attention_workspace(ctypes.byref(d)) == 0
        assert nv.lib().prefix_attention(ctypes.byref(d), P, 1 << 40, None, None) == nv.VIT_ERR_LIMIT


def test_prefix_attention_workspace_is_checked(nv):
    d = _desc(nv, n_seq=100, total_q=200, prefix_len=5000)     # long enough for parts
    need = nv.lib().prefix_attention_workspace(ctypes.byref(d))
    assert need > 0
    assert nv.lib().prefix_attention(ctypes.byref(d), None, 0, None, None) == nv.VIT_ERR_ARG
    assert nv.lib().prefix_attention(ctypes.byref(d), P, need - 1, None, None) == nv.VIT_ERR_ARG
    assert nv.lib().prefix_attention(ctypes.byref(d), OFF, need, None, None) == nv.VIT_ERR_ALIGN
    assert nv.lib().prefix_attention(None, P, need, None, None) == nv.VIT_ERR_ARG
    empty = _desc(nv, total_q=0)
    assert nv.lib().prefix_attention(ctypes.byref(empty), None, 0, None, None) == nv.VIT_OK


def test_binding_refuses_wrong_tensors(nv):
    x = torch.zeros(4, 2, 32, dtype=torch.bfloat16)
    pos = torch.zeros(3, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        nv.mrope_norm_apply(x, None, pos, sections=(4, 6, 6))                   # not on a GPU
    with pytest.raises(ValueError):
        nv.mrope_norm_apply(None, None, pos)
    with pytest.raises(ValueError):
        nv.mrope_norm_apply(x.double(), None, pos)
    with pytest.raises(ValueError):
        nv.mrope_norm_apply(x, x[:2], pos)
    with pytest.raises(ValueError):
        nv.mrope_norm_apply(x, None, pos.long())
    with pytest.raises(ValueError):
        nv.mrope_norm_grad(x[:, :1], None, x, None, pos)
    with pytest.raises(ValueError):
        nv.embed_vision_tokens(torch.zeros(3, dtype=torch.int64), x[0])
    with pytest.raises(ValueError):
        nv.embed_vision_tokens_grad(torch.zeros(4, dtype=torch.int32), x[:, 0], 8, table_dtype=torch.float16)
    with pytest.raises(ValueError):
        nv.embed_vision_tokens_grad(torch.zeros(4, dtype=torch.int32), x[:, 0], 8, accumulate=True)
    kv = torch.zeros(4, 5, 1, 32, dtype=torch.bfloat16)
    lens = torch.zeros(4, dtype=torch.int32)
    for bad in (dict(q=x.float()), dict(k=kv, v=None), dict(lens=None), dict(lens=lens[:3]), dict(max_len=6),
                dict(v=kv[..., :16]), dict(max_q=2), dict(k=kv[:3], v=kv[:3], lens=lens[:3])):
        a = dict(q=x, k=kv, v=kv, lens=lens)
        a.update(bad)
        with pytest.raises(ValueError):
            nv.prefix_attention(**a)
    with pytest.raises(ValueError):
        nv.prefix_attention(x)


def test_norm_sections_default(nv):
    assert sum(nv.MROPE_SECTIONS) == 64 and np.asarray(nv.MROPE_SECTIONS).shape == (3,)
