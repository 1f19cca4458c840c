"""Decoder-side steps with types and gradients on a B200 against the fp64 oracle.

Tolerances, from the arithmetic (u: half a step of the element type, torch.finfo(t).eps / 2):
* norm + rotation: the mean of squares (at most 256 terms, 20 additions deep), 1/sqrt, the angle (one
  fp32 rounding of a value below pi, 2^-23) and six products are off by less than 2^-18 relative to
  |n_lo| + |n_hi| of a pair; one rounding to the type: u |ref|.
* its gradient: two sums of that kind and a difference; 2^-17 of the size of the terms, then u |ref|.
  The weights' gradient is a sum over rows: 2^-17 of the sum of |terms| (depth under 64).
* embedding rows: a product in fp32 and one rounding: (u + 2^-24) |ref|; their gradient: a sum of n terms
  in fp32, n 2^-24 of the sum of |terms|, then u |ref|.
"""
import numpy as np
import pytest
import torch

from oracle import decoder_oracle as do
from oracle import decoder_ops_oracle as oo
from resolution_vit_vision_b200 import native as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IMG, VID = do.IMAGE_TOKEN_ID, do.VIDEO_TOKEN_ID


def _u(t):
    return torch.finfo(t).eps / 2


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, t, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(t)


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _within(got, ref, bound, what):
    got = _np(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    bad = np.abs(got - ref) > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {(np.abs(got - ref) - bound).max():.3e}"


def _secs(D):
    t = D // 8
    h = (D // 2 - t) // 2
    return t, h, D // 2 - t - h


def _norm_case(L, H, Hk, D, t, seed, packed=False, far=0, scale=1.5):
    g = _gen(seed)
    if packed:
        qkv = _randn(g, (L, (H + 2 * Hk) * D), t, scale)
        q, k = qkv[:, :H * D].view(L, H, D), qkv[:, H * D:(H + Hk) * D].view(L, Hk, D)
    else:
        q, k = _randn(g, (L, H, D), t, scale), _randn(g, (L, Hk, D), t, scale)
    qw, kw = (1 + _randn(g, (D,), torch.float32, 0.2)).to(t), (1 + _randn(g, (D,), torch.float32, 0.2)).to(t)
    pos = torch.randint(0, 2000, (3, L), generator=g, device=DEV, dtype=torch.int32) + far
    return q, k, qw, kw, pos


def _norm_bound(x, w, ref, t, eps=1e-6):
    x = _np(x)
    n = np.abs(x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * (1.0 if w is None else _np(w)))
    h = n.shape[-1] // 2
    pair = n[..., :h] + n[..., h:]
    return _u(t) * np.abs(ref) + 2.0 ** -18 * np.concatenate([pair, pair], -1) + (2.0 ** -24 if t == torch.float16 else 0)


CASES = [(1, 28, 4, 128, "bf16", True, 0), (3, 28, 4, 128, "fp16", False, 120000), (7, 3, 1, 16, "bf16", True, 0),
         (5, 2, 2, 16, "fp32", False, 3), (19, 5, 5, 80, "bf16", True, 50), (9, 4, 2, 80, "fp32", True, 50),
         (11, 8, 1, 64, "fp16", True, 7), (6, 3, 2, 96, "bf16", False, 0), (4, 2, 1, 256, "fp32", True, 9),
         (4, 2, 1, 256, "bf16", False, 9), (1237, 12, 2, 128, "bf16", True, 0), (5, 41, 3, 128, "bf16", True, 0)]


@pytest.mark.parametrize("L, H, Hk, D, t, packed, far", CASES)
def test_norm_apply(L, H, Hk, D, t, packed, far):
    t = TYPES[t]
    q, k, qw, kw, pos = _norm_case(L, H, Hk, D, t, 100 + L + D, packed, far)
    q0, k0 = q.clone(), k.clone()
    qo, ko = nv.mrope_norm_apply(q, k, pos, qw, kw, sections=_secs(D))
    for x, x0, w, got, what in ((q, q0, qw, qo, "q"), (k, k0, kw, ko, "k")):
        ref = oo.norm_rope(_np(x0), _np(w), pos.cpu().numpy(), _secs(D))
        _within(got, ref, _norm_bound(x0, w, ref, t), what)
        assert torch.equal(x, x0)
    # in place, without weights, one of the two alone
    ref = oo.norm_rope(_np(k0), None, pos.cpu().numpy(), _secs(D))
    none, same = nv.mrope_norm_apply(None, k, pos, sections=_secs(D), k_out=k)
    assert none is None and same is k
    _within(k, ref, _norm_bound(k0, None, ref, t), "k in place")
    assert torch.equal(q, q0)                         # the neighbours in the packed rows are untouched


def test_norm_apply_extremes():
    # a zero row gives zeros, a tiny row is ruled by eps, a large one stays finite
    x = torch.zeros(3, 1, 64, dtype=torch.float32, device=DEV)
    x[1] = 1e-6
    x[2] = 1e15
    pos = torch.zeros(3, 3, dtype=torch.int32, device=DEV)
    y, _ = nv.mrope_norm_apply(x, None, pos, sections=(8, 12, 12))
    ref = oo.norm_rope(_np(x), None, np.zeros((3, 3)), (8, 12, 12))
    _within(y, ref, _norm_bound(x, None, ref, torch.float32), "extremes")
    assert (y[0] == 0).all()
    e, _ = nv.mrope_norm_apply(x[:0], None, pos[:, :0].contiguous(), sections=(8, 12, 12))
    assert e.shape == (0, 1, 64)


@pytest.mark.parametrize("L, H, Hk, D, t, packed, far", CASES)
def test_norm_grad(L, H, Hk, D, t, packed, far):
    t = TYPES[t]
    q, k, qw, kw, pos = _norm_case(L, H, Hk, D, t, 300 + L + D, packed, far)
    g = _gen(17)
    dqo, dko = _randn(g, q.shape, t), _randn(g, k.shape, t)
    found = nv.mrope_norm_grad(dqo, dko, q, k, pos, qw, kw, sections=_secs(D))
    again = nv.mrope_norm_grad(dqo, dko, q, k, pos, qw, kw, sections=_secs(D))
    assert all(torch.equal(a, b) for a, b in zip(found, again))
    p = pos.cpu().numpy()
    for x, w, d, dx, dw, what in ((q, qw, dqo, found[0], found[2], "q"), (k, kw, dko, found[1], found[3], "k")):
        rx, rw = oo.norm_rope_grad(_np(d), _np(x), _np(w), p, _secs(D))
        X, W, dd = _np(x), _np(w), np.abs(_np(d))
        rms = np.sqrt((X ** 2).mean(-1, keepdims=True) + 1e-6)
        pair = dd[..., :D // 2] + dd[..., D // 2:]
        dn = np.concatenate([pair, pair], -1)
        gr = dn * np.abs(W)
        size = (gr + np.abs(X) * (gr * np.abs(X)).mean(-1, keepdims=True) / rms ** 2) / rms
        _within(dx, rx, _u(t) * np.abs(rx) + 2.0 ** -17 * size + (2.0 ** -24 if t == torch.float16 else 0), "d" + what)
        assert dw.dtype == torch.float32
        _within(dw, rw, 2.0 ** -17 * (dn * np.abs(X) / rms).sum((0, 1)), f"d{what}_weight")
    # into the buffer of the incoming gradient, weights' gradients left out
    dq2, dk2, a, b = nv.mrope_norm_grad(dqo, dko, q, k, pos, qw, kw, sections=_secs(D), dq=dqo, dk=dko, weight_grads=False)
    assert dq2 is dqo and a is None and b is None and torch.equal(dqo, found[0]) and torch.equal(dko, found[1])


def test_norm_grad_against_differences():
    t = torch.float32
    q, k, qw, kw, pos = _norm_case(3, 2, 1, 32, t, 5)
    d = _randn(_gen(6), q.shape, t)
    dq, _, dqw, _ = nv.mrope_norm_grad(d, None, q, None, pos, qw, None, sections=_secs(32))

    def f(x, w):     # fp64 sum of the fp32 kernel's outputs
        return (nv.mrope_norm_apply(x, None, pos, w, None, sections=_secs(32))[0].double() * d.double()).sum().item()
    h = 2.0 ** -6    # differences: h^2 of the third derivative, and 2 * 96 * 2^-22 / 2h of rounding, under 1e-2
    for i in ((0, 0, 3), (1, 1, 20), (2, 0, 31)):
        e = torch.zeros_like(q)
        e[i] = h
        assert abs(dq[i].item() - (f(q + e, qw) - f(q - e, qw)) / (2 * h)) < 1e-2
    for i in (0, 17):
        e = torch.zeros_like(qw)
        e[i] = h
        assert abs(dqw[i].item() - (f(q, qw + e) - f(q, qw - e)) / (2 * h)) < 1e-2


def test_norm_grad_no_tokens_writes_zero_weight_gradients():
    x = torch.zeros(0, 2, 32, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(3, 0, dtype=torch.int32, device=DEV)
    _, _, dw, _ = nv.mrope_norm_grad(x, None, x, None, pos, sections=_secs(32))
    assert (dw == 0).all()


# ------------------------------------------------------------------------------------------ embedding
def _ids(L, vocab, seed, vision=0.4):
    rng = np.random.default_rng(seed)
    ids = np.minimum((np.exp(rng.random(L) * np.log(vocab)) - 1).astype(np.int64), vocab - 1)   # heavy repeats
    i = 0
    while i < L:
        run = int(rng.integers(1, 40))
        if rng.random() < vision:
            ids[i:i + run] = IMG if rng.random() < 0.5 else VID
        i += run
    return ids


def _dev_ids(ids):
    return torch.from_numpy(np.ascontiguousarray(ids, np.int32)).to(DEV)


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("L, vocab, dim, scale", [(1, 10, 8, 2.5), (3, 3000, 264, 1.0), (517, 900, 1536, 39.25),
                                                  (5003, 152064, 72, -0.3)])
def test_embed_rows(L, vocab, dim, scale, t):
    t = TYPES[t]
    g = _gen(L)
    ids = _ids(L, vocab, L, 0.4 if L > 1 else 0.0)
    n_vis = int(((ids == IMG) | (ids == VID)).sum())
    table, vis = _randn(g, (vocab, dim), t), _randn(g, (n_vis, dim), t)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = nv.embed_vision_tokens(_dev_ids(ids), table, vis, scale=scale, status=st)
    ref = oo.embed_rows(ids, _np(table), _np(vis), float(np.float32(scale)))
    slots = (ids == IMG) | (ids == VID)
    exact = slots[:, None] | np.full(ref.shape, scale == 1.0)
    _within(out, ref, np.where(exact, 0.0, (_u(t) + 2.0 ** -24) * np.abs(ref) + (2.0 ** -24 if t == torch.float16 else 0)),
            "rows")
    assert st.item() == 0


def test_embed_rows_errors_leave_rows():
    g = _gen(3)
    table, vis = _randn(g, (16, 64), torch.float16), _randn(g, (1, 64), torch.float16)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full((5, 64), -3.0, dtype=torch.float16, device=DEV)
    nv.embed_vision_tokens(_dev_ids([3, IMG, 16, VID, -1]), table, vis, scale=2.0, out=out, status=st)
    assert st.item() == nv.VIT_ERR_TOKENS
    assert torch.equal(out[0], table[3] * 2) and torch.equal(out[1], vis[0]) and (out[2:] == -3.0).all()


@pytest.mark.parametrize("t, gt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("L, vocab, dim, scale", [(1, 7, 8, 2.0), (65, 40, 1032, 1.0), (700, 3, 136, 0.5),
                                                  (4096, 100000, 8, 1.0), (4097, 520, 264, 3.0), (20011, 152064, 16, 1.5)])
def test_embed_grad(L, vocab, dim, scale, t, gt):
    t, gt = TYPES[t], TYPES[gt]
    g = _gen(L + dim)
    ids = _ids(L, vocab, L + 1, 0.4 if L > 1 else 0.0)
    n_vis = int(((ids == IMG) | (ids == VID)).sum())
    d = _randn(g, (L, dim), t)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    dt, dv = nv.embed_vision_tokens_grad(_dev_ids(ids), d, vocab, n_vis, scale=scale, table_dtype=gt, status=st)
    rt, rv = oo.embed_rows_grad(ids, _np(d), vocab, scale)
    size, _ = oo.embed_rows_grad(ids, np.abs(_np(d)), vocab, scale)
    text = ids[(ids != IMG) & (ids != VID)]
    n = np.bincount(text, minlength=vocab)[:, None]
    _within(dt, rt, _u(gt) * np.abs(rt) + (n + 2) * 2.0 ** -24 * size + (2.0 ** -24 if gt == torch.float16 else 0), "d_table")
    if n_vis:
        np.testing.assert_array_equal(_np(dv), rv)
    assert st.item() == 0 and dt.dtype == gt
    dt2, _ = nv.embed_vision_tokens_grad(_dev_ids(ids), d, vocab, n_vis, scale=scale, table_dtype=gt)
    assert torch.equal(dt, dt2)
    # added to what is there; rows without a token keep their bits
    old = _randn(g, (vocab, dim), gt)
    acc = old.clone()
    nv.embed_vision_tokens_grad(_dev_ids(ids), d, vocab, n_vis, scale=scale, d_table=acc, accumulate=True)
    ra = _np(old) + rt
    _within(acc, ra, _u(gt) * np.abs(ra) + (n + 3) * 2.0 ** -24 * (size + np.abs(_np(old)))
            + (2.0 ** -24 if gt == torch.float16 else 0), "accumulated")
    idle = torch.from_numpy(n[:, 0] == 0).to(DEV)
    assert torch.equal(acc[idle], old[idle])


def test_embed_grad_one_id_throughout():
    # one run over every chunk of the sorted list, and over the cluster's shares
    L, dim = 9001, 24
    d = _randn(_gen(8), (L, dim), torch.bfloat16)
    dt, _ = nv.embed_vision_tokens_grad(_dev_ids(np.full(L, 5)), d, 9, table_dtype=torch.float32)
    ref = _np(d).sum(0)
    _within(dt[5], ref, L * 2.0 ** -24 * np.abs(_np(d)).sum(0), "sum")
    assert (dt[[0, 1, 2, 3, 4, 6, 7, 8]] == 0).all()


def test_embed_grad_errors_and_empty():
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = _randn(_gen(9), (6, 16), torch.float32)
    ids = _dev_ids([2, IMG, 99, -4, 2, VID])
    dt, dv = nv.embed_vision_tokens_grad(ids, d, 5, 3, status=st)       # two ids outside, one vision token too many
    assert st.item() == nv.VIT_ERR_TOKENS
    assert torch.equal(dt[2], d[0] + d[4]) and (dt[[0, 1, 3, 4]] == 0).all()
    assert torch.equal(dv[:2], d[[1, 5]]) and (dv[2] == 0).all()
    st.zero_()
    dt, dv = nv.embed_vision_tokens_grad(ids, d, 100, 1, status=st)     # more placeholders than vision tokens
    assert st.item() == nv.VIT_ERR_TOKENS and torch.equal(dv[0], d[1]) and torch.equal(dt[99], d[2])
    dt, dv = nv.embed_vision_tokens_grad(ids[:0], d[:0], 5)
    assert (dt == 0).all() and dv is None
    acc = torch.ones(5, 16, device=DEV)
    nv.embed_vision_tokens_grad(ids[:0], d[:0], 5, d_table=acc, accumulate=True)
    assert (acc == 1).all()


def test_embed_grad_longest_prompt():
    L, vocab = 1 << 18, 70000
    ids = _ids(L, vocab, 4)
    n_vis = int(((ids == IMG) | (ids == VID)).sum())
    d = torch.ones(L, 8, dtype=torch.float32, device=DEV)
    dt, dv = nv.embed_vision_tokens_grad(_dev_ids(ids), d, vocab, n_vis)
    text = ids[(ids != IMG) & (ids != VID)]
    np.testing.assert_array_equal(_np(dt)[:, 3], np.bincount(text, minlength=vocab).astype(np.float64))   # exact below 2^24
    assert (dv == 1).all()


def test_other_stream_and_graph():
    L, dim, vocab = 300, 64, 500
    ids = _ids(L, vocab, 12)
    n_vis = int(((ids == IMG) | (ids == VID)).sum())
    t_ids = _dev_ids(ids)
    d = _randn(_gen(1), (L, dim), torch.bfloat16)
    q, k, qw, kw, pos = _norm_case(L, 4, 2, 64, torch.bfloat16, 2)
    want = nv.embed_vision_tokens_grad(t_ids, d, vocab, n_vis) + nv.mrope_norm_grad(q, k, q, k, pos, qw, kw, sections=_secs(64))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = nv.embed_vision_tokens_grad(t_ids, d, vocab, n_vis, stream=s) + \
        nv.mrope_norm_grad(q, k, q, k, pos, qw, kw, sections=_secs(64), stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = nv.embed_vision_tokens_grad(t_ids, d, vocab, n_vis) + \
            nv.mrope_norm_grad(q, k, q, k, pos, qw, kw, sections=_secs(64))
    d.mul_(2)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0] * 2) and torch.equal(got[1], want[1] * 2)
    assert all(torch.equal(a, b) for a, b in zip(want[2:], got[2:]))


@pytest.mark.parametrize("L", [1, 700])
@pytest.mark.parametrize("graph", [False, True])
def test_norm_calls_follow_what_the_stream_did_before(L, graph):
    # launches may start early: operands written by slow kernels just before, results read by the next call,
    # operands overwritten behind it
    q, k, qw, kw, pos = _norm_case(L, 12, 2, 128, torch.bfloat16, 60)
    ops = [q, k, qw, kw, pos]
    kwargs = dict(sections=_secs(128))

    def steps(q, k, qw, kw, pos, sync):
        for _ in range(3):
            nv.mrope_norm_apply(q, k, pos, qw, kw, q_out=q, k_out=k, **kwargs)
            sync()
        y = nv.mrope_norm_apply(q, k, pos, qw, kw, **kwargs)
        sync()
        g = nv.mrope_norm_grad(*y, q, k, pos, qw, kw, **kwargs)
        sync()
        return list(y) + list(g)
    want = steps(*[t.clone() for t in ops], torch.cuda.synchronize)
    slow = torch.zeros(64 << 20, dtype=torch.float32, device=DEV)
    mine = [torch.zeros_like(t) for t in ops]

    def chain():
        slow.add_(1.0)
        for a, b in zip(mine, ops):
            a.copy_(b)
        out = steps(*mine, lambda: None)
        for a in mine:
            a.zero_()
        return out
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = chain()
        s.synchronize()
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                got = chain()
        for _ in range(5):
            if graph:
                for t in got:
                    t.zero_()
                g.replay()
            else:
                got = chain()
        s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
