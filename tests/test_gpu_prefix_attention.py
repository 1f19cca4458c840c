"""Attention over a shared prefix on a B200 against the fp64 oracle.

Tolerances (u: half a step of the type). Scores: q . k is summed in fp32, off by at most head_dim 2^-24 of
sum |q_i k_i| times the scale, under 1e-4 at the sizes here, so the weights are off by 1e-4 relatively.
P is rounded to the type for P V (u, weights sum to 1), o once more: |err| <= (2 u + 4e-4) max |v|.
lse: 1e-4 + 2^-22 |lse|.
"""
import numpy as np
import pytest
import torch

from oracle import decoder_ops_oracle as oo
from resolution_vit_vision_b200 import native as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _case(seed, B, n_q, lens, Lp, H, Hk, D, t, cap=None, std=1.0):
    """n_q: a number (uniform) or a list (ragged); lens None: no own keys."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def rn(*shape):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(TYPES[t])
    ragged = not isinstance(n_q, int)
    cu = np.concatenate([[0], np.cumsum(n_q if ragged else [n_q] * B)])
    q = rn(cu[-1], H, D)
    pk, pv = (rn(Lp, Hk, D), rn(Lp, Hk, D)) if Lp else (None, None)
    k = v = tl = None
    if lens is not None:
        cap = max(lens) if cap is None else cap
        k, v = rn(B, cap, Hk, D), rn(B, cap, Hk, D)
        tl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    t_cu = torch.tensor(cu, dtype=torch.int32, device=DEV) if ragged else None
    return dict(q=q, prefix_k=pk, prefix_v=pv, k=k, v=v, lens=tl, cu_q=t_cu, max_q=int(max(n_q)) if ragged else n_q), cu


def _check(a, cu, got, causal=True, scale=None, rows=None):
    out, lse = got
    ref, rlse = oo.prefix_attention(_np(a["q"]), _np(a["prefix_k"]), _np(a["prefix_v"]), _np(a["k"]), _np(a["v"]),
                                    None if a["lens"] is None else a["lens"].tolist(), cu,
                                    a["q"].shape[-1] ** -0.5 if scale is None else scale, causal)
    vmax = max([np.abs(_np(x)).max() for x in (a["prefix_v"], a["v"]) if x is not None and x.numel()] + [0.0])
    bound = (2 * torch.finfo(a["q"].dtype).eps / 2 + 4e-4) * vmax
    o, s = _np(out)[:cu[-1]], _np(lse)[:cu[-1]]
    assert np.isfinite(o).all()
    assert np.abs(o - ref).max() <= bound, f"out off by {np.abs(o - ref).max():.3e}, bound {bound:.3e}"
    none = np.isneginf(rlse)
    np.testing.assert_array_equal(np.isneginf(s), none)
    assert (o[none] == 0).all()
    off = np.abs(s[~none] - rlse[~none]) - (1e-4 + 2.0 ** -22 * np.abs(rlse[~none]))
    assert off.size == 0 or off.max() <= 0, f"lse off by {off.max():.3e} over the bound"


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("H, Hk, D", [(28, 4, 128), (4, 4, 64), (8, 1, 80), (3, 1, 8), (5, 5, 120), (16, 1, 96), (2, 2, 16)])
def test_decoding(H, Hk, D, t):
    # one query per sequence; lengths from one to past a key tile, the prefix ending inside a tile
    a, cu = _case(1, 5, 1, [1, 2, 63, 64, 130], 201, H, Hk, D, t, cap=137)
    _check(a, cu, nv.prefix_attention(**a))


@pytest.mark.parametrize("Lp", [0, 1, 63, 64, 65, 127, 128, 129, 1000])
@pytest.mark.parametrize("B", [1, 3, 40])
def test_prefix_lengths(B, Lp):
    lens = [1 + (37 * b) % 70 for b in range(B)]
    a, cu = _case(2 + Lp, B, 1, lens, Lp, 14, 2, 128, "bf16")
    _check(a, cu, nv.prefix_attention(**a))


@pytest.mark.parametrize("n_q, lens", [([3, 1, 17], [3, 1, 17]), ([40, 1, 0, 65], [40, 200, 5, 65]), ([130], [131]),
                                       ([1, 300], [1, 300]), ([0, 0, 2], [0, 3, 2])])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_questions(n_q, lens, causal):
    a, cu = _case(5, len(n_q), n_q, lens, 77, 6, 2, 128, "bf16", cap=max(lens) + 3)
    _check(a, cu, nv.prefix_attention(**a, causal=causal), causal)


@pytest.mark.parametrize("n_q", [2, 5, 9, 33, 70])
def test_several_queries_each(n_q):
    a, cu = _case(6, 3, n_q, [n_q, n_q + 1, n_q + 90], 150, 8, 2, 64, "fp16")
    _check(a, cu, nv.prefix_attention(**a))


@pytest.mark.parametrize("Lp", [0, 3])
@pytest.mark.parametrize("n_q, lens", [([5, 4, 2], [2, 0, 0]), ([200, 131, 3], [100, 0, 2])])
def test_rows_without_keys(n_q, lens, Lp):
    # more queries than own keys: the first rows see the prefix only, or nothing
    a, cu = _case(7, 3, n_q, lens, Lp, 4, 2, 64, "bf16", cap=109)
    _check(a, cu, nv.prefix_attention(**a))


def test_prefix_only():
    a, cu = _case(8, 6, 3, None, 333, 12, 2, 128, "bf16")
    _check(a, cu, nv.prefix_attention(**a))
    a, cu = _case(8, 1, [50], None, 1333, 12, 2, 128, "fp16")
    _check(a, cu, nv.prefix_attention(**a))


def test_long_prefix_few_rows():
    # the prefix is cut into many parts
    a, cu = _case(9, 2, 1, [3, 700], 9001, 7, 1, 128, "bf16")
    _check(a, cu, nv.prefix_attention(**a))
    a, cu = _case(10, 1, 1, [2], 9001, 4, 2, 64, "fp16")
    _check(a, cu, nv.prefix_attention(**a))


def test_large_scores_and_scale():
    # the running maximum moves from tile to tile; weights underflow
    a, cu = _case(11, 4, 2, [100, 3, 260, 9], 300, 8, 2, 128, "bf16", std=2.0)
    a["prefix_k"][200:] *= 4
    for scale in (1e-30, 0.02, 0.5):
        _check(a, cu, nv.prefix_attention(**a, scale=scale), scale=scale)


@pytest.mark.parametrize("n_q", [1, 20, 80])
def test_strides_and_garbage_outside(n_q):
    # head-major caches, packed q rows, NaN in every place that no row may see
    B, H, Hk, D, Lp, cap = 3, 6, 2, 64, 90, 200
    lens = [n_q, n_q + 1, 200]
    a, cu = _case(12, B, n_q, lens, Lp, H, Hk, D, "bf16", cap=cap)
    ref = dict(a)
    qkv = torch.full((B * n_q, (H + 4) * D), float("nan"), dtype=torch.bfloat16, device=DEV)
    qkv[:, D:(H + 1) * D] = a["q"].view(B * n_q, H * D)
    b = dict(a, q=qkv[:, D:(H + 1) * D].view(B * n_q, H, D))
    for n in ("prefix_k", "prefix_v"):
        big = torch.full((Hk, Lp + 70, D + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
        big[:, :Lp, :D] = a[n].transpose(0, 1)
        b[n] = big[:, :Lp, :D].transpose(0, 1)
    for n in ("k", "v"):
        big = torch.full((B, Hk, cap + 10, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        for i, L in enumerate(lens):
            big[i, :, :L] = a[n][i, :L].transpose(0, 1)
        b[n] = big[:, :, :cap].transpose(1, 2)
    store = torch.full((B * n_q + 2, H + 3, D), 7.0, dtype=torch.bfloat16, device=DEV)
    b["out"] = store[1:-1, :H]
    got = nv.prefix_attention(**b)
    assert got[0].data_ptr() == b["out"].data_ptr()
    _check(ref, cu, got)
    assert (store[0] == 7).all() and (store[-1] == 7).all() and (store[:, H:] == 7).all()


@pytest.mark.parametrize("n_q, Lp", [([1, 1, 1], 50), ([1, 1, 1], 0), ([40, 3, 90], 50), ([40, 3, 90], 0)])
def test_rows_behind_the_last_sequence_stay(n_q, Lp):
    a, cu = _case(13, 3, n_q, [95, 3, 91], Lp, 4, 1, 64, "fp16")
    pad = torch.randn(7, 4, 64, device=DEV).to(torch.float16)
    a["q"] = torch.cat([a["q"], pad])
    out = torch.full_like(a["q"], 3.0)
    lse = torch.full(out.shape[:2], 5.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    nv.prefix_attention(**a, out=out, lse=lse, status=st)
    _check(dict(a, q=a["q"][:cu[-1]]), cu, (out, lse))
    assert (out[cu[-1]:] == 3).all() and (lse[cu[-1]:] == 5).all() and st.item() == 0


def test_bad_lengths_are_flagged_and_stay_inside():
    # decided on the device: clamped, reported, the other sequences right
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    a, cu = _case(14, 3, 1, [5, 9, 3], 40, 4, 2, 64, "bf16")
    good = nv.prefix_attention(**a)
    for bad in (-1, 10, 2 ** 31 - 1, -2 ** 31):
        st.zero_()
        lens = a["lens"].clone()
        lens[1] = bad
        got = nv.prefix_attention(**dict(a, lens=lens), status=st)
        assert st.item() == nv.VIT_ERR_LIMIT
        assert torch.equal(got[0][[0, 2]], good[0][[0, 2]])
    a, cu = _case(15, 3, [2, 3, 2], [5, 9, 3], 40, 4, 2, 64, "bf16")
    good = nv.prefix_attention(**a)
    for bad in ([0, 2, 1, 3], [0, 2, 100, 101], [0, 2, 5, 2 ** 31 - 1], [0, 2, -7, -5], [0, 2, 7, 7]):
        st.zero_()
        cu_bad = torch.tensor(bad, dtype=torch.int32, device=DEV)
        got = nv.prefix_attention(**dict(a, cu_q=cu_bad), status=st)
        torch.cuda.synchronize()
        assert st.item() == nv.VIT_ERR_LIMIT, bad
        assert torch.equal(got[0][:1], good[0][:1])      # row 1 is named twice by the first of them


def test_bad_query_ranges_of_a_prefix_alone():
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    a, cu = _case(15, 3, [2, 3, 2], None, 40, 4, 2, 64, "bf16")
    good = nv.prefix_attention(**a, status=st)
    assert st.item() == 0
    for bad in ([0, 2, 1, 3], [1, 2, 5, 7], [0, 2, 5, 9]):
        st.zero_()
        nv.prefix_attention(**dict(a, cu_q=torch.tensor(bad, dtype=torch.int32, device=DEV)), status=st)
        assert st.item() == nv.VIT_ERR_LIMIT, bad
    again = nv.prefix_attention(**a)
    assert torch.equal(again[0], good[0])


@pytest.mark.parametrize("n_q", [1, 150])
def test_offsets_beyond_32_bits(n_q):
    # sequences 2^32 + 64 bytes apart in the keys' cache and 2^31 elements + 64 in the values'
    a, cu = _case(34, 2, n_q, [n_q + 30, n_q + 77], 70, 4, 2, 64, "bf16")
    want = nv.prefix_attention(**a)
    far = dict(a)
    for n, seq in (("k", (1 << 31) + 64), ("v", (1 << 31) + (1 << 30))):
        store = torch.empty(seq + a[n][0].numel(), dtype=torch.bfloat16, device=DEV)
        far[n] = store.as_strided(a[n].shape, (seq,) + a[n].stride()[1:])
        far[n].copy_(a[n])
    got = nv.prefix_attention(**far)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_calls_on_two_streams_at_once():
    a, cu = _case(35, 5, 2, [30, 60, 64, 100, 7], 900, 14, 2, 128, "bf16")
    b, _ = _case(36, 40, 1, [1 + 3 * i for i in range(40)], 700, 28, 4, 128, "bf16")
    want_a, want_b = nv.prefix_attention(**a), nv.prefix_attention(**b)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(nv.prefix_attention(**a, stream=s), nv.prefix_attention(**b, stream=t)) for _ in range(10)]
    torch.cuda.synchronize()
    for ga, gb in got:
        assert torch.equal(ga[0], want_a[0]) and torch.equal(gb[0], want_b[0])


def test_wrong_stream_device_is_refused():
    a, _ = _case(37, 1, 1, [3], 5, 4, 2, 64, "bf16")

    class Elsewhere:
        device = torch.device("cuda", 77)
    with pytest.raises(ValueError):
        nv.prefix_attention(**a, stream=Elsewhere())


def test_lengths_read_by_a_replayed_graph():
    a, cu = _case(16, 4, 1, [3, 60, 64, 100], 500, 14, 2, 128, "bf16", cap=130)
    out = torch.empty_like(a["q"])
    nv.prefix_attention(**a, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = nv.prefix_attention(**a, out=out)
    for step in range(3):
        a["lens"] += 7
        g.replay()
        torch.cuda.synchronize()
        _check(a, cu, got)


def test_other_stream():
    a, cu = _case(17, 4, 2, [30, 60, 64, 100], 300, 14, 2, 128, "bf16")
    want = nv.prefix_attention(**a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = nv.prefix_attention(**a, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_same_bits_every_time():
    a, cu = _case(18, 9, 1, [1 + 50 * i for i in range(9)], 3000, 28, 4, 128, "bf16")
    want = nv.prefix_attention(**a)
    for _ in range(3):
        got = nv.prefix_attention(**a)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_queries():
    a, cu = _case(19, 2, 1, [4, 4], 10, 4, 2, 64, "bf16")
    out, lse = nv.prefix_attention(a["q"][:0], a["prefix_k"], a["prefix_v"])
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_decoder_step_end_to_end():
    """Prompt rows -> q, k, v -> head norm and rotation -> image prefix shared by three questions: the
    framework's steps in a row against the oracle's, one long sequence per question."""
    from oracle import decoder_oracle as do
    from oracle import mrope_oracle as mo
    rng = np.random.default_rng(20)
    H, Hk, D, C, vocab, B, n = 6, 2, 64, 256, 1000, 3, 9
    sec = (8, 12, 12)
    grid = [(1, 16, 16)]
    pre = [1, 2, mo.VISION_START] + [do.IMAGE_TOKEN_ID] * 64 + [mo.VISION_END, 4]
    pre_ids = np.array(pre)
    pre_ids[[2, -2]] = [7, 8]                                      # embeddable ids for the embedding step
    qs = rng.integers(0, vocab, size=(B, n))
    pos, delta = mo.mrope_index(pre, grid)
    P = len(pre)

    def dev(x, t=torch.bfloat16):
        return torch.from_numpy(np.ascontiguousarray(x)).to(DEV).to(t)
    table, vis = dev(rng.normal(size=(vocab, C))), dev(rng.normal(size=(64, C)))
    w = dev(rng.normal(size=((H + 2 * Hk) * D, C)) / C ** 0.5)
    qw, kw = dev(1 + 0.1 * rng.normal(size=D)), dev(1 + 0.1 * rng.normal(size=D))
    ids = np.concatenate([pre_ids, qs.reshape(-1)]).astype(np.int32)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    rows = nv.embed_vision_tokens(torch.from_numpy(ids).to(DEV), table, vis, scale=0.5, status=st)
    qkv = rows @ w.t()
    q_pos = np.broadcast_to(P + delta + np.arange(n), (B, n)).reshape(-1)
    allpos = np.concatenate([pos, np.stack([q_pos] * 3)], 1).astype(np.int32)
    L = len(ids)
    q, k = qkv[:, :H * D].view(L, H, D), qkv[:, H * D:(H + Hk) * D].view(L, Hk, D)
    v = qkv[:, (H + Hk) * D:].view(L, Hk, D)
    q, k = nv.mrope_norm_apply(q, k, torch.from_numpy(allpos).to(DEV), qw, kw, sections=sec)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    out, lse = nv.prefix_attention(q[P:], k[:P], v[:P], k[P:].view(B, n, Hk, D), v[P:].view(B, n, Hk, D), lens, max_q=n,
                                   status=st)
    assert st.item() == 0
    # the oracle on the framework's rounded inputs of each step
    r_rows = oo.embed_rows(ids, _np(table), _np(vis), 0.5)
    assert np.abs(_np(rows) - r_rows).max() <= 2.0 ** -8 * np.abs(r_rows).max()
    x = _np(qkv)
    rq = oo.norm_rope(x[:, :H * D].reshape(L, H, D), _np(qw), allpos, sec)
    rk = oo.norm_rope(x[:, H * D:(H + Hk) * D].reshape(L, Hk, D), _np(kw), allpos, sec)
    rv = x[:, (H + Hk) * D:].reshape(L, Hk, D)
    vmax = np.abs(rv).max()
    for b in range(B):
        at = np.concatenate([np.arange(P), P + b * n + np.arange(n)])
        ref, _ = oo.prefix_attention(rq[at][P:], None, None, rk[at][None], rv[at][None], [P + n], [0, n], D ** -0.5)
        # q and k rounded to bf16 move a score by 2 * 2^-8 * sum|q k| * scale <= 2^-7 * 64^0.5 * max rms product ~ 0.08;
        # the weights by 8%, the output by 2 * 0.08 * max|v| at the very most
        assert np.abs(_np(out[b * n:(b + 1) * n]) - ref).max() <= 0.16 * vmax
        same, _ = oo.prefix_attention(_np(q)[at][P:], None, None, _np(k)[at][None], rv[at][None], [P + n], [0, n], D ** -0.5)
        assert np.abs(_np(out[b * n:(b + 1) * n]) - same).max() <= (2 * 2.0 ** -8 + 4e-4) * vmax


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("H, Hk, D", [(28, 4, 128), (8, 8, 64), (10, 2, 80), (3, 1, 24), (6, 2, 104)])
@pytest.mark.parametrize("B, n_q, Lp", [(40, 1, 700), (9, 31, 333), (3, 100, 161)])
def test_many_rows(B, n_q, Lp, H, Hk, D, t):
    # enough rows for the tensor-core tiles: stacked decoding, and sequences of their own
    lens = [n_q + (13 * b) % 90 for b in range(B)]
    a, cu = _case(30, B, n_q, lens, Lp, H, Hk, D, t, cap=n_q + 95)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    _check(a, cu, nv.prefix_attention(**a, status=st))
    assert st.item() == 0


@pytest.mark.parametrize("n_q, lens", [([256, 1, 257], [256, 400, 257]), ([129], [300]), ([65, 200, 1, 0], [65, 200, 79, 80])])
def test_long_questions_of_single_heads(n_q, lens):
    a, cu = _case(31, len(n_q), n_q, lens, 0, 2, 2, 64, "bf16", cap=max(lens) + 1)
    _check(a, cu, nv.prefix_attention(**a))
    a, cu = _case(32, len(n_q), n_q, lens, 81, 2, 2, 128, "fp16", cap=max(lens) + 1)
    _check(a, cu, nv.prefix_attention(**a, causal=False), causal=False)


def test_dimensions_of_one_element_have_any_stride():
    a, cu = _case(33, 1, 1, [1], 1, 4, 1, 64, "bf16")
    want = nv.prefix_attention(**a)
    b = dict(a, prefix_k=a["prefix_k"].as_strided((1, 1, 64), (1, 3, 1)), k=a["k"].as_strided((1, 1, 1, 64), (0, 7, 1, 1)))
    got = nv.prefix_attention(**b)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_prefix_and_sequences_on_the_tensor_cores_twice_at_once():
    # both launches of a call take tensor memory, and the second starts beside the first; so do another stream's
    cases = [_case(40 + i, 12, 200, [200 + 9 * b for b in range(12)], 2001, 12, 2, 64, "bf16") for i in range(2)]
    streams = [torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = nv.prefix_attention(**cases[i][0])
    torch.cuda.synchronize()
    for (a, cu), g in zip(cases, got):
        _check(a, cu, g)


@pytest.mark.parametrize("B, Lp, H, Hk, D", [(1, 200, 12, 2, 128), (40, 700, 28, 4, 64), (3, 2000, 8, 1, 128)])
@pytest.mark.parametrize("graph", [False, True])
def test_calls_follow_what_the_stream_did_before(B, Lp, H, Hk, D, graph):
    # launches may start early: inputs written by a slow kernel just before the call, each call's output the next
    # one's queries, buffers overwritten behind it
    a, cu = _case(50, B, 1, [30 + b for b in range(B)], Lp, H, Hk, D, "bf16")
    want = [nv.prefix_attention(**a)]
    torch.cuda.synchronize()
    for _ in range(3):
        want.append(nv.prefix_attention(**dict(a, q=want[-1][0])))
        torch.cuda.synchronize()
    slow = torch.zeros(64 << 20, dtype=torch.float32, device=DEV)
    b = {n: torch.zeros_like(t) if isinstance(t, torch.Tensor) else t for n, t in a.items()}
    got = [(torch.zeros_like(a["q"]), torch.zeros(B, H, device=DEV)) for _ in range(4)]

    def chain():
        slow.add_(1.0)
        for n, t in a.items():
            if isinstance(t, torch.Tensor):
                b[n].copy_(t)
        for i, (out, lse) in enumerate(got):
            nv.prefix_attention(**dict(b, q=b["q"] if i == 0 else got[i - 1][0]), out=out, lse=lse)
        for n, t in a.items():
            if isinstance(t, torch.Tensor):
                b[n].zero_()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        chain()
        s.synchronize()
        if graph:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                chain()
        for _ in range(5):
            for out, lse in got:
                out.zero_()
            g.replay() if graph else chain()
        s.synchronize()
    for (out, lse), (w, wl) in zip(got, want):
        assert torch.equal(out, w) and torch.equal(lse, wl)
