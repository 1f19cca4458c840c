"""Cases for the decoder-side operators: the q / k head norms fused with the M-RoPE rotation, the scaled
embedding lookup with vision tokens, their gradients, and attention over a prefix that a batch shares.

A case is a dict of plain values. ``prepare`` draws its inputs on the GPU from the seed, ``run`` makes one
pass (the plain torch form, or the framework's kernels where ``own`` is true), ``exact`` is the definition
in 64 bits, ``work`` the bytes and operations that a pass cannot do without.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IMAGE_ID, VIDEO_ID = 151655, 151656      # placeholders of the framework's prompts
TEXT_IDS = 151643                        # text ids lie below
THETA = 1.0e6
EPS = 1e-6


def _sections(head_dim):
    """(16, 24, 24) at head_dim 128, the same proportions elsewhere."""
    half = head_dim // 2
    t = half // 4
    h = (half - t) // 2
    return (t, h, half - t - h)


# ------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of one sequence being decoded: the call's latency
        {"name": "norm_decode_1", "op": "norm", "tokens": 1, "heads": 28, "kv_heads": 4, "head_dim": 128,
         "dtype": "bf16", "packed": True},
        # a batch of long prompts in one packed QKV product
        {"name": "norm_prompts_40961", "op": "norm", "tokens": 40961, "heads": 28, "kv_heads": 4, "head_dim": 128,
         "dtype": "fp16", "packed": True},
        # training on one text / image / video prompt of about 3.2K tokens
        {"name": "norm_grad_3211", "op": "norm_grad", "tokens": 3211, "heads": 28, "kv_heads": 4, "head_dim": 128,
         "dtype": "bf16", "packed": True},
        # a training batch in 32 bits on the narrower decoder
        {"name": "norm_grad_16411_fp32", "op": "norm_grad", "tokens": 16411, "heads": 12, "kv_heads": 2,
         "head_dim": 128, "dtype": "fp32", "packed": False},
        # the input row of a decoding step for a few sequences
        {"name": "embed_decode_3", "op": "embed", "tokens": 3, "vision": 0, "vocab": 152064, "dim": 3584,
         "scale": 1.0, "dtype": "bf16"},
        # a batch of long multi-image prompts
        {"name": "embed_prompts_40007", "op": "embed", "tokens": 40007, "vision": 26112, "vocab": 152064, "dim": 3584,
         "scale": 59.866518188383, "dtype": "bf16"},
        # gradient of the ~3.2K-token image / video prompt's rows, the whole table's gradient written
        {"name": "embed_grad_3211", "op": "embed_grad", "tokens": 3211, "vision": 2560, "vocab": 152064, "dim": 3584,
         "scale": 1.0, "dtype": "bf16", "grad_dtype": "bf16"},
        # a large training batch, table gradient kept in 32 bits
        {"name": "embed_grad_65521", "op": "embed_grad", "tokens": 65521, "vision": 28672, "vocab": 152064,
         "dim": 1536, "scale": 39.191835884531, "dtype": "bf16", "grad_dtype": "fp32"},
        # one question token about one 448 x 448 image: the call's latency
        {"name": "attn_decode_1", "op": "attn", "seqs": 1, "max_q": 1, "ragged": False, "heads": 12, "kv_heads": 2,
         "head_dim": 128, "prefix": 265, "max_len": 21, "dtype": "bf16"},
        # 64 answers being decoded about one 1792 x 1792 image
        {"name": "attn_decode_64", "op": "attn", "seqs": 64, "max_q": 1, "ragged": False, "heads": 28, "kv_heads": 4,
         "head_dim": 128, "prefix": 4113, "max_len": 517, "dtype": "bf16"},
        # 256 answers being decoded about a long video
        {"name": "attn_decode_256", "op": "attn", "seqs": 256, "max_q": 1, "ragged": False, "heads": 28, "kv_heads": 4,
         "head_dim": 128, "prefix": 16405, "max_len": 777, "dtype": "fp16"},
        # 16 questions of different lengths read in one pass after a ~3.2K-token image / video prompt
        {"name": "attn_questions_16", "op": "attn", "seqs": 16, "max_q": 389, "ragged": True, "heads": 28,
         "kv_heads": 4, "head_dim": 128, "prefix": 3209, "max_len": 389, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "embed", "embed_grad", "attn", "attn"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op in ("norm", "norm_grad"):
        heads, kv = rng.choice([(28, 4), (12, 2), (16, 16), (8, 1)])
        head_dim = rng.choice([64, 80, 128])
        most = (40961 * 32 * 128 if op == "norm" else 16411 * 28 * 128) // ((heads + kv) * head_dim)
        return {"op": op, "tokens": _log_int(rng, 1, min(40961, most)), "heads": heads, "kv_heads": kv,
                "head_dim": head_dim, "dtype": dtype, "packed": rng.random() < 0.5}
    if op == "embed":
        tokens = _log_int(rng, 1, 40007)
        return {"op": op, "tokens": tokens, "vision": rng.randint(0, tokens * 3 // 4), "vocab": 152064,
                "dim": rng.choice([256, 1536, 3584]) if dtype != "fp32" else rng.choice([256, 1536]),
                "scale": rng.choice([1.0, 39.191835884531, 59.866518188383]), "dtype": dtype}
    if op == "embed_grad":
        tokens = _log_int(rng, 1, 65521)
        return {"op": op, "tokens": tokens, "vision": rng.randint(0, tokens * 3 // 4), "vocab": 152064,
                "dim": rng.choice([256, 1536]), "scale": rng.choice([1.0, 39.191835884531]), "dtype": dtype,
                "grad_dtype": rng.choice([dtype, "fp32"])}
    heads, kv = rng.choice([(28, 4), (12, 2), (16, 16), (8, 1)])
    dtype = rng.choice(["bf16", "fp16"])
    head_dim = rng.choice([64, 80, 128])
    if rng.random() < 0.5:     # decoding: one token of each sequence, or a few
        seqs, max_q = _log_int(rng, 1, 256), rng.choice([1, 1, 1, 2, 5])
        max_len = _log_int(rng, max_q, 777)
    else:                      # questions of different lengths
        seqs, max_q = _log_int(rng, 1, 16), _log_int(rng, 8, 389)
        max_len = max_q + rng.choice([0, rng.randint(1, 200)])
    prefix = _log_int(rng, 1, 16405)
    while 4 * seqs * max_q * heads * (prefix + max_len) * head_dim > 4 * 256 * 28 * 17182 * 128:
        prefix, max_q = max(1, prefix // 2), max(1, max_q // 2)
    return {"op": "attn", "seqs": seqs, "max_q": max_q, "ragged": max_q > 1 and rng.random() < 0.7, "heads": heads,
            "kv_heads": kv, "head_dim": head_dim, "prefix": prefix, "max_len": max_len, "dtype": dtype}


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _prompt_positions(g, n):
    """(t, h, w) ids as a prompt far along a conversation has them: text counts up on all three axes,
    image runs spread over h and w."""
    start = int(torch.randint(0, 100000, (1,), generator=g, device="cuda"))
    i = torch.arange(n, device="cuda")
    run = i // 1024
    image = run % 2 == 1
    j = i % 1024
    base = start + run * 600
    t = torch.where(image, base, base + j)
    h = torch.where(image, base + j // 32, base + j)
    w = torch.where(image, base + j % 32, base + j)
    return torch.stack([t, h, w]).to(torch.int32).contiguous()


def _prompt_ids(g, n, n_vision):
    """Text ids with the heavy repeats of real text (log-uniform ranks), placeholders in runs."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(TEXT_IDS)) - 1).long().clamp_(0, TEXT_IDS - 1)
    if n_vision:
        # up to 8 runs of placeholders, spread over the prompt
        runs = min(8, n_vision, n - n_vision + 1)
        per = torch.full((runs,), n_vision // runs, dtype=torch.long)
        per[: n_vision % runs] += 1
        gap = (n - n_vision) // (runs + 1)
        begin = gap + torch.cat([torch.zeros(1, dtype=torch.long), torch.cumsum(per + gap, 0)[:-1]])
        i = torch.arange(n)
        r = torch.searchsorted(begin, i, right=True) - 1
        inside = (r >= 0) & (i < begin[r.clamp(min=0)] + per[r.clamp(min=0)])
        kind = torch.where(r % 2 == 0, IMAGE_ID, VIDEO_ID)
        inside, kind = inside.cuda(), kind.cuda()
        ids = torch.where(inside, kind, ids)
    return ids.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        L, H, Hk, D = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"]
        if case["packed"]:     # views of the QKV product's rows
            qkv = _randn(g, (L, (H + 2 * Hk) * D), dt, 1.5)
            s["q"] = qkv[:, : H * D].view(L, H, D)
            s["k"] = qkv[:, H * D: (H + Hk) * D].view(L, Hk, D)
        else:
            s["q"], s["k"] = _randn(g, (L, H, D), dt, 1.5), _randn(g, (L, Hk, D), dt, 1.5)
        s["q_weight"] = (1 + _randn(g, (D,), torch.float32, 0.1)).to(dt)
        s["k_weight"] = (1 + _randn(g, (D,), torch.float32, 0.1)).to(dt)
        s["pos"] = _prompt_positions(g, L)
        s["sections"] = _sections(D)
        if op == "norm_grad":
            s["dq_out"], s["dk_out"] = _randn(g, (L, H, D), dt), _randn(g, (L, Hk, D), dt)
    elif op in ("embed", "embed_grad"):
        L, n_vis, V, C = case["tokens"], case["vision"], case["vocab"], case["dim"]
        s["ids"] = _prompt_ids(g, L, n_vis)
        if op == "embed":
            s["table"] = _randn(g, (V, C), dt, 0.02)
            s["vision"] = _randn(g, (n_vis, C), dt) if n_vis else None
        else:
            s["d_out"] = _randn(g, (L, C), dt, 0.01)
    else:
        B, H, Hk, D = case["seqs"], case["heads"], case["kv_heads"], case["head_dim"]
        mq, cap = case["max_q"], case["max_len"]
        if case["ragged"]:
            # lengths spread over 1 .. max_q (the same total for every seed), in an order of the seed's
            n_q = torch.tensor([mq] + [1 + int(b * 0.6180339887 % 1.0 * mq) for b in range(1, B)], device="cuda")
            n_q = n_q[torch.randperm(B, generator=g, device="cuda")]
            s["cu_q"] = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.cumsum(n_q, 0)]).to(torch.int32)
            total = int(n_q.sum())
        else:
            n_q = torch.full((B,), mq, device="cuda")
            s["cu_q"] = None
            total = B * mq
        # the new tokens' keys are part of the suffix, with 0 .. max_len - n_q earlier ones
        more = (torch.rand(B, generator=g, device="cuda") * (cap - n_q + 1)).long()
        s["lens"] = (n_q + more).to(torch.int32)
        s["q"] = _randn(g, (total, H, D), dt)
        s["prefix_k"], s["prefix_v"] = (_randn(g, (case["prefix"], Hk, D), dt) for _ in range(2))
        s["k"], s["v"] = (_randn(g, (B, cap, Hk, D), dt) for _ in range(2))
    return s


# ------------------------------------------------------------------------------------------ plain forms
def _cos_sin(pos, head_dim, sections):
    axis = torch.repeat_interleave(torch.arange(3, device=pos.device), torch.tensor(sections, device=pos.device),
                                   output_size=head_dim // 2)
    j = torch.arange(head_dim // 2, device=pos.device, dtype=torch.float64)
    ang = pos[axis].t().double() * THETA ** (-2.0 * j / head_dim)
    return torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]      # [L, 1, D/2]


def _norm_plain(x, w, c, s):
    xf = x.float()
    half = x.shape[-1] // 2
    y = xf * torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS) * w.float()
    lo, hi = y[..., :half], y[..., half:]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1).to(x.dtype)


def _norm_grad_plain(dy, x, w, c, s):
    dyf, xf = dy.float(), x.float()
    half = x.shape[-1] // 2
    lo, hi = dyf[..., :half], dyf[..., half:]
    dn = torch.cat([lo * c + hi * s, hi * c - lo * s], -1)
    r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
    xh = xf * r
    dw = (dn * xh).sum((0, 1), dtype=torch.float64).float()
    gr = dn * w.float()
    dx = r * (gr - xh * (gr * xh).mean(-1, keepdim=True))
    return dx.to(x.dtype), dw


def _embed_plain(ids, table, vision, scale):
    slot = (ids == IMAGE_ID) | (ids == VIDEO_ID)
    out = (table[ids.long()].float() * scale).to(table.dtype)
    if vision is not None:
        rank = torch.cumsum(slot, 0) - 1
        out = torch.where(slot[:, None], vision[rank.clamp(0, vision.shape[0] - 1)], out)
    return out


def _embed_grad_plain(ids, d_out, vocab, n_vision, scale, grad_dtype):
    slot = (ids == IMAGE_ID) | (ids == VIDEO_ID)
    text = torch.where(slot[:, None], 0.0, d_out.float())
    d_table = torch.zeros((vocab, d_out.shape[1]), dtype=torch.float32, device=d_out.device)
    d_table.index_add_(0, ids.long(), text)
    first = torch.argsort(slot.int(), descending=True, stable=True)[:n_vision]
    return d_table.mul_(scale).to(grad_dtype), d_out[first]


def _attn_plain(q, prefix_k, prefix_v, k, v, lens, cu_q, max_q):
    T, H, D = q.shape
    B, cap, Hk, _ = k.shape
    G, Lp = H // Hk, prefix_k.shape[0]
    scale = 1.0 / math.sqrt(D)
    dev = q.device
    cu = cu_q.long() if cu_q is not None else torch.arange(B + 1, device=dev) * max_q
    n_q = cu[1:] - cu[:-1]
    j = torch.arange(max_q, device=dev)
    slot = (cu[:-1, None] + j).clamp(max=T - 1)                                   # [B, max_q] -> token
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu, t, right=True) - 1
    back = seq * max_q + t - cu[seq]                                              # token -> padded row
    qf = q.float().view(T, Hk, G, D)
    # prefix: every query of the batch against the same keys
    sp = torch.matmul(qf.permute(1, 0, 2, 3).reshape(Hk, T * G, D), prefix_k.float().permute(1, 2, 0)) * scale
    sp = sp.view(Hk, T, G, Lp)
    # suffix: each sequence's queries against its own keys
    qp = qf[slot]                                                                 # [B, max_q, Hk, G, D]
    qp = qp.permute(0, 2, 1, 3, 4).reshape(B, Hk, max_q * G, D)
    ss = torch.matmul(qp, k.float().permute(0, 2, 3, 1)) * scale
    ss = ss.view(B, Hk, max_q, G, cap)
    last = lens.long()[:, None] - n_q[:, None] + j                                # last visible key
    seen = torch.arange(cap, device=dev) <= last[..., None]                       # [B, max_q, cap]
    ss = torch.where(seen[:, None, :, None], ss, -math.inf)
    st = ss.permute(1, 0, 2, 3, 4).reshape(Hk, B * max_q, G, cap)[:, back]        # [Hk, T, G, cap]
    m = torch.maximum(sp.amax(-1), st.amax(-1))
    safe = torch.where(torch.isinf(m), 0.0, m)[..., None]
    pp, pt = torch.exp(sp - safe), torch.exp(st - safe)
    l = pp.sum(-1) + pt.sum(-1)
    o = torch.matmul(pp.view(Hk, T * G, Lp), prefix_v.float().permute(1, 0, 2)).view(Hk, T, G, D)
    ptp = torch.zeros((Hk, B * max_q, G, cap), device=dev)
    ptp[:, back] = pt
    ot = torch.matmul(ptp.view(Hk, B, max_q * G, cap), v.float().permute(2, 0, 1, 3))
    o = o + ot.view(Hk, B * max_q, G, D)[:, back]
    o = o / torch.where(l > 0, l, 1.0)[..., None]
    lse = m + torch.log(l)
    return o.permute(1, 0, 2, 3).reshape(T, H, D).to(q.dtype), lse.permute(1, 0, 2).reshape(T, H)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        c, sn = _cos_sin(s["pos"], case["head_dim"], s["sections"])
        return _norm_plain(s["q"], s["q_weight"], c, sn), _norm_plain(s["k"], s["k_weight"], c, sn)
    if op == "norm_grad":
        c, sn = _cos_sin(s["pos"], case["head_dim"], s["sections"])
        dq, dqw = _norm_grad_plain(s["dq_out"], s["q"], s["q_weight"], c, sn)
        dk, dkw = _norm_grad_plain(s["dk_out"], s["k"], s["k_weight"], c, sn)
        return dq, dk, dqw, dkw
    if op == "embed":
        return _embed_plain(s["ids"], s["table"], s["vision"], case["scale"])
    if op == "embed_grad":
        return _embed_grad_plain(s["ids"], s["d_out"], case["vocab"], case["vision"], case["scale"],
                                 DTYPES[case["grad_dtype"]])
    return _attn_plain(s["q"], s["prefix_k"], s["prefix_v"], s["k"], s["v"], s["lens"], s["cu_q"], case["max_q"])


def _run_own(s):
    from resolution_vit_vision_b200 import native as nv
    case = s["case"]
    op = case["op"]
    if op == "norm":
        return nv.mrope_norm_apply(s["q"], s["k"], s["pos"], s["q_weight"], s["k_weight"], eps=EPS, theta=THETA,
                                   sections=s["sections"])
    if op == "norm_grad":
        return nv.mrope_norm_grad(s["dq_out"], s["dk_out"], s["q"], s["k"], s["pos"], s["q_weight"], s["k_weight"],
                                  eps=EPS, theta=THETA, sections=s["sections"])
    if op == "embed":
        return nv.embed_vision_tokens(s["ids"], s["table"], s["vision"], scale=case["scale"])
    if op == "embed_grad":
        return nv.embed_vision_tokens_grad(s["ids"], s["d_out"], case["vocab"], case["vision"], scale=case["scale"],
                                           table_dtype=DTYPES[case["grad_dtype"]])
    return nv.prefix_attention(s["q"], s["prefix_k"], s["prefix_v"], s["k"], s["v"], s["lens"], cu_q=s["cu_q"],
                               max_q=case["max_q"])


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    e = size[case["dtype"]]
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["head_dim"]
        if op == "norm":
            return {"bytes": 2 * n * e + 12 * case["tokens"], "flops": 8 * n}
        return {"bytes": 3 * n * e + 12 * case["tokens"], "flops": 16 * n}
    if op == "embed":
        n = case["tokens"] * case["dim"]
        return {"bytes": 2 * n * e + 4 * case["tokens"], "flops": n}
    if op == "embed_grad":
        n = case["tokens"] * case["dim"]
        return {"bytes": n * e + case["vision"] * case["dim"] * e + case["vocab"] * case["dim"] * size[case["grad_dtype"]]
                + 4 * case["tokens"], "flops": n}
    B, H, Hk, D, Lp, mq = (case[x] for x in ("seqs", "heads", "kv_heads", "head_dim", "prefix", "max_q"))
    n_q = (mq + 1) / 2 if case["ragged"] else mq                  # averages over the drawn lengths
    length = n_q + (case["max_len"] - n_q) / 2
    rows = B * n_q
    seen = length - (n_q - 1) / 2
    return {"bytes": int(rows * H * (2 * D * e + 4) + 2 * (Lp + B * length) * Hk * D * e),
            "flops": int(4 * rows * H * D * (Lp + seen))}


# ------------------------------------------------------------------------------------------ 64 bits
def _norm64(x, w, pos, sections):
    """Norm, then each pair (j, j + D/2) as a complex number times e^(i angle)."""
    D = x.shape[-1]
    n = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / D + EPS) * w
    z = torch.complex(n[..., : D // 2], n[..., D // 2:])
    parts = torch.split(torch.tensor([THETA ** (-2.0 * j / D) for j in range(D // 2)], dtype=torch.float64,
                                     device=x.device), list(sections))
    ang = torch.cat([pos[a].double()[:, None] * f for a, f in enumerate(parts)], 1)
    z = z * torch.polar(torch.ones_like(ang), ang)[:, None]
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        grad = op == "norm_grad"
        found = []
        for x, w, dy in (("q", "q_weight", "dq_out"), ("k", "k_weight", "dk_out")):
            xd = s[x].double().requires_grad_(grad)
            wd = s[w].double().requires_grad_(grad)
            y = _norm64(xd, wd, s["pos"], s["sections"])
            found.append(torch.autograd.grad(y, (xd, wd), s[dy].double()) if grad else y)
        if not grad:
            return tuple(found)
        return found[0][0], found[1][0], found[0][1], found[1][1]
    if op == "embed":
        ids = s["ids"].long()
        out = s["table"].double().index_select(0, ids) * case["scale"]
        slots = torch.nonzero((ids == IMAGE_ID) | (ids == VIDEO_ID))[:, 0]
        if len(slots):
            out[slots] = s["vision"].double()
        return out
    if op == "embed_grad":
        ids = s["ids"].long()
        vis = (ids == IMAGE_ID) | (ids == VIDEO_ID)
        slots, text = torch.nonzero(vis)[:, 0], torch.nonzero(~vis)[:, 0]
        d = torch.zeros((case["vocab"], case["dim"]), dtype=torch.float64, device="cuda")
        d.index_put_((ids[text],), s["d_out"][text].double(), accumulate=True)
        return d * case["scale"], s["d_out"][slots].double()
    q, pk, pv, k, v = (s[n].double() for n in ("q", "prefix_k", "prefix_v", "k", "v"))
    B, G = case["seqs"], case["heads"] // case["kv_heads"]
    cu = s["cu_q"].tolist() if s["cu_q"] is not None else [b * case["max_q"] for b in range(B + 1)]
    lens = s["lens"].tolist()
    out, lse = [], []
    for b in range(B):
        n, L = cu[b + 1] - cu[b], lens[b]
        keys = torch.cat([pk, k[b, :L]])[:, :, None].expand(-1, -1, G, -1).flatten(1, 2)      # [N, H, D]
        vals = torch.cat([pv, v[b, :L]])[:, :, None].expand(-1, -1, G, -1).flatten(1, 2)
        x = torch.einsum("qhd,nhd->hqn", q[cu[b]: cu[b + 1]], keys) / case["head_dim"] ** 0.5
        hidden = torch.ones((n, L), dtype=torch.bool, device=q.device).triu(L - n + 1)
        x[:, :, pk.shape[0]:].masked_fill_(hidden, -math.inf)
        out.append(torch.einsum("hqn,nhd->qhd", torch.softmax(x, -1), vals))
        lse.append(torch.logsumexp(x, -1).t())
    return torch.cat(out), torch.cat(lse)
