"""CPU oracle (fp64, numpy) for the decoder-side steps with gradients and for attention over a shared
prefix: per-head norm with M-RoPE, the scaled input rows, and prefix attention.

TEST INFRASTRUCTURE ONLY; it shares no code with the CUDA path. The rotation, the token rules and
their sources are those of ``oracle/decoder_oracle.py``; the pages say nothing about head norms,
gradients or a shared prefix, so the definitions stand here:

* norm: n = x / sqrt(mean(x^2) + eps) * w over the head dim, then the rotation R of decoder_oracle;
  gradient by the chain rule: dn = R^T dy, dw = sum over tokens and heads of dn * x / rms,
  dx = (dn w - x mean(dn w x) / rms^2) / rms.
* input rows: scale * embedding for text, vision tokens unscaled at the placeholders; the gradient adds
  scale * d_out to the row each text id names and hands the placeholders' rows to the vision tokens.
* prefix attention: query j of sequence b sees every prefix key and its sequence's own keys s < len,
  with a causal mask s <= len - n + j; softmax over all of them together; no key: zeros, lse -inf.
"""
from __future__ import annotations

import numpy as np

from . import decoder_oracle as do


def norm_rope(x, w, pos, sections, theta=do.MROPE_THETA, eps=1e-6):
    x = np.asarray(x, np.float64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, np.float64)
    rms = np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    return do.mrope_apply(x / rms * w, pos, sections, theta)


def norm_rope_grad(dy, x, w, pos, sections, theta=do.MROPE_THETA, eps=1e-6):
    """(dx, dw) of sum(dy * norm_rope(x, w))."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, np.float64)
    dn = do.mrope_apply(dy, -np.asarray(pos, np.float64), sections, theta)      # R^T turns back
    rms = np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    g = dn * w
    dx = (g - x * (g * x).mean(-1, keepdims=True) / rms ** 2) / rms
    return dx, (dn * x / rms).sum((0, 1))


def embed_rows(ids, table, vision, scale):
    ids = np.asarray(ids)
    slots = (ids == do.IMAGE_TOKEN_ID) | (ids == do.VIDEO_TOKEN_ID)
    out = np.empty((ids.size, table.shape[1]), np.float64)
    out[~slots] = scale * np.asarray(table, np.float64)[ids[~slots]]
    if slots.any():
        out[slots] = np.asarray(vision, np.float64)
    return out


def embed_rows_grad(ids, d_out, vocab, scale):
    """(d_table, d_vision)."""
    ids, d_out = np.asarray(ids), np.asarray(d_out, np.float64)
    slots = (ids == do.IMAGE_TOKEN_ID) | (ids == do.VIDEO_TOKEN_ID)
    d_table = np.zeros((vocab, d_out.shape[1]))
    np.add.at(d_table, ids[~slots], scale * d_out[~slots])
    return d_table, d_out[slots]


def prefix_attention(q, prefix_k, prefix_v, k, v, lens, cu_q, scale, causal=True):
    """(out [T, H, D], lse [T, H]); k, v [B, cap, Hk, D] and lens may be None."""
    q = np.asarray(q, np.float64)
    T, H, D = q.shape
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    Hk = (prefix_k if prefix_k is not None else k).shape[-2]
    for b in range(len(cu_q) - 1):
        n = cu_q[b + 1] - cu_q[b]
        L = 0 if k is None else int(lens[b])
        keys, vals = np.zeros((0, Hk, D)), np.zeros((0, Hk, D))
        if prefix_k is not None:
            keys, vals = np.asarray(prefix_k, np.float64), np.asarray(prefix_v, np.float64)
        n_pre = len(keys)
        if L:
            keys = np.concatenate([keys, np.asarray(k[b, :L], np.float64)])
            vals = np.concatenate([vals, np.asarray(v[b, :L], np.float64)])
        for j in range(n):
            seen = n_pre + (max(0, min(L, L - n + j + 1)) if causal else L)
            if seen == 0:
                continue
            for h in range(H):
                g = h // (H // Hk)
                s = scale * keys[:seen, g] @ q[cu_q[b] + j, h]
                m = s.max()
                p = np.exp(s - m)
                out[cu_q[b] + j, h] = p @ vals[:seen, g] / p.sum()
                lse[cu_q[b] + j, h] = m + np.log(p.sum())
    return out, lse
