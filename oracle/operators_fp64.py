"""Plain fp64 CPU oracle of the passes around attention.

TEST INFRASTRUCTURE ONLY, like ``attention_fp64``: NumPy float64, written from the formulas in
``include/fa.h``, one head, one request and one token at a time; no code shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from .attention_fp64 import attention_head, depage, to_f64

__all__ = ["norm_rope", "norm_rope_bwd", "norm_rope_append", "decode_shared", "decode_scored", "evict"]


def _angles(positions, inv_freq, sections):
    """[B, N, pairs] angles; positions [axes, B, N]."""
    pos, freq = np.asarray(positions, dtype=np.float64), to_f64(inv_freq)
    axis = np.repeat(np.arange(len(sections)), sections)
    return np.stack([pos[a] * f for a, f in zip(axis, freq)], axis=-1)


def _pair_index(pairs, interleaved):
    i = np.arange(pairs)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)


def _turn(y, t, interleaved):
    """y [B,H,N,d] with its pairs turned by t [B,N,pairs]."""
    a, b = _pair_index(t.shape[-1], interleaved)
    c, s = np.cos(t)[:, None], np.sin(t)[:, None]
    out = y.copy()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., a] * s + y[..., b] * c
    return out


def norm_rope(x, w, positions, inv_freq, sections, interleaved, eps):
    """One of q or k: x [B,H,N,d], w [d] or None -> the normed and turned rows."""
    x = to_f64(x)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * to_f64(w)
    return _turn(x, _angles(positions, inv_freq, sections), interleaved)


def norm_rope_bwd(dy, x, w, positions, inv_freq, sections, interleaved, eps):
    """-> (dx, dw): the transpose of the turn is the turn back; then the norm's gradient by the quotient
    rule, dx_c = sum_j h_j d(x_j r)/dx_c with d(x_j r)/dx_c = r delta_jc - x_j x_c r^3 / d."""
    g = _turn(to_f64(dy), -_angles(positions, inv_freq, sections), interleaved)
    if w is None:
        return g, None
    x, w = to_f64(x), to_f64(w)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = g * w
    dx = h * r - x * r**3 * (h * x).sum(-1, keepdims=True) / x.shape[-1]
    return dx, (g * x * r).reshape(-1, x.shape[-1]).sum(0)


def norm_rope_append(q, k, v, wq, wk, positions, inv_freq, sections, interleaved, eps, k_cache, v_cache, block_table,
                     ctx_lens, q_lens, q_out, block_size):
    """-> (q_out, k_cache, v_cache) after the call; copies, fp64."""
    qo, kc, vc = to_f64(q_out).copy(), to_f64(k_cache).copy(), to_f64(v_cache).copy()
    qn = norm_rope(q, wq, positions, inv_freq, sections, interleaved, eps)
    kn = norm_rope(k, wk, positions, inv_freq, sections, interleaved, eps)
    vv, table = to_f64(v), np.asarray(block_table)
    for r, (L, m) in enumerate(zip(np.asarray(ctx_lens), np.asarray(q_lens))):
        for i in range(m):
            at = L - m + i
            block = table[r, at // block_size]
            qo[r, :, i] = qn[r, :, i]
            kc[block, :, at % block_size] = kn[r, :, i]
            vc[block, :, at % block_size] = vv[r, :, i]
    return qo, kc, vc


def _decode(q, keys, values, scale):
    """Heads q [Hq,d] over keys, values [Hkv][n,d] -> (o [Hq,d], lse [Hq], weights [Hkv,n])."""
    Hq, G = q.shape[0], q.shape[0] // len(keys)
    o, lse = np.zeros_like(q), np.full(Hq, -np.inf)
    w = np.zeros((len(keys), keys[0].shape[0]))
    for h in range(Hq):
        if keys[0].shape[0] == 0:
            continue
        oh, lh, ph = attention_head(q[h][None], keys[h // G], values[h // G], scale)
        o[h], lse[h] = oh[0], lh[0]
        w[h // G] += ph[0]
    return o, lse, w


def decode_shared(q, k_cache, v_cache, prefix_table, prefix_len, block_table, ctx_lens, block_size, scale):
    q, table = to_f64(q), np.asarray(block_table)
    k_cache, v_cache = to_f64(k_cache), to_f64(v_cache)
    Hkv, P = k_cache.shape[1], int(prefix_len)
    pre = [[depage(c, np.asarray(prefix_table), P, g, block_size) for g in range(Hkv)] for c in (k_cache, v_cache)]
    o, lse = np.empty_like(q), np.empty(q.shape[:2])
    for r, n in enumerate(np.asarray(ctx_lens)):
        kv = [[np.concatenate([pre[i][g], depage(c, table[r], int(n), g, block_size)]) for g in range(Hkv)]
              for i, c in enumerate((k_cache, v_cache))]
        o[r], lse[r], _ = _decode(q[r], kv[0], kv[1], scale)
    return o, lse


def decode_scored(q, k_cache, v_cache, block_table, ctx_lens, weights, block_size, scale):
    q, table, w = to_f64(q), np.asarray(block_table), to_f64(weights).copy()
    k_cache, v_cache = to_f64(k_cache), to_f64(v_cache)
    o, lse = np.empty_like(q), np.empty(q.shape[:2])
    for r, n in enumerate(np.asarray(ctx_lens)):
        kv = [[depage(c, table[r], int(n), g, block_size) for g in range(k_cache.shape[1])] for c in (k_cache, v_cache)]
        o[r], lse[r], p = _decode(q[r], kv[0], kv[1], scale)
        w[r, :, :n] += p
    return o, lse, w


def evict(k_cache, v_cache, block_table, ctx_lens, seq_lens, weights, slot_pos, keep, recent, block_size):
    """-> (k_cache, v_cache, new_ctx, weights, slot_pos) after the call."""
    kc, vc, table = to_f64(k_cache).copy(), to_f64(v_cache).copy(), np.asarray(block_table)
    w_in, p_in = to_f64(weights), np.asarray(slot_pos)
    w_out, p_out = np.zeros_like(w_in), np.full(p_in.shape, -1, dtype=np.int32)
    new_ctx = np.minimum(np.asarray(ctx_lens), keep).astype(np.int32)
    for r, (n, seq) in enumerate(zip(np.asarray(ctx_lens).tolist(), np.asarray(seq_lens).tolist())):
        for h in range(kc.shape[1]):
            pos = [int(p_in[r, h, s]) if p_in[r, h, s] >= 0 else seq - n + s for s in range(n)]

            def rank(s):
                w = w_in[r, h, s]
                if pos[s] >= seq - recent:
                    return (0, 0.0, s)
                return (2, 0.0, s) if np.isnan(w) else (1, -w, s)

            kept = sorted(sorted(range(n), key=rank)[:keep])
            at = {s: s for s in kept if s < keep}
            free = [s for s in range(min(n, keep)) if s not in at]
            at.update(zip([s for s in kept if s >= keep], free))
            old_k, old_v = kc[:, h].copy(), vc[:, h].copy()
            for s, t in at.items():
                a, b = (table[r, s // block_size], s % block_size), (table[r, t // block_size], t % block_size)
                kc[b[0], h, b[1]], vc[b[0], h, b[1]] = old_k[a], old_v[a]
                w_out[r, h, t], p_out[r, h, t] = w_in[r, h, s], pos[s]
    return kc, vc, new_ctx, w_out, p_out
