"""fp64 CPU oracle of the decode-step calls -- test infrastructure only.

Only ``tests/`` may import this module; it shares no code with the CUDA library.  Each function
computes the definition that include/gdn.h states for its call, one request, token or head at a
time (the single-token form of the core needs none: it is ``oracle.fwd`` with T = 1).
"""
from __future__ import annotations

import numpy as np


def attn_decode(q, k_cache, v_cache, block_table, seq_len, scale=None):
    """o [B,Hq,D], lse [B,Hq] of q [B,Hq,D] over caches [pages,P,Hk,D]; a page outside the cache
    leaves its tokens out, a length outside [0, max_blocks P] is clamped."""
    q = np.asarray(q, dtype=np.float64)
    B, Hq, D = q.shape
    pages, P, Hk, _ = k_cache.shape
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    o, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    for b in range(B):
        n = min(max(int(seq_len[b]), 0), block_table.shape[1] * P)
        rows = [(int(block_table[b, j // P]), j % P) for j in range(n)]
        rows = [r for r in rows if 0 <= r[0] < pages]
        if not rows:
            continue
        at = tuple(np.array(rows).T)
        k, v = k_cache[at].astype(np.float64), v_cache[at].astype(np.float64)  # [n, Hk, D]
        for h in range(Hq):
            s = k[:, h // (Hq // Hk)] @ q[b, h] * scale
            m = s.max()
            e = np.exp(s - m)
            lse[b, h] = m + np.log(e.sum())
            o[b, h] = e @ v[:, h // (Hq // Hk)] / e.sum()
    return o, lse


def _pairs(R, interleaved):
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def rotate(n, positions, inv_freq, interleaved, rope_scale=1.0, transpose=False):
    """The rotation of the first 2 len(inv_freq) elements of n [N, H, D] (or its transpose)."""
    inv_freq = np.asarray(inv_freq, dtype=np.float64)
    ang = np.asarray(positions, dtype=np.float64)[:, None, None] * inv_freq
    c, s = rope_scale * np.cos(ang), rope_scale * np.sin(ang) * (-1 if transpose else 1)
    a, b = _pairs(2 * len(inv_freq), interleaved)
    y = n.copy()
    y[..., a] = n[..., a] * c - n[..., b] * s
    y[..., b] = n[..., b] * c + n[..., a] * s
    return y


def norm_rope_fwd(x, w, positions, inv_freq, interleaved=False, eps=1e-6, rope_scale=1.0):
    """y [N,H,D] of x [N,H,D]."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * w
    return rotate(n, positions, inv_freq, interleaved, rope_scale)


def norm_rope_bwd(x, w, positions, inv_freq, dy, interleaved=False, eps=1e-6, rope_scale=1.0):
    """(dx [N,H,D], dw [D])."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    dn = rotate(np.asarray(dy, dtype=np.float64), positions, inv_freq, interleaved, rope_scale,
                transpose=True)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    g = dn * w
    dx = r * (g - x * r * np.mean(g * x * r, axis=-1, keepdims=True))
    return dx, np.sum(dn * x * r, axis=(0, 1))


def slot_map(ctx_len, new_len, free_pages, block_table, page_size, pages, n_tokens):
    """(seq_len, cu_seqlens, positions, slots, block_table, used), token by token."""
    P, table = page_size, np.array(block_table)
    pos, slots = np.zeros(n_tokens, np.int64), np.full(n_tokens, -1, np.int64)
    seq, cu, taken, t = [], [0], 0, 0
    cap = table.shape[1] * P
    for b, (c, n) in enumerate(zip(ctx_len, new_len)):
        c, n = max(int(c), 0), max(int(n), 0)
        n = min(n, n_tokens - t)  # tokens without a row are not part of the step
        held = -(-c // P)
        for p in range(c, c + n):
            i = p // P
            if p % P == 0 and i < table.shape[1]:  # the first row of a page that it does not have
                page = int(free_pages[taken]) if taken < len(free_pages) else -1
                taken += 1
                table[b, i] = page if 0 <= page < pages else -1
            page = int(table[b, i]) if i < table.shape[1] else -1
            pos[t] = p
            slots[t] = page * P + p % P if 0 <= page < pages else -1
            t += 1
        assert held <= -(-(c + n) // P)
        seq.append(min(c + n, cap))
        cu.append(cu[-1] + n)
    return np.array(seq), np.array(cu), pos, slots, table, taken
