"""fp64 CPU oracle of the full-attention calls over whole prompts and of the 8-bit cache -- test
infrastructure only.

Only ``tests/`` may import this module; it shares no code with the CUDA library.  Each function
computes the definition that include/gdn.h states for its call: attention and its gradients one
sequence and head at a time, the cache one token at a time, e4m3 numbers from a table.
"""
from __future__ import annotations

import numpy as np

BLOCK = 16


def cut(cu, n):
    """Offsets as they count: outside [0, n] or below an earlier one they are cut or raised."""
    return np.maximum.accumulate(np.clip(np.asarray(cu, dtype=np.int64), 0, n))


def sequences(cu_q, cu_k, Nq, Nk):
    """(query rows, key rows) of every sequence."""
    a, b = cut(cu_q, Nq), cut(cu_k, Nk)
    return [(slice(a[i], a[i + 1]), slice(b[i], b[i + 1])) for i in range(len(a) - 1)]


def seen(nq, nk, causal):
    """[nq, nk]: whether query i sees key j."""
    if not causal:
        return np.ones((nq, nk), bool)
    return np.arange(nk)[None, :] <= np.arange(nq)[:, None] + nk - nq


def attn_fwd(q, k, v, cu_q, cu_k, causal=True, scale=None):
    """o [Nq,Hq,D], lse [Nq,Hq] of q [Nq,Hq,D], k, v [Nk,Hk,D] (rows of no sequence: 0, -inf)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    Nq, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    o, lse = np.zeros(q.shape), np.full((Nq, Hq), -np.inf)
    for rows, keys in sequences(cu_q, cu_k, Nq, len(k)):
        mask = seen(rows.stop - rows.start, keys.stop - keys.start, causal)
        live = mask.any(1)
        if not live.any():
            continue
        for h in range(Hq):
            s = np.where(mask, q[rows, h] @ k[keys, h // G].T * scale, -np.inf)[live]
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            z = e.sum(1, keepdims=True)
            at = np.arange(rows.start, rows.stop)[live]
            o[at, h] = e @ v[keys, h // G] / z
            lse[at, h] = (m + np.log(z))[:, 0]
    return o, lse


def attn_bwd(q, k, v, o, lse, dO, cu_q, cu_k, causal=True, scale=None):
    """(dq, dk, dv) at the given o and lse."""
    q, k, v, o, lse, dO = (np.asarray(x, dtype=np.float64) for x in (q, k, v, o, lse, dO))
    Nq, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)
    for rows, keys in sequences(cu_q, cu_k, Nq, len(k)):
        mask = seen(rows.stop - rows.start, keys.stop - keys.start, causal)
        for h in range(Hq):
            l = lse[rows, h][:, None]
            with np.errstate(invalid="ignore"):
                p = np.where(mask & np.isfinite(l),
                             np.exp(q[rows, h] @ k[keys, h // G].T * scale - l), 0.0)
            dv[keys, h // G] += p.T @ dO[rows, h]
            delta = (dO[rows, h] * o[rows, h]).sum(1, keepdims=True)
            ds = p * (dO[rows, h] @ v[keys, h // G].T - delta) * scale
            dq[rows, h] = ds @ k[keys, h // G]
            dk[keys, h // G] += ds.T @ q[rows, h]
    return dq, dk, dv


def _e4m3_table():
    """Value of every code 0 .. 255: sign, 4 bits of exponent (bias 7), 3 of mantissa; 0x7f, 0xff NaN."""
    out = np.zeros(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = np.nan if c & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = -x if c & 128 else x
    return out


E4M3 = _e4m3_table()


def e4m3_codes(x):
    """The nearest code of each x (|x| <= 448; ties to the even code), NaN where it is not finite."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.abs(np.where(np.isfinite(x), x, 0.0))
    up = np.searchsorted(E4M3[:127], mag)  # the first code that is not below
    lo = np.maximum(up - 1, 0)
    a, b = mag - E4M3[lo], E4M3[np.minimum(up, 126)] - mag
    c = np.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, up)
    c = np.where(np.isfinite(x), c, 127)
    return (c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def block_scale(top):
    """The smallest power of two, 2^-100 at least, that 448 times is not below top."""
    s = 2.0 ** -100
    while 448.0 * s < top:
        s *= 2.0
    return s


def cache_write8(x, cache, scale, block_table, ctx_len, cu_seqlens):
    """One cache's (codes [pages,P,Hk,D] uint8, scales [pages,P/16,Hk]) after the step's packed
    rows x [N,Hk,D], request by request and block by block."""
    x = np.asarray(x, dtype=np.float64)
    cache, scale = np.array(cache), np.array(scale, dtype=np.float64)
    pages, P, Hk, _ = cache.shape
    cu_seqlens = cut(cu_seqlens, len(x))
    for b, ctx in enumerate(ctx_len):
        t, end, pos = int(cu_seqlens[b]), int(cu_seqlens[b + 1]), max(int(ctx), 0)
        while t < end:
            n = min(BLOCK - pos % BLOCK, end - t)
            i = pos // P
            page = int(block_table[b, i]) if i < block_table.shape[1] else -1
            if 0 <= page < pages:
                blk, r = pos % P // BLOCK, pos % P
                for h in range(Hk):
                    new = x[t:t + n, h]
                    fin = np.abs(new[np.isfinite(new)])
                    s = block_scale(fin.max() if fin.size else 0.0)
                    if pos % BLOCK:
                        before = scale[page, blk, h]
                        s = max(s, before)
                        old = E4M3[cache[page, r - pos % BLOCK:r, h]]
                        cache[page, r - pos % BLOCK:r, h] = e4m3_codes(old * (before / s))
                    scale[page, blk, h] = s
                    cache[page, r:r + n, h] = e4m3_codes(new / s)
            t, pos = t + n, pos + n
    return cache, scale


def values(cache, scale):
    """The numbers [pages,P,Hk,D] that codes and scales stand for."""
    return E4M3[np.asarray(cache)] * np.repeat(np.asarray(scale, np.float64), BLOCK, 1)[..., None]


def cache_read8(cache, scale, block_table, cu_seqlens, n_tokens):
    """Packed rows [n_tokens,Hk,D] (NaN where there is no token; 0 where its page is missing)."""
    val = values(cache, scale)
    pages, P, Hk, D = val.shape
    out = np.full((n_tokens, Hk, D), np.nan)
    cu_seqlens = cut(cu_seqlens, n_tokens)
    for b in range(len(cu_seqlens) - 1):
        for j in range(int(cu_seqlens[b + 1]) - int(cu_seqlens[b])):
            i = j // P
            page = int(block_table[b, i]) if i < block_table.shape[1] else -1
            out[cu_seqlens[b] + j] = val[page, j % P] if 0 <= page < pages else 0.0
    return out
