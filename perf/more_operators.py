"""The full-attention layers of a hybrid model over whole prompts, in training and in serving with
a key-value cache held in 8 bits: what is timed, on which inputs, and the plain forms.

- ``fwd`` / ``bwd``  gdn_attn_fwd / gdn_attn_bwd: attention of packed sequences of different
  lengths, causal, query heads grouped on key heads, over the prompt itself or over a longer
  context that it continues; and its gradients.
- ``cache``  gdn_cache_write8, then gdn_cache_read8: a step's keys and values quantised into the
  paged cache (e4m3, a power of two as scale for every 16 tokens and head) and every request's
  whole context read back into packed rows.
- ``dec8``   gdn_attn_decode8: one new token per request over that cache.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn
BLOCK = 16  # tokens that share a scale
ROWS = 2 ** 28  # scores that a plain form holds at a time


def listed():
    return [
        # a short question in an interactive session: one tile per head, latency
        {"name": "fwd_one_short", "op": "fwd", "B": 1, "lo": 97, "hi": 97, "ctx": 0, "Hq": 16,
         "Hk": 2, "D": 256, "causal": True, "dtype": "bf16"},
        # a step that takes a batch of prompts in
        {"name": "fwd_packed", "op": "fwd", "B": 37, "lo": 500, "hi": 4000, "ctx": 0, "Hq": 32,
         "Hk": 8, "D": 128, "causal": True, "dtype": "bf16"},
        # one long document, or a training row of the benchmark's length
        {"name": "fwd_long", "op": "fwd", "B": 1, "lo": 32768, "hi": 32768, "ctx": 0, "Hq": 16,
         "Hk": 2, "D": 256, "causal": True, "dtype": "bf16"},
        # the next turns of conversations whose context is cached
        {"name": "fwd_context", "op": "fwd", "B": 9, "lo": 40, "hi": 600, "ctx": 16000, "Hq": 32,
         "Hk": 8, "D": 128, "causal": True, "dtype": "bf16"},
        # a small model checked in fp32, three query heads to a key head
        {"name": "fwd_fp32", "op": "fwd", "B": 9, "lo": 1, "hi": 700, "ctx": 0, "Hq": 12, "Hk": 4,
         "D": 64, "causal": True, "dtype": "fp32"},
        # training on packed samples
        {"name": "bwd_packed", "op": "bwd", "B": 8, "lo": 1000, "hi": 4000, "ctx": 0, "Hq": 32,
         "Hk": 8, "D": 128, "causal": True, "dtype": "bf16"},
        # training on one long row
        {"name": "bwd_long", "op": "bwd", "B": 1, "lo": 16001, "hi": 16001, "ctx": 0, "Hq": 16,
         "Hk": 2, "D": 256, "causal": True, "dtype": "bf16"},
        # a decode step of a full server: a token each, into blocks that are partly filled
        {"name": "cache_decode", "op": "cache", "B": 250, "lo": 1, "hi": 1, "ctx": 300, "Hk": 2,
         "D": 256, "page": 16, "dtype": "bf16"},
        # a step that takes whole prompts in, some behind a cached context
        {"name": "cache_prefill", "op": "cache", "B": 37, "lo": 500, "hi": 4000, "ctx": 5000,
         "Hk": 8, "D": 128, "page": 64, "dtype": "bf16"},
        # one interactive request early in its answer
        {"name": "dec8_one_short", "op": "dec8", "B": 1, "lo": 517, "hi": 517, "Hq": 16, "Hk": 2,
         "D": 256, "page": 16, "dtype": "bf16"},
        # one request over a long document: the cache's length has to be split
        {"name": "dec8_one_long", "op": "dec8", "B": 1, "lo": 131001, "hi": 131001, "Hq": 32,
         "Hk": 8, "D": 128, "page": 64, "dtype": "bf16"},
        # a full server: bandwidth
        {"name": "dec8_large", "op": "dec8", "B": 128, "lo": 2000, "hi": 16000, "Hq": 16, "Hk": 2,
         "D": 256, "page": 32, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "cache", "dec8", "dec8"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    D, Hk = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8])
    case = {"op": op, "Hk": Hk, "D": D, "dtype": dtype}
    if op in ("fwd", "bwd"):
        Hq = Hk * rng.choice([1, 2, 3, 4, 8])
        # the scores' products stay below those of the largest listed cases; in fp32, which no
        # tensor core does at full rate, far below
        most = (2 ** 36 if op == "fwd" else 2 ** 34) if dtype == "bf16" else 2 ** 30
        hi = _spread(rng, 16, min(16384, int(math.sqrt(most / (Hq * D / 64)))))
        ctx = rng.choice([0, 0, 0, hi, 4 * hi])
        B = _spread(rng, 1, max(1, min(64, int(most / (Hq * D / 64) / (hi * (hi + ctx))),
                                       2 ** 27 // ((Hq + 2 * Hk) * D * (hi + ctx)))))
        case.update(B=B, lo=rng.choice([0, 1, max(1, hi // 2), hi]), hi=hi, ctx=ctx, Hq=Hq,
                    causal=rng.random() < 0.8)
    elif op == "cache":
        hi = rng.choice([1, 4, 700, 3500])
        B = _spread(rng, 1, 500 if hi < 100 else 30)
        case.update(B=B, lo=rng.choice([0, 1]), hi=hi, page=rng.choice([16, 32, 48, 64, 128]),
                    ctx=_spread(rng, 1, max(2, min(8000, 2 ** 28 // (B * Hk * D)))))
    else:
        B = _spread(rng, 1, 128)
        hi = _spread(rng, 16, min(131072, 2 ** 28 // (B * Hk * D)))
        case.update(B=B, lo=rng.choice([0, 1, max(1, hi // 2)]), hi=hi,
                    Hq=Hk * rng.choice([1, 2, 3, 4, 8, 12]),
                    page=rng.choice([16, 32, 48, 64, 128]))
    return case


# ------------------------------------------------------------------------------ inputs

def _lengths(case, seed):
    """Lengths in [lo, hi], spread over their logarithm, the first of them 1 at least; the same
    ones for every seed (the buffers of a step keep their sizes), in another order."""
    lo, hi = case["lo"], case["hi"]
    r = random.Random(lo * 31 + hi)
    lens = [min(hi, max(lo, int(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1))) - 0.5)))
            for _ in range(case["B"])]
    lens[0] = max(1, lens[0])
    random.Random(seed * 7 + 1).shuffle(lens)
    return lens


def _contexts(case, seed):
    """Tokens in front of each sequence's own, up to ctx, spread evenly; ordered by the seed."""
    r = random.Random(case["ctx"])
    ctx = [r.randint(0, case["ctx"]) if case["ctx"] else 0 for _ in range(case["B"])]
    random.Random(seed * 7 + 2).shuffle(ctx)
    return ctx


def _rand(gen, shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(lens):
    return [0] + np.cumsum(lens).tolist()


def _pages(case, lens, seed):
    """Shuffled pages for requests of these lengths: (table, pages); unused entries hold none."""
    P = case["page"]
    counts = [-(-n // P) for n in lens]
    pages = sum(lens) // P + len(lens) + 3
    perm = np.random.RandomState((seed * 7 + 3) % 2 ** 31).permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(1, max(counts))), -1, dtype=np.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = perm[at:at + c]
        at += c
    return torch.from_numpy(table).cuda(), pages


def _power(exp):
    """2^exp, whole numbers, in 32 bits."""
    return ((exp.int() + 127) << 23).view(torch.float32)


def _cache8(gen, pages, case):
    """A filled cache: codes and power-of-two scales, another size for each head and block."""
    P, Hk, D = case["page"], case["Hk"], case["D"]
    codes = (100.0 * _rand(gen, (pages, P, Hk, D), torch.bfloat16)).clamp(-448, 448).to(F8)
    exp = torch.randint(-9, -5, (pages, P // BLOCK, Hk), generator=gen, device="cuda")
    return codes, _power(exp)


def prepare(case, seed):
    st = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt, Hk, D = case["op"], DT[case["dtype"]], case["Hk"], case["D"]
    if op == "dec8":
        lens = _lengths(case, seed)
        st["block_table"], pages = _pages(case, lens, seed)
        st["k_cache"], st["k_scale"] = _cache8(gen, pages, case)
        st["v_cache"], st["v_scale"] = _cache8(gen, pages, case)
        st["q"] = _rand(gen, (case["B"], case["Hq"], D), dt)
        st["seq_len"], st["top"] = _i32(lens), max(lens)
        return st
    new, ctx = _lengths(case, seed), _contexts(case, seed)
    whole = [c + n for c, n in zip(ctx, new)]
    cu, cu_k = _offsets(new), _offsets(whole)
    st["cu"], st["cu_k"] = _i32(cu), _i32(cu_k)
    st["cu_host"], st["cu_k_host"] = cu, cu_k
    if op == "cache":
        st["block_table"], pages = _pages(case, whole, seed)
        st["k_cache"], st["k_scale"] = _cache8(gen, pages, case)
        st["v_cache"], st["v_scale"] = _cache8(gen, pages, case)
        # heads of different sizes, a few channels far larger than the rest, as keys have them
        size = torch.exp(0.5 * _rand(gen, (Hk, 1))) * torch.where(
            torch.rand((Hk, D), generator=gen, device="cuda") < 0.03, 8.0, 1.0)
        st["k"] = (size * _rand(gen, (cu[-1], Hk, D))).to(dt)
        st["v"] = _rand(gen, (cu[-1], Hk, D), dt)
        st["ctx_len"], st["n"] = _i32(ctx), cu_k[-1]
        return st
    Hq = case["Hq"]
    st["q"] = _rand(gen, (cu[-1], Hq, D), dt)
    kv = _rand(gen, (cu_k[-1], 2 * Hk, D), dt)  # v as a projection leaves it, beside k
    st["k"], st["v"] = kv[:, :Hk].contiguous(), kv[:, Hk:]
    if op == "bwd":
        st["o"], st["lse"] = _fwd(st)
        st["do"] = _rand(gen, (cu[-1], Hq, D), dt)
    return st


# ------------------------------------------------------------------------- plain forms

def _pieces(st):
    """(query rows, key rows, first visible offset) of every sequence, cut into runs of queries
    whose scores fit."""
    cu, ck = st["cu_host"], st["cu_k_host"]
    G = st["Hq"] // st["Hk"]
    for b in range(st["B"]):
        nq, nk = cu[b + 1] - cu[b], ck[b + 1] - ck[b]
        step = max(1, ROWS // max(1, G * nk))
        for r in range(0, nq, step):
            n = min(step, nq - r)
            # keys that no query of the run sees are left out
            seen = max(0, min(nk, r + n + nk - nq)) if st["causal"] else nk
            yield (slice(cu[b] + r, cu[b] + r + n), slice(ck[b], ck[b] + seen), r + nk - nq)


def _scores(st, q, k, shift):
    """[G, n, m] of q [n, G, D] and k [m, D] in their type, masked."""
    s = torch.matmul(q.transpose(0, 1), k.T) * st["D"] ** -0.5
    if st["causal"]:
        i = torch.arange(q.shape[0], device="cuda")[:, None] + shift
        s = torch.where(torch.arange(k.shape[0], device="cuda") > i, -math.inf, s)
    return s


def _fwd(st):
    G, dt = st["Hq"] // st["Hk"], st["q"].dtype
    o = torch.zeros_like(st["q"])
    lse = torch.full(o.shape[:2], -math.inf, device="cuda")
    for rows, keys, shift in _pieces(st):
        if keys.stop == keys.start:
            continue
        for h in range(st["Hk"]):
            heads = slice(h * G, (h + 1) * G)
            s = _scores(st, st["q"][rows, heads].float(), st["k"][keys, h].float(), shift)
            m = s.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, 0.0, m)
            e = torch.exp(s - m)
            z = e.sum(-1, keepdim=True)
            x = torch.matmul(e, st["v"][keys, h].float()) / torch.where(z == 0, 1.0, z)
            o[rows, heads] = x.transpose(0, 1).to(dt)
            lse[rows, heads] = (m + torch.log(z))[..., 0].T
    return o, lse


def _bwd(st):
    G, dt, scale = st["Hq"] // st["Hk"], st["q"].dtype, st["D"] ** -0.5
    dq = torch.zeros_like(st["q"])
    dk = torch.zeros(st["k"].shape, device="cuda")
    dv = torch.zeros(st["k"].shape, device="cuda")
    for rows, keys, shift in _pieces(st):
        if keys.stop == keys.start:
            continue
        for h in range(st["Hk"]):
            heads = slice(h * G, (h + 1) * G)
            q, do = st["q"][rows, heads].float(), st["do"][rows, heads].float()
            k, v = st["k"][keys, h].float(), st["v"][keys, h].float()
            lse = st["lse"][rows, heads].T[..., None]
            p = torch.exp(_scores(st, q, k, shift) - torch.where(lse == -math.inf, 0.0, lse))
            delta = (st["o"][rows, heads].float() * do).sum(-1).T[..., None]
            dp = torch.matmul(do.transpose(0, 1), v.T)
            ds = p * (dp - delta) * scale
            dq[rows, heads] = torch.matmul(ds, k).transpose(0, 1).to(dt)
            dk[keys, h] += torch.matmul(ds.transpose(1, 2), q.transpose(0, 1)).sum(0)
            dv[keys, h] += torch.matmul(p.transpose(1, 2), do.transpose(0, 1)).sum(0)
    return dq, dk.to(dt), dv.to(dt)


def _request_of(cu, n):
    """Request and place in it of packed rows 0 .. n - 1."""
    t = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu.long(), t, right=True) - 1
    return b, t - cu.long()[b]


def _write8(st, x, cache, scale):
    """One of the two caches, in place."""
    P, Hk, D = st["page"], st["Hk"], st["D"]
    flat, sc = cache.view(-1, Hk, D), scale.view(-1, Hk)
    ctx, table = st["ctx_len"].long(), st["block_table"].long()
    b, i = _request_of(st["cu"], x.shape[0])
    pos = ctx[b] + i
    row = table[b, pos // P] * P + pos % P
    x = x.float()
    top = torch.zeros_like(sc)
    top.scatter_reduce_(0, (row // BLOCK)[:, None].expand(-1, Hk), x.abs().amax(-1), "amax")
    mant, exp = torch.frexp(top)  # top = mant 2^exp; 448 = 0.875 2^9
    want = _power((exp - 9 + (mant > 0.875).int()).clamp(-100, 120))
    want = torch.where(top == 0, 2.0 ** -100, want)
    # blocks that a request's earlier tokens share with its new ones
    live = (st["cu"][1:] > st["cu"][:-1]) & (ctx % BLOCK != 0)
    r = torch.arange(BLOCK, device="cuda")
    start = ctx // BLOCK * BLOCK
    page = table.gather(1, (start // P).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    first = page * P + start % P                              # [B]
    old = (first[:, None] + r)[live[:, None] & (r < (ctx % BLOCK)[:, None])]
    shared = first[live] // BLOCK
    before = sc[old // BLOCK]
    want[shared] = torch.maximum(want[shared], sc[shared])
    values = flat[old].float() * (before / want[old // BLOCK])[..., None]
    flat.view(torch.uint8)[old] = values.to(F8).view(torch.uint8)
    codes = (x / want[row // BLOCK][..., None]).to(F8)
    flat.view(torch.uint8)[row] = codes.view(torch.uint8)
    blocks = row // BLOCK
    sc[blocks] = want[blocks]


def _read8(st, cache, scale):
    P, Hk, D = st["page"], st["Hk"], st["D"]
    b, pos = _request_of(st["cu_k"], st["n"])
    row = st["block_table"].long()[b, pos // P] * P + pos % P
    x = cache.view(torch.uint8).view(-1, Hk, D)[row].view(F8).float()
    return (x * scale.view(-1, Hk)[row // BLOCK][..., None]).to(DT[st["dtype"]])


def _cache(st):
    for x in ("k", "v"):
        _write8(st, st[x], st[x + "_cache"], st[x + "_scale"])
    return (_read8(st, st["k_cache"], st["k_scale"]), _read8(st, st["v_cache"], st["v_scale"]),
            st["k_scale"], st["v_scale"])


def _dec8(st):
    P, Hk, D = st["page"], st["Hk"], st["D"]
    pos = torch.arange(max(st["top"], 1), device="cuda")
    page = st["block_table"].long()[:, pos // P].clamp(min=0)
    at = page * P + pos % P                                             # [B, L]
    dead = pos[None, :] >= st["seq_len"][:, None]

    def values(x):
        codes = st[x + "_cache"].view(torch.uint8).view(-1, Hk, D)[at].view(F8).float()
        return codes * st[x + "_scale"].view(-1, Hk)[at // BLOCK][..., None]

    k = values("k")                                                     # [B, L, Hk, D]
    q = st["q"].float().reshape(st["B"], Hk, -1, D)                     # [B, Hk, G, D]
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * D ** -0.5              # [B, Hk, G, L]
    del k
    v = torch.where(dead[:, :, None, None], 0.0, values("v"))
    s = torch.where(dead[:, None, None, :], -math.inf, s)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v.permute(0, 2, 1, 3)) / torch.where(z == 0, 1.0, z)
    lse = (m + torch.log(z)).reshape(st["B"], -1)
    return o.reshape(st["q"].shape).to(st["q"].dtype), lse


PLAIN = {"fwd": _fwd, "bwd": _bwd, "cache": _cache, "dec8": _dec8}


# ------------------------------------------------------------------ the framework's calls

def _own(st):
    import chunked_state_scan_gated_gb300 as gdn
    op = st["op"]
    if op == "fwd":
        return gdn.gdn_attn_fwd(st["q"], st["k"], st["v"], st["cu"], st["cu_k"],
                                causal=st["causal"])
    if op == "bwd":
        return gdn.gdn_attn_bwd(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], st["cu"],
                                st["cu_k"], causal=st["causal"])
    cache = (st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
    if op == "dec8":
        return gdn.gdn_attn_decode8(st["q"], *cache, st["block_table"], st["seq_len"])
    gdn.gdn_cache_write8(st["k"], st["v"], *cache, st["block_table"], st["ctx_len"], st["cu"])
    k, v = gdn.gdn_cache_read8(*cache, st["block_table"], st["cu_k"], n_tokens=st["n"],
                               dtype=DT[st["dtype"]])
    return k, v, st["k_scale"], st["v_scale"]


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# -------------------------------------------------------------------------------- work

def _pairs(case, lens, ctx):
    """Query-key pairs that count."""
    if not case["causal"]:
        return sum(n * (c + n) for n, c in zip(lens, ctx))
    return sum(n * c + n * (n + 1) // 2 for n, c in zip(lens, ctx))


def work(case):
    """Mean over the lengths' orders (a sequence's own tokens and those in front of it meet)."""
    total = {"bytes": 0.0, "flops": 0.0}
    draws = 16 if case.get("ctx") else 1
    for seed in range(draws):
        bytes_, flops = _work(case, _lengths(case, seed),
                              _contexts(case, seed) if "ctx" in case else None)
        total["bytes"] += bytes_ / draws
        total["flops"] += flops / draws
    return total


def _work(case, lens, ctx):
    op, w, Hk, D = case["op"], 2 if case["dtype"] == "bf16" else 4, case["Hk"], case["D"]
    n = sum(lens)
    if op == "dec8":
        Hq = case["Hq"]
        return (2 * n * Hk * (D + 4 / BLOCK) + 2 * w * case["B"] * Hq * D + 4 * case["B"] * Hq
                + 4 * n / case["page"], 4 * n * Hq * D)
    m = n + sum(ctx)
    if op == "cache":  # new tokens in; the cache's blocks written, every token read and out
        return (2 * n * Hk * (w * D + D + 4 / BLOCK) + 2 * m * Hk * (D + 4 / BLOCK + w * D)
                + 4 * m / case["page"], 0)
    Hq = case["Hq"]
    pairs = _pairs(case, lens, ctx)
    if op == "fwd":
        return w * D * (2 * n * Hq + 2 * m * Hk) + 4 * n * Hq, 4 * pairs * Hq * D
    return w * D * (4 * n * Hq + 4 * m * Hk) + 4 * n * Hq, 10 * pairs * Hq * D


# ------------------------------------------------------------------------- in 64 bits

def _exact_rows(st):
    """(b, first query row, queries, keys, key rows) by runs of queries that fit in 64 bits."""
    cu, ck = st["cu_host"], st["cu_k_host"]
    for b in range(st["B"]):
        nq, nk = cu[b + 1] - cu[b], ck[b + 1] - ck[b]
        for r in range(0, nq, 2048):
            n = min(2048, nq - r)
            m = min(nk, r + n + nk - nq) if st["causal"] else nk
            if m > 0:
                hidden = None
                if st["causal"]:
                    hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(
                        r + nk - nq + 1)
                yield cu[b] + r, n, ck[b], m, hidden


def _exact_fwd(st):
    G = st["Hq"] // st["Hk"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for q0, n, k0, m, hidden in _exact_rows(st):
        for h in range(st["Hq"]):
            s = st["q"][q0:q0 + n, h].double() @ st["k"][k0:k0 + m, h // G].double().T
            s /= math.sqrt(st["D"])
            if hidden is not None:
                s.masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(s, 1)
            lse[q0:q0 + n, h] = z
            w = torch.exp(s - torch.where(z == -math.inf, 0.0, z)[:, None])
            out[q0:q0 + n, h] = w @ st["v"][k0:k0 + m, h // G].double()
    return out, lse


def _exact_bwd(st):
    """Gradients of sum(do * attention(q, k, v)) at the forward's own o and lse, as the call is
    given them."""
    G, c = st["Hq"] // st["Hk"], 1 / math.sqrt(st["D"])
    dq = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    dk = torch.zeros(st["k"].shape, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    for q0, n, k0, m, hidden in _exact_rows(st):
        for h in range(st["Hq"]):
            q, do = st["q"][q0:q0 + n, h].double(), st["do"][q0:q0 + n, h].double()
            k, v = st["k"][k0:k0 + m, h // G].double(), st["v"][k0:k0 + m, h // G].double()
            z = st["lse"][q0:q0 + n, h].double()
            w = torch.exp(q @ k.T * c - torch.where(z == -math.inf, 0.0, z)[:, None])
            if hidden is not None:
                w.masked_fill_(hidden, 0.0)
            dv[k0:k0 + m, h // G] += w.T @ do
            mean = torch.einsum("nd,nd->n", do, st["o"][q0:q0 + n, h].double())
            w *= (do @ v.T - mean[:, None]) * c
            dq[q0:q0 + n, h] = w @ k
            dk[k0:k0 + m, h // G] += w.T @ q
    return dq, dk, dv


def _grid(x):
    """x rounded to e4m3's numbers (|x| <= 448), ties to even: steps of an eighth of the power of
    two below |x|, of 2^-9 at the bottom."""
    step = torch.full_like(x, 2.0 ** -9)
    for e in range(-5, 9):
        step = torch.where(x.abs() >= 2.0 ** e, 2.0 ** (e - 3), step)
    return torch.round(x / step) * step


def _exact_cache(st):
    """Request by request and block by block."""
    P, cu, ck = st["page"], st["cu_host"], st["cu_k_host"]
    out = []
    for x in ("k", "v"):
        codes = st[x + "_cache"].double().flatten(0, 1)       # [rows, Hk, D]
        scale = st[x + "_scale"].double().flatten(0, 1)       # [blocks, Hk]
        back = []
        for b, pages in enumerate(st["block_table"].tolist()):
            new = st[x][cu[b]:cu[b + 1]].double()
            n = ck[b + 1] - ck[b]
            ctx = n - new.shape[0]
            held = torch.tensor(pages[:-(-n // P)], device="cuda", dtype=torch.long)
            rows = (held[:, None] * P + torch.arange(P, device="cuda")).flatten()
            first = ctx // BLOCK if new.shape[0] else n // BLOCK + 1
            blocks = rows[::BLOCK] // BLOCK                   # of the whole request
            val = codes[rows] * scale[rows // BLOCK][..., None]
            val[n:] = 0
            if new.shape[0]:
                val[ctx:n] = new
                top = val.abs().amax(-1).unflatten(0, (-1, BLOCK))
                fresh = torch.zeros(len(rows), 1, dtype=torch.bool, device="cuda")
                fresh[ctx:n] = True
                top = torch.where(fresh.unflatten(0, (-1, BLOCK)), top, 0.0).amax(1)
                s = torch.full_like(top, 2.0 ** -100)
                for e in range(-99, 121):  # the lowest power of two that 448 times is not below
                    s = torch.where(top > s * 448, 2.0 ** e, s)
                if ctx % BLOCK:
                    s[first] = torch.maximum(s[first], scale[blocks[first]])
                scale[blocks[first:-(-n // BLOCK)]] = s[first:-(-n // BLOCK)]
                sc = scale[rows // BLOCK][..., None]
                val = torch.cat((val[:first * BLOCK],
                                 (_grid(val / sc) * sc)[first * BLOCK:]))
            back.append(val[:n])
        out.append((torch.cat(back), scale.reshape(st[x + "_scale"].shape)))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _exact_dec8(st):
    B, G, D, P = st["B"], st["Hq"] // st["Hk"], st["D"], st["page"]
    out = torch.zeros(B, st["Hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, st["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["seq_len"].tolist()):
        if n == 0:
            continue
        ids = st["block_table"][b, :-(-n // P)].long()
        k, v = ((st[x + "_cache"].view(torch.uint8)[ids].view(F8).double()
                 * st[x + "_scale"][ids].double().repeat_interleave(BLOCK, 1)[..., None])
                .flatten(0, 1)[:n] for x in ("k", "v"))
        for h in range(st["Hq"]):
            s = (k[:, h // G] @ st["q"][b, h].double()) / math.sqrt(D)
            lse[b, h] = torch.logsumexp(s, 0)
            out[b, h] = torch.exp(s - lse[b, h]) @ v[:, h // G]
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    return {"fwd": _exact_fwd, "bwd": _exact_bwd, "cache": _exact_cache,
            "dec8": _exact_dec8}[case["op"]](st)
