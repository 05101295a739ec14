"""The operators of one decode step of a hybrid Gated DeltaNet / full-attention model, and of
the attention layer's training step: what is timed, on which inputs, and their plain forms.

- ``attn``  gdn_attn_decode: one new token per request over a paged key-value cache.
- ``step``  gdn_step: the Gated DeltaNet recurrence of one token over a pool of states.
- ``rope_fwd`` / ``rope_bwd`` / ``rope_cache``  gdn_qk_norm_rope_*: RMSNorm of every query and
  key head with the position rotation, its backward, and the form that writes K and V to the
  paged cache.
- ``slots`` gdn_slot_map: block tables, slots and positions from request lengths.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one interactive request early in its answer: three dependent reads, latency
        {"name": "attn_one_short", "op": "attn", "B": 1, "lo": 517, "hi": 517, "Hq": 16, "Hk": 2,
         "D": 256, "page": 16, "dtype": "bf16"},
        # one request over a long document: the cache's length has to be split
        {"name": "attn_one_long", "op": "attn", "B": 1, "lo": 131001, "hi": 131001, "Hq": 32,
         "Hk": 8, "D": 128, "page": 64, "dtype": "bf16"},
        # a mixed batch, a few tokens to long contexts
        {"name": "attn_ragged", "op": "attn", "B": 61, "lo": 1, "hi": 16384, "Hq": 32, "Hk": 8,
         "D": 128, "page": 16, "dtype": "bf16"},
        # a full server: bandwidth
        {"name": "attn_large", "op": "attn", "B": 128, "lo": 2000, "hi": 16000, "Hq": 16,
         "Hk": 2, "D": 256, "page": 32, "dtype": "bf16"},
        # a small model checked in fp32, three query heads to a key head
        {"name": "attn_fp32", "op": "attn", "B": 9, "lo": 100, "hi": 5000, "Hq": 12, "Hk": 4,
         "D": 64, "page": 32, "dtype": "fp32"},
        # the GDN layer of one interactive request
        {"name": "step_one", "op": "step", "B": 1, "Hqk": 16, "H": 32, "dk": 128, "dv": 128,
         "dtype": "bf16"},
        # the GDN layer of a full server, states picked from a pool
        {"name": "step_large", "op": "step", "B": 250, "Hqk": 16, "H": 32, "dk": 128, "dv": 128,
         "dtype": "bf16"},
        # training, a quarter of each head rotated, halves paired, q and k slices of one projection
        {"name": "rope_train_fwd", "op": "rope_fwd", "N": 32768, "Hq": 16, "Hk": 2, "D": 256,
         "R": 64, "inter": False, "far": 0, "dtype": "bf16"},
        # its backward with whole heads rotated in neighbouring pairs, positions past 2^19
        {"name": "rope_train_bwd", "op": "rope_bwd", "N": 16001, "Hq": 32, "Hk": 8, "D": 128,
         "R": 128, "inter": True, "far": 600000, "dtype": "bf16"},
        # a decode step's new tokens into the cache
        {"name": "rope_decode_cache", "op": "rope_cache", "N": 64, "Hq": 16, "Hk": 2, "D": 256,
         "R": 64, "inter": False, "far": 100000, "page": 16, "dtype": "bf16"},
        # a decode step's slots: one new token each
        {"name": "slots_decode", "op": "slots", "B": 250, "ctx": 20000, "lo": 1, "hi": 1,
         "page": 16},
        # a step that takes whole prompts in
        {"name": "slots_prefill", "op": "slots", "B": 37, "ctx": 5000, "lo": 500, "hi": 4000,
         "page": 64},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "step", "rope_fwd", "rope_bwd", "rope_cache", "slots"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "attn":
        D, B = rng.choice([64, 128, 256]), _spread(rng, 1, 128)
        Hk = rng.choice([1, 2, 4, 8])
        hi = _spread(rng, 16, min(131072, 2 ** 28 // (B * Hk * D)))
        return {"op": op, "B": B, "lo": rng.choice([0, 1, max(1, hi // 2)]), "hi": hi,
                "Hq": Hk * rng.choice([1, 2, 3, 4, 8, 12]), "Hk": Hk, "D": D,
                "page": rng.choice([16, 32, 48, 64, 128]), "dtype": dtype}
    if op == "step":
        Hqk = rng.choice([1, 2, 4, 8, 16])
        if dtype == "bf16":
            dk = dv = 128
        else:
            dk, dv = rng.choice([16, 64, 80, 128]), rng.choice([16, 48, 64, 128])
        return {"op": op, "B": _spread(rng, 1, 200), "Hqk": Hqk, "H": Hqk * rng.choice([1, 2, 3]),
                "dk": dk, "dv": dv, "dtype": dtype}
    if op == "slots":
        hi = rng.choice([1, 4, 700, 3500])
        B = _spread(rng, 1, 1500 if hi < 100 else 40)
        return {"op": op, "B": B, "ctx": _spread(rng, 1, min(30000, 2 ** 21 // B)), "lo": rng.choice([0, 1]), "hi": hi,
                "page": rng.choice([1, 16, 24, 64, 256])}
    D = rng.choice([64, 80, 128, 256])
    R = rng.choice([r for r in (16, 32, 64, 80, 128, 256) if r <= D])
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 4, 8])
    top = min(16384, 2 ** 27 // ((Hq + Hk) * D))
    case = {"op": op, "N": _spread(rng, 1, top if op != "rope_cache" else min(top, 4000)),
            "Hq": Hq, "Hk": Hk, "D": D, "R": R, "inter": rng.random() < 0.5,
            "far": rng.choice([0, 1000, 1000000]), "dtype": dtype}
    if op == "rope_cache":
        case["page"] = rng.choice([16, 32, 64])
    return case


# ------------------------------------------------------------------------------ inputs

def _lengths(case, seed):
    """Request lengths in [lo, hi], spread over their logarithm."""
    r = random.Random(seed * 7 + 1)
    lo, hi = case["lo"], case["hi"]
    return [min(hi, max(lo, int(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1))) - 0.5)))
            for _ in range(case["B"])]


def _token_rows(case):
    """Token rows of the step's buffers: enough for any lengths, as a captured step has them."""
    return -(-case["B"] * case["hi"] // 64) * 64


def _shuffled(seed, n):
    return np.random.RandomState(seed % 2 ** 31).permutation(n).astype(np.int32)


def _gpu(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(gen, shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    st = dict(case)
    gen = _gpu(seed)
    op = case["op"]
    if op == "attn":
        dt, B, P = DT[case["dtype"]], case["B"], case["page"]
        lens = _lengths(case, seed)
        width = max(1, -(-case["hi"] // P))
        counts = [-(-n // P) for n in lens]
        pages = sum(counts) + 3
        perm = _shuffled(seed * 7 + 2, pages)
        table = np.full((B, width), -1, dtype=np.int32)  # unused entries hold no page
        at = 0
        for b, c in enumerate(counts):
            table[b, :c] = perm[at:at + c]
            at += c
        st["k_cache"] = _rand(gen, (pages, P, case["Hk"], case["D"]), dt)
        st["v_cache"] = _rand(gen, (pages, P, case["Hk"], case["D"]), dt)
        st["q"] = _rand(gen, (B, case["Hq"], case["D"]), dt)
        st["block_table"] = torch.from_numpy(table).cuda()
        st["seq_len"] = _i32(lens)
        st["top"] = max(lens)
    elif op == "step":
        dt, B, H = DT[case["dtype"]], case["B"], case["H"]
        pool = B + B // 8 + 1  # some slots belong to requests that are not in this step
        st["q"] = _rand(gen, (B, 1, case["Hqk"], case["dk"]), dt)
        st["k"] = _rand(gen, (B, 1, case["Hqk"], case["dk"]), dt)
        st["v"] = _rand(gen, (B, 1, H, case["dv"]), dt)
        st["a"] = _rand(gen, (B, 1, H), dt)
        st["b"] = _rand(gen, (B, 1, H), dt)
        st["A_log"] = (1.0 + 15.0 * torch.rand(H, generator=gen, device="cuda")).log()
        st["dt_bias"] = -6.0 + 0.1 * _rand(gen, (H,))  # slow decay: the state matters
        st["state"] = 0.1 * _rand(gen, (pool, H, case["dk"], case["dv"]))
        st["slots"] = _i32(random.Random(seed * 7 + 3).sample(range(pool), B))
    elif op == "slots":
        P, r = case["page"], random.Random(seed * 7 + 4)
        new = _lengths(case, seed)
        ctx = [r.randint(0, case["ctx"]) for _ in new]
        held = [-(-c // P) for c in ctx]
        want = sum(-(-(c + n) // P) - h for c, n, h in zip(ctx, new, held))
        width = -(-(case["ctx"] + case["hi"]) // P)
        pages = sum(held) + want + 5
        perm = _shuffled(seed * 7 + 6, pages)
        table = np.full((case["B"], width), -1, dtype=np.int32)
        at = 0
        for b, c in enumerate(held):
            table[b, :c] = perm[at:at + c]
            at += c
        st["block_table"] = torch.from_numpy(table).cuda()
        st["free"] = torch.from_numpy(perm[at:]).cuda()
        st["ctx_len"], st["new_len"] = _i32(ctx), _i32(new)
        st["pages"] = pages
        st["n_tokens"] = _token_rows(case)
    else:
        dt, N, Hq, Hk, D = DT[case["dtype"]], case["N"], case["Hq"], case["Hk"], case["D"]
        qkv = _rand(gen, (N, (Hq + 2 * Hk) * D), dt)  # one projection's output
        st["q"] = qkv[:, :Hq * D].view(N, Hq, D)
        st["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(N, Hk, D)
        st["v"] = qkv[:, (Hq + Hk) * D:].view(N, Hk, D)
        st["wq"] = 1.0 + 0.1 * _rand(gen, (D,))
        st["wk"] = 1.0 + 0.1 * _rand(gen, (D,))
        half = case["R"] // 2
        st["inv_freq"] = torch.tensor([1e6 ** (-i / half) for i in range(half)],
                                      dtype=torch.float32, device="cuda")
        if case["far"]:
            st["pos"] = torch.randint(0, case["far"], (N,), generator=gen, device="cuda",
                                      dtype=torch.int32)
        else:
            st["pos"] = torch.arange(N, device="cuda", dtype=torch.int32)
        if op == "rope_bwd":
            st["dqo"] = _rand(gen, (N, Hq, D), dt)
            st["dko"] = _rand(gen, (N, Hk, D), dt)
        if op == "rope_cache":
            P = case["page"]
            pages = -(-N // P) + 8
            st["k_cache"] = _rand(gen, (pages, P, Hk, D), dt)
            st["v_cache"] = _rand(gen, (pages, P, Hk, D), dt)
            slot = random.Random(seed * 7 + 5).sample(range(pages * P), N)
            if N > 4:
                slot[N // 2] = -1  # a padded row of the batch: written nowhere
            st["slots"] = _i32(slot)
    return st


# ------------------------------------------------------------------------- plain forms

def _attn(st):
    P, Hk, D = st["page"], st["Hk"], st["D"]
    pos = torch.arange(max(st["top"], 1), device="cuda")
    page = st["block_table"].long()[:, pos // P].clamp(min=0)
    at = page * P + pos % P                                             # [B, L]
    dead = pos[None, :] >= st["seq_len"][:, None]
    k = st["k_cache"].reshape(-1, Hk, D)[at].float()                    # [B, L, Hk, D]
    v = st["v_cache"].reshape(-1, Hk, D)[at].float()
    v = torch.where(dead[:, :, None, None], 0.0, v)
    q = st["q"].float().reshape(st["B"], Hk, -1, D)                     # [B, Hk, G, D]
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) * D ** -0.5              # [B, Hk, G, L]
    s = torch.where(dead[:, None, None, :], -math.inf, s)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v.permute(0, 2, 1, 3)) / torch.where(z == 0, 1.0, z)
    lse = (m + torch.log(z)).reshape(st["B"], -1)
    return o.reshape(st["q"].shape).to(st["q"].dtype), lse


def _step(st):
    q, k, v = st["q"][:, 0].float(), st["k"][:, 0].float(), st["v"][:, 0].float()
    r = st["H"] // st["Hqk"]
    q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + EPS) * st["dk"] ** -0.5
    k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + EPS)
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)         # [B, H, dk]
    x = st["a"][:, 0].float() + st["dt_bias"]
    soft = torch.where(x > 20, x, torch.log1p(torch.exp(x.clamp(max=20))))
    alpha = torch.exp(-torch.exp(st["A_log"]) * soft)[..., None, None]
    beta = (1 / (1 + torch.exp(-st["b"][:, 0].float())))[..., None, None]
    at = st["slots"].long()
    S = st["state"][at]
    u = torch.matmul(k[..., None, :], S)                                # [B, H, 1, dv]
    S = alpha * (S - beta * k[..., None] * u) + beta * k[..., None] * v[..., None, :]
    st["state"][at] = S
    o = torch.matmul(q[..., None, :], S)[..., 0, :]
    return o[:, None].to(st["v"].dtype), st["state"]


def _cos_sin(st):
    ang = st["pos"].double()[:, None] * st["inv_freq"].double()
    return ang.cos().float()[:, None], ang.sin().float()[:, None]       # [N, 1, R/2]


def _halves(st, x):
    R = st["R"]
    if st["inter"]:
        return x[..., 0:R:2], x[..., 1:R:2]
    return x[..., :R // 2], x[..., R // 2:R]


def _whole(st, x1, x2, x):
    if st["inter"]:
        y = torch.stack((x1, x2), -1).flatten(-2)
    else:
        y = torch.cat((x1, x2), -1)
    return torch.cat((y, x[..., st["R"]:]), -1)


def _norm_rope(st, x, w, cos, sin):
    x = x.float()
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    n1, n2 = _halves(st, n)
    return _whole(st, n1 * cos - n2 * sin, n2 * cos + n1 * sin, n)


def _norm_rope_bwd(st, x, w, dy, cos, sin):
    x, dy = x.float(), dy.float()
    d1, d2 = _halves(st, dy)
    dn = _whole(st, d1 * cos + d2 * sin, d2 * cos - d1 * sin, dy)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    dw = (dn * n).double().sum((0, 1)).float()
    g = dn * w
    return r * (g - n * (g * n).mean(-1, keepdim=True)), dw


def _rope_fwd(st):
    cos, sin = _cos_sin(st)
    dt = st["q"].dtype
    return (_norm_rope(st, st["q"], st["wq"], cos, sin).to(dt),
            _norm_rope(st, st["k"], st["wk"], cos, sin).to(dt))


def _rope_bwd(st):
    cos, sin = _cos_sin(st)
    dt = st["q"].dtype
    dq, dwq = _norm_rope_bwd(st, st["q"], st["wq"], st["dqo"], cos, sin)
    dk, dwk = _norm_rope_bwd(st, st["k"], st["wk"], st["dko"], cos, sin)
    return dq.to(dt), dk.to(dt), dwq, dwk


def _rope_cache(st):
    q, k = _rope_fwd(st)
    _write(st["k_cache"].view(-1, st["Hk"], st["D"]), st["slots"], k)
    _write(st["v_cache"].view(-1, st["Hk"], st["D"]), st["slots"], st["v"])
    return q, st["k_cache"], st["v_cache"]


def _write(table, at, rows):
    """table[at] = rows, where the place -1 is nowhere (a row behind the last, dropped again)."""
    longer = torch.cat((table, table[:1]))
    longer[at.long()] = rows
    table.copy_(longer[:-1])


def _slots(st):
    P, n = st["page"], st["n_tokens"]
    ctx, new = st["ctx_len"].long(), st["new_len"].long()
    held = (ctx + P - 1) // P
    need = (ctx + new + P - 1) // P - held
    cu = torch.cat((new.new_zeros(1), new.cumsum(0)))
    first = need.cumsum(0) - need
    t = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    live = b < st["B"]
    b = b.clamp(max=st["B"] - 1)
    pos = ctx[b] + t - cu[b]
    i = pos // P
    fresh = i >= held[b]
    pick = (first[b] + i - held[b]).clamp(0, st["free"].numel() - 1)
    old = st["block_table"][b, i.clamp(max=st["block_table"].shape[1] - 1)]
    page = torch.where(fresh, st["free"][pick], old)
    slots = torch.where(live, page * P + pos % P, -1).int()
    width = st["block_table"].shape[1]
    _write(st["block_table"].view(-1), torch.where(live & fresh, b * width + i, -1), page)
    return ((ctx + new).int(), cu.int(), torch.where(live, pos, 0).int(), slots,
            st["block_table"], need.sum().int().reshape(1))


PLAIN = {"attn": _attn, "step": _step, "rope_fwd": _rope_fwd, "rope_bwd": _rope_bwd,
         "rope_cache": _rope_cache, "slots": _slots}


# ------------------------------------------------------------------ the framework's calls

def _own(st):
    import chunked_state_scan_gated_gb300 as gdn
    op = st["op"]
    if op == "attn":
        return gdn.gdn_attn_decode(st["q"], st["k_cache"], st["v_cache"], st["block_table"],
                                   st["seq_len"])
    if op == "step":
        o = gdn.gdn_step(st["q"], st["k"], st["v"], st["a"], st["b"], st["A_log"],
                         st["dt_bias"], st["state"], st["slots"])
        return o, st["state"]
    if op == "slots":
        seq_len, cu, pos, slots, used = gdn.gdn_slot_map(
            st["ctx_len"], st["new_len"], st["free"], st["block_table"], page_size=st["page"],
            pages=st["pages"], n_tokens=st["n_tokens"])
        return seq_len, cu, pos, slots, st["block_table"], used
    rope = (st["wq"], st["wk"], st["inv_freq"], st["pos"])
    if op == "rope_fwd":
        return gdn.gdn_qk_norm_rope_fwd(st["q"], st["k"], *rope, interleaved=st["inter"], eps=EPS)
    if op == "rope_bwd":
        return gdn.gdn_qk_norm_rope_bwd(st["q"], st["k"], *rope, st["dqo"], st["dko"],
                                        interleaved=st["inter"], eps=EPS)
    q = gdn.gdn_qk_norm_rope_cache(st["q"], st["k"], st["v"], *rope, st["slots"], st["k_cache"],
                                   st["v_cache"], interleaved=st["inter"], eps=EPS)
    return q, st["k_cache"], st["v_cache"]


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# -------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "slots":
        B, pages = case["B"], case["B"] * _mean_len(case) / case["page"]
        return {"bytes": 12 * B + 8 * pages + 8 * _token_rows(case) + 8 * B, "flops": 0}
    w = 2 if case["dtype"] == "bf16" else 4
    if op == "attn":
        tokens = case["B"] * _mean_len(case)
        return {"bytes": 2 * w * tokens * case["Hk"] * case["D"]
                + 2 * w * case["B"] * case["Hq"] * case["D"] + 4 * case["B"] * case["Hq"]
                + 4 * tokens / case["page"],
                "flops": 4 * tokens * case["Hq"] * case["D"]}
    if op == "step":
        B, H, dk, dv = case["B"], case["H"], case["dk"], case["dv"]
        return {"bytes": 8 * B * H * dk * dv + w * B * (2 * case["Hqk"] * dk + 2 * H * dv + 2 * H),
                "flops": 8 * B * H * dk * dv}
    N, D = case["N"], case["D"]
    rows = N * (case["Hq"] + case["Hk"])
    if op == "rope_fwd":
        return {"bytes": 2 * w * rows * D + 4 * N, "flops": 8 * rows * D}
    if op == "rope_bwd":
        return {"bytes": 3 * w * rows * D + 4 * N + 16 * D, "flops": 16 * rows * D}
    return {"bytes": 2 * w * (rows + N * case["Hk"]) * D + 8 * N, "flops": 8 * rows * D}


def _mean_len(case):
    """The mean of _lengths: log-uniform between lo + 1 and hi + 1, less one."""
    lo, hi = case["lo"], case["hi"]
    if lo == hi:
        return hi
    return (hi - lo) / math.log((hi + 1) / (lo + 1)) - 1


# ------------------------------------------------------------------------- in 64 bits

def _exact_attn(st):
    B, G, D = st["B"], st["Hq"] // st["Hk"], st["D"]
    lens, table = st["seq_len"].tolist(), st["block_table"].long()
    out = torch.zeros(B, st["Hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, st["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        ids = table[b, :-(-n // st["page"])]
        k = st["k_cache"][ids].flatten(0, 1)[:n].double()
        v = st["v_cache"][ids].flatten(0, 1)[:n].double()
        for h in range(st["Hq"]):
            s = (k[:, h // G] @ st["q"][b, h].double()) / math.sqrt(D)
            lse[b, h] = torch.logsumexp(s, 0)
            out[b, h] = torch.exp(s - lse[b, h]) @ v[:, h // G]
    return out, lse


def _exact_step(st):
    r = st["H"] // st["Hqk"]
    state = st["state"].double()
    o = torch.zeros(st["v"].shape, dtype=torch.float64, device="cuda")
    for i, at in enumerate(st["slots"].tolist()):
        q, k = st["q"][i, 0].double(), st["k"][i, 0].double()
        q = q / torch.sqrt(q.square().sum(-1, keepdim=True) + EPS) / math.sqrt(st["dk"])
        k = k / torch.sqrt(k.square().sum(-1, keepdim=True) + EPS)
        g = -st["A_log"].double().exp() * torch.nn.functional.softplus(
            st["a"][i, 0].double() + st["dt_bias"].double())
        beta = torch.sigmoid(st["b"][i, 0].double())
        head = torch.arange(st["H"], device="cuda") // r
        qh, kh = q[head], k[head]
        S = state[at] * g.exp()[:, None, None]
        err = st["v"][i, 0].double() - torch.einsum("hk,hkv->hv", kh, S)
        S = S + torch.einsum("h,hk,hv->hkv", beta, kh, err)
        state[at] = S
        o[i, 0] = torch.einsum("hk,hkv->hv", qh, S)
    return o, state


def _turn(st, x, sign):
    """The rotation of the pairs as a product of complex numbers."""
    R = st["R"]
    ang = torch.outer(st["pos"].double(), st["inv_freq"].double()) * sign
    z = torch.polar(torch.ones_like(ang), ang)[:, None]
    y = x.clone()
    if st["inter"]:
        c = torch.view_as_complex(x[..., :R].reshape(*x.shape[:-1], R // 2, 2).contiguous()) * z
        y[..., :R] = torch.view_as_real(c).reshape(*x.shape[:-1], R)
    else:
        c = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * z
        y[..., :R // 2], y[..., R // 2:R] = c.real, c.imag
    return y


def _exact_rows(st, x, w):
    x = x.double()
    return _turn(st, x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double(), 1.0)


def _exact_rows_bwd(st, x, w, dy):
    x = x.double()
    rms = torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    dn = _turn(st, dy.double(), -1.0)
    g = dn * w.double()
    dot = (g * x).sum(-1, keepdim=True)
    return g / rms - x * dot / (st["D"] * rms ** 3), (dn * x / rms).sum((0, 1))


def exact(case, seed):
    op = case["op"]
    if op == "slots":
        return None
    st = prepare(case, seed)
    if op == "attn":
        return _exact_attn(st)
    if op == "step":
        return _exact_step(st)
    if op == "rope_bwd":
        dq, dwq = _exact_rows_bwd(st, st["q"], st["wq"], st["dqo"])
        dk, dwk = _exact_rows_bwd(st, st["k"], st["wk"], st["dko"])
        return dq, dk, dwq, dwk
    q, k = _exact_rows(st, st["q"], st["wq"]), _exact_rows(st, st["k"], st["wk"])
    if op == "rope_fwd":
        return q, k
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    for i, at in enumerate(st["slots"].tolist()):
        if at >= 0:
            kc[at // case["page"], at % case["page"]] = k[i]
            vc[at // case["page"], at % case["page"]] = st["v"][i].double()
    return q, kc, vc
