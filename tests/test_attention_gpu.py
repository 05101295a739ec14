"""GPU parity of the full-attention calls and of the 8-bit cache against their fp64 definitions
(oracle/attention.py), element by element.

Bounds.  `half(dtype)` = finfo.eps / 2 is one rounding to the type; U = 2^-24 one fp32 rounding;
T = 2^-22 what a step of a tensor core's sum may lose of its running magnitude (a rounding of an
ordinary fp32 sum is less).  Each bound is relative to the sum of the absolute values of the terms
that are added, so cancellation is accounted for; the counts are written beside each."""
import numpy as np
import pytest
import torch

import chunked_state_scan_gated_gb300 as gdn
from oracle import attention, decode

pytestmark = pytest.mark.gpu
U, T, TINY = 2.0 ** -24, 2.0 ** -22, 2.0 ** -126
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load_library()


def half(dt):
    return torch.finfo(dt).eps / 2


def n64(t):
    return t.detach().cpu().double().numpy()


def rand(gen, shape, dt=F32):
    return torch.randn(shape, generator=gen).to(dt).cuda()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def within(name, x, ref, bound):
    x = n64(x) if torch.is_tensor(x) else x
    assert x.shape == ref.shape
    assert np.isfinite(x).all(), f"{name}: non-finite values"
    over = np.abs(x - ref) - bound
    if not over.size:
        return
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, (f"{name}{at}: {x[at]} against {ref[at]}, bound "
                           f"{np.broadcast_to(bound, x.shape)[at]}")


# ------------------------------------------------------------------ attention over packed rows

def seq_inputs(lens, klens, Hq, Hk, D, dt, seed=0, tail=5, scale=1.0):
    """q, k, v as slices of projections; rows of no sequence (in front, behind) hold NaN."""
    gen = torch.Generator().manual_seed(seed)
    klens = lens if klens is None else klens
    cu, ck = np.cumsum([2] + list(lens)), np.cumsum([3] + list(klens))
    q = rand(gen, (cu[-1] + tail, Hq + 1, D))[:, :Hq] * scale
    q = torch.cat((q, q[:, :1]), 1).to(dt)[:, :Hq]
    kv = rand(gen, (ck[-1] + tail, 2 * Hk, D), dt)
    k, v = kv[:, :Hk], kv[:, Hk:]
    for x, c in ((q, cu), (k, ck), (v, ck)):
        x[:c[0]] = float("nan")
        x[c[-1]:] = float("nan")
    return q, k, v, cu, ck


def sums(q, k, v, o, lse, dO, cu, ck, causal, scale):
    """What the bounds are made of, as oracle-side arrays: for every output the sums of the absolute
    values of its terms, with the terms' own relative and absolute errors inside."""
    dt, D = q.dtype, q.shape[-1]
    q, k, v, o, dO = (n64(x) for x in (q, k, v, o, dO))
    lse = np.asarray(lse)
    Hq, Hk = q.shape[1], k.shape[1]
    G, sc = Hq // Hk, scale or D ** -0.5
    w_round = half(BF) if dt == BF else 0.0
    out = {n: np.zeros(s) for n, s in (("o", q.shape), ("lse", lse.shape), ("dq", q.shape),
                                       ("dk", k.shape), ("dv", k.shape))}
    for rows, keys in attention.sequences(cu, ck, len(q), len(k)):
        nq, nk = rows.stop - rows.start, keys.stop - keys.start
        mask = attention.seen(nq, nk, causal)
        if not mask.any():
            continue
        for h in range(Hq):
            qq, kk, vv, do = q[rows, h], k[keys, h // G], v[keys, h // G], dO[rows, h]
            s = qq @ kk.T * sc
            l = np.where(np.isfinite(lse[rows, h]), lse[rows, h], 0.0)[:, None]
            p = np.where(mask, np.exp(s - l), 0.0)
            # score: D products on tensor cores; scaling and the subtraction of the reference
            # (or of lse) round once each at the size of the score; exp2 2^-21
            S = np.abs(qq) @ np.abs(kk).T * sc * (D + 8) * T
            e = S + 4 * U * (np.abs(s) + np.abs(l) + 1) + 2.0 ** -21
            top = np.where(mask, e, 0).max(1, keepdims=True)  # the row's l has that error too
            n = nk + 16
            # numbers below the smallest normal one (the same for fp32 and bf16) become zero: a
            # weight, a product of one and a sum are each off by TINY at most, absolutely
            low = np.where(mask, TINY, 0.0)
            out["o"][rows, h] = (p * (e + top + w_round + n * T) + low) @ np.abs(vv) * (
                1 + half(dt)) + TINY
            out["lse"][rows, h] = (top + n * U + 4 * U * (np.abs(l) + 1))[:, 0]
            # backward: p from the given lse; dP and delta D products each
            dp = do @ vv.T - (do * o[rows, h]).sum(1, keepdims=True)
            adp = (np.abs(do) @ np.abs(vv).T * (D + 8) * T
                   + (np.abs(do) * np.abs(o[rows, h])).sum(1, keepdims=True) * (D + 8) * U
                   + 2 * U * np.abs(dp))
            ds = p * (np.abs(dp) * (e + w_round) + adp * (1 + e + w_round)) + low * (
                1 + np.abs(dp) + adp)
            terms = p * np.abs(dp)
            m = (nq * G + 16) * T
            out["dq"][rows, h] = (ds + terms * (n * T)) @ np.abs(kk) * sc + TINY
            out["dk"][keys, h // G] += (ds + terms * m).T @ np.abs(qq) * sc + TINY
            out["dv"][keys, h // G] += (p * (e + w_round + m) + low).T @ np.abs(do) + TINY
    return out


def rows_of(cu, n):
    at = np.zeros(n, bool)
    at[cu[0]:cu[-1]] = True
    return at


def check_seq(lens, klens, Hq, Hk, D, dt, causal, seed=0, scale=None, q_scale=1.0):
    q, k, v, cu, ck = seq_inputs(lens, klens, Hq, Hk, D, dt, seed, scale=q_scale)
    gen = torch.Generator().manual_seed(seed + 1)
    kw = dict(causal=causal, scale=scale or 0.0)
    cuq, cuk = i32(cu), None if klens is None and len(q) == len(k) else i32(ck)
    word = gdn.status_word()
    o = torch.full(q.shape, 7.0, dtype=dt, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    got = gdn.gdn_attn_fwd(q, k, v, cuq, cuk, o=o, lse=lse, status=word, **kw)
    assert got[0] is o and got[1] is lse
    inq, ink = rows_of(cu, len(q)), rows_of(ck, len(k))
    nq, nk = torch.from_numpy(~inq).cuda(), torch.from_numpy(~ink).cuda()
    assert (o[nq] == 7).all() and (lse[nq] == 7).all()  # rows of no sequence: as they were
    z = [x.masked_fill(m[:, None, None], 0) for x, m in ((q, nq), (k, nk), (v, nk))]
    ro, rl = attention.attn_fwd(*(n64(x) for x in z), cu, ck, causal, scale)
    dO = rand(gen, q.shape, dt)
    b = sums(*z, o.masked_fill(nq[:, None, None], 0), rl, dO, cu, ck, causal, scale)
    empty = np.isneginf(rl) & inq[:, None]
    assert (n64(o)[empty] == 0).all() and np.isneginf(n64(lse)[empty]).all()
    within("o", n64(o)[inq], ro[inq], (half(dt) * np.abs(ro) + b["o"])[inq])
    fin = np.where(np.isfinite(rl), rl, 0)
    within("lse", np.where(np.isfinite(rl), n64(lse), 0)[inq], fin[inq], b["lse"][inq])
    # backward, at the call's own o and lse; rows of no sequence hold NaN there too
    for x in (o, dO):
        x[nq] = float("nan")
    outs = [torch.full(x.shape, 7.0, dtype=dt, device="cuda") for x in (q, k, k)]
    gdn.gdn_attn_bwd(q, k, v, o, lse, dO, cuq, cuk, dq=outs[0], dk=outs[1], dv=outs[2],
                     status=word, **kw)
    clean = [x.masked_fill(nq[:, None, None], 0) for x in (o, dO)]
    refs = attention.attn_bwd(*(n64(x) for x in z), n64(clean[0]), n64(lse), n64(clean[1]), cu,
                              ck, causal, scale)
    b = sums(*z, clean[0], n64(lse), clean[1], cu, ck, causal, scale)
    for name, x, ref, rows, out in zip(("dq", "dk", "dv"), outs, refs, (inq, ink, ink),
                                       (nq, nk, nk)):
        assert (x[out] == 7).all(), name
        within(name, n64(x)[rows], ref[rows],
               ((half(dt) * np.abs(ref) + b[name]) * (1 + half(dt)))[rows])
    assert gdn.gdn_check_device_status(word) == gdn.GDN_OK
    again = gdn.gdn_attn_fwd(q, k, v, cuq, cuk, **kw)  # deterministic
    seq = torch.from_numpy(inq).cuda()
    assert torch.equal(again[0][seq], o[seq]) and torch.equal(again[1][seq], lse[seq])
    more = gdn.gdn_attn_bwd(q, k, v, o, lse, dO, cuq, cuk, **kw)
    for x, y, r in zip(outs, more, (inq, ink, ink)):
        at = torch.from_numpy(r).cuda()
        assert torch.equal(x[at], y[at])


EDGES = [1, 15, 16, 17, 0, 63, 64, 65]
TILES = [127, 128, 129, 255, 0, 256, 257]
CASES = [  # lens, key lens (None: the same), Hq, Hk, causal
    ([1], None, 1, 1, True), ([97], None, 4, 2, True), (EDGES, None, 6, 2, True),
    (TILES, None, 2, 1, True), ([700], None, 8, 1, True), ([40, 385, 3], None, 3, 3, False),
    (EDGES, [200, 15, 3, 0, 9, 300, 64, 130], 4, 2, True),   # contexts; rows that see no key
    (TILES, [128, 400, 129, 100, 5, 256, 700], 2, 1, True),
    (TILES, [128, 400, 129, 100, 5, 256, 700], 2, 1, False),
    ([3, 1, 200], [0, 0, 0], 2, 2, True), ([0, 0], [70, 3], 2, 1, False),
    ([2] * 300, None, 2, 1, True), ([1] * 9, [i * 50 for i in range(9)], 8, 1, True),
]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=[
    f"n{len(c[0])}_max{max(c[0])}_{'same' if c[1] is None else 'ctx' + str(max(c[1]))}_h{c[2]}x{c[3]}"
    f"{'' if c[4] else '_full'}" for c in CASES])
def test_attention_matches_definition(case, dt, D):
    lens, klens, Hq, Hk, causal = case
    check_seq(lens, klens, Hq, Hk, D, dt, causal, seed=len(lens) + D)


@pytest.mark.parametrize("D,dt", [(64, BF), (128, BF), (256, BF), (128, F32)])
def test_attention_longer_rows(D, dt):
    """Several blocks per tile, several turns of the ring, lists sorted by work."""
    check_seq([1500, 333, 20, 900], None, 4, 2, D, dt, True, seed=1)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_large_scores_and_given_scale(dt, D):
    """The row maximum moves far from block to block: the accumulator is rescaled."""
    check_seq([400, 150], None, 2, 1, D, dt, True, seed=2, scale=float(np.float32(0.11)),
              q_scale=20.0)


@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_rows_of_one_length_need_no_offsets(dt):
    gen = torch.Generator().manual_seed(3)
    B, n, m, Hq, Hk, D = 3, 50, 70, 4, 2, 128
    q, k, v = rand(gen, (B, n, Hq, D), dt), rand(gen, (B, m, Hk, D), dt), rand(gen, (B, m, Hk, D), dt)
    dO = rand(gen, q.shape, dt)
    o, lse = gdn.gdn_attn_fwd(q, k, v)
    grads = gdn.gdn_attn_bwd(q, k, v, o, lse, dO)
    assert o.shape == q.shape and lse.shape == q.shape[:3]
    cu, ck = i32(range(0, B * n + 1, n)), i32(range(0, B * m + 1, m))
    f = [x.flatten(0, 1) for x in (q, k, v, o, lse, dO)]
    want = gdn.gdn_attn_fwd(*f[:3], cu, ck)
    assert torch.equal(want[0], f[3]) and torch.equal(want[1], f[4])
    for x, y in zip(grads, gdn.gdn_attn_bwd(*f, cu, ck)):
        assert torch.equal(x.flatten(0, 1), y)
    one = gdn.gdn_attn_fwd(*(x[1].contiguous() for x in (q, k, v)))  # a single sequence
    assert torch.equal(one[0], o[1]) and torch.equal(one[1], lse[1])
    by_offsets = gdn.gdn_attn_fwd(*(x[1] for x in (q, k, v)), i32([0, n]), i32([0, m]))
    assert torch.equal(by_offsets[0], o[1])
    assert gdn.gdn_attn_fwd(q, k, v, want_lse=False)[1] is None


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_of_a_sequence_beside_one_of_nan(D, dt):
    """A packed sequence whose every number is NaN leaves its neighbours as they are without it."""
    lens = [40, 133, 55, 250, 7]
    q, k, v, cu, ck = seq_inputs(lens, [50, 133, 70, 300, 19], 4, 2, D, dt, seed=20)
    gen = torch.Generator().manual_seed(21)
    dO = rand(gen, q.shape, dt)
    cuq, cuk = i32(cu), i32(ck)
    want = gdn.gdn_attn_fwd(q, k, v, cuq, cuk)
    grads = gdn.gdn_attn_bwd(q, k, v, *want, dO, cuq, cuk)
    for b in (1, 3):
        for x, c in ((q, cu), (dO, cu), (k, ck), (v, ck)):
            x[c[b]:c[b + 1]] = float("nan")
    o, lse = gdn.gdn_attn_fwd(q, k, v, cuq, cuk)
    got = gdn.gdn_attn_bwd(q, k, v, o, lse, dO, cuq, cuk)
    for b in (0, 2, 4):
        rows, keys = slice(cu[b], cu[b + 1]), slice(ck[b], ck[b + 1])
        assert torch.equal(o[rows], want[0][rows]) and torch.equal(lse[rows], want[1][rows])
        for x, y, r in zip(got, grads, (rows, keys, keys)):
            assert torch.isfinite(y[r]).all() and torch.equal(x[r], y[r])


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 256])
def test_attention_without_keys_or_without_queries(D, dt):
    q = torch.randn(70, 4, D, device="cuda").to(dt)
    none = q[:0, :2]
    cu, zero = i32([0, 30, 70]), i32([0, 0, 0])
    o, lse = gdn.gdn_attn_fwd(q, none, none, cu, zero)
    assert not o.any() and torch.isneginf(lse).all()
    dq, dk, dv = gdn.gdn_attn_bwd(q, none, none, o, lse, q, cu, zero)
    assert not dq.any() and dk.shape == dv.shape == none.shape
    k = q[:, :2].contiguous()
    o, lse = gdn.gdn_attn_fwd(q[:0], k, k, zero, cu)
    dq, dk, dv = gdn.gdn_attn_bwd(q[:0], k, k, o, lse, o, zero, cu)
    assert dq.numel() == 0 and not dk.any() and not dv.any()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_few_new_tokens_behind_a_long_context(D):
    """The keys of every tile divided over several CTAs, and their parts joined."""
    check_seq([40, 3, 90], [3000, 9000, 90], 8, 2, D, BF, True, seed=22)
    check_seq([5], [5000], 4, 4, D, BF, False, seed=23)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_fp32_divides_keys_and_heads(D):
    """The same in fp32; and gradients whose key tiles are few, so that their query heads are divided
    (by 3 and by 5, where no power of two does) and tiles begin anywhere in a block of queries."""
    check_seq([40, 3, 90], [3000, 9000, 90], 8, 2, D, F32, True, seed=24)
    check_seq([5], [5000], 4, 4, D, F32, False, seed=25)
    check_seq([130, 0, 77], [300, 20, 77], 15, 1, D, F32, True, seed=26)
    check_seq([90, 1], [33, 100], 9, 3, D, F32, True, seed=27)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_sequences_without_work_among_others(D):
    """Beside one long context, sequences of a few keys and of none: they share a class of work, so
    that a CTA meets tiles without keys between others."""
    klens = [8000] + [(0, 5, 0, 16, 3, 0, 0)[i % 7] for i in range(450)]
    for seed in range(3):
        check_seq([1] * 451, klens, 4, 2, D, BF, True, seed=seed)
    check_seq([700] + [1 - i % 2 for i in range(450)], [700] + [(9, 4, 0, 16)[i % 4] for i in range(450)],
              4, 2, D, BF, True, seed=3)


@pytest.mark.parametrize("dt,D", [(BF, 128), (BF, 256), (F32, 64)])
def test_attention_rows_far_apart(dt, D):
    """Tokens 2^25 bytes apart: offsets past 2^32."""
    N, step = 150, 2 ** 25 // (2 if dt == BF else 4)
    big = torch.empty((N, step), dtype=dt, device="cuda")
    gen = torch.Generator().manual_seed(24)
    parts = [rand(gen, (N, h, D), dt) for h in (4, 2, 2)]
    views, at = [], 0
    for x in parts:
        y = big[:, at:at + x[0].numel()].view(x.shape)
        y.copy_(x)
        views.append(y)
        at += x[0].numel()
    cu, dO = i32([0, 60, 150]), rand(gen, parts[0].shape, dt)
    want = gdn.gdn_attn_fwd(*parts, cu)
    got = gdn.gdn_attn_fwd(*views, cu)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for x, y in zip(gdn.gdn_attn_bwd(*views, *got, dO, cu), gdn.gdn_attn_bwd(*parts, *want, dO, cu)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_outputs_aligned_to_16_bytes(D):
    """Outputs that begin in the middle of 32 bytes get the bits that others get, and nothing beside
    them is written."""
    q, k, v, cu, ck = seq_inputs([40, 300, 7], [90, 300, 7], 4, 2, D, BF, 31)
    cuq, cuk = i32(cu), i32(ck)
    dO = rand(torch.Generator().manual_seed(32), q.shape, BF)
    o, lse = gdn.gdn_attn_fwd(q, k, v, cuq, cuk, o=torch.full_like(q, 7.0))
    base = [torch.full_like(x, 7.0) for x in (q, k, k)]
    gdn.gdn_attn_bwd(q, k, v, o, lse, dO, cuq, cuk, dq=base[0], dk=base[1], dv=base[2])
    odd = []
    for x in (q, q, k, k):
        flat = torch.full((x.numel() + 16,), 7.0, dtype=BF, device="cuda")
        odd.append((flat, flat[8:8 + x.numel()].view(x.shape)))
        assert odd[-1][1].data_ptr() % 32 == 16
    gdn.gdn_attn_fwd(q, k, v, cuq, cuk, o=odd[0][1])
    gdn.gdn_attn_bwd(q, k, v, o, lse, dO, cuq, cuk, dq=odd[1][1], dk=odd[2][1], dv=odd[3][1])
    for (flat, x), want in zip(odd, [o] + base):
        assert torch.equal(x, want)
        assert (flat[:8] == 7).all() and (flat[-8:] == 7).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("n_seqs", [1, 3])
def test_attention_offsets_out_of_order_are_cut(dt, n_seqs):
    """No row outside the sequences is written; what is left of each is computed."""
    D, N = 64, 300
    gen = torch.Generator().manual_seed(4)
    q, k, v, dO = (rand(gen, (N, 2, D), dt) for _ in range(4))
    bad = [-5, 400] if n_seqs == 1 else [20, 150, 90, 1000]
    good = [0, 300] if n_seqs == 1 else [20, 150, 150, 300]
    word = gdn.status_word()
    o = torch.full(q.shape, 7.0, dtype=dt, device="cuda")
    lse = torch.zeros((N, 2), device="cuda")
    gdn.gdn_attn_fwd(q, k, v, i32(bad), o=o, lse=lse, status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_ERR_INVALID_ARG
    assert (o[:good[0]] == 7).all()
    want = gdn.gdn_attn_fwd(q, k, v, i32(good), status=word)
    assert torch.equal(o[good[0]:], want[0][good[0]:])
    got = gdn.gdn_attn_bwd(q, k, v, o, lse, dO, i32(bad), status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_ERR_INVALID_ARG
    for x, y in zip(got, gdn.gdn_attn_bwd(q, k, v, o, lse, dO, i32(good), status=word)):
        assert torch.equal(x[good[0]:], y[good[0]:])
    assert gdn.gdn_check_device_status(word) == gdn.GDN_OK


@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_gradients_match_differences(dt):
    """The loss of the fp64 definition at inputs moved along the call's own gradient."""
    q, k, v, cu, ck = seq_inputs([30, 45], [40, 50], 4, 2, 64, dt, seed=5, tail=0)
    q, k, v = q[2:].contiguous(), k[3:].contiguous(), v[3:].contiguous()
    cu, ck = cu - 2, ck - 3
    dO = rand(torch.Generator().manual_seed(6), q.shape, dt)
    o, lse = gdn.gdn_attn_fwd(q, k, v, i32(cu), i32(ck))
    grads = gdn.gdn_attn_bwd(q, k, v, o, lse, dO, i32(cu), i32(ck))
    x = [n64(t) for t in (q, k, v)]
    exact = attention.attn_bwd(*x, *attention.attn_fwd(*x, cu, ck), n64(dO), cu, ck)
    for i, g in enumerate(grads):
        d = n64(g) / np.linalg.norm(n64(g))
        def loss(t):
            y = [a + t * d if j == i else a for j, a in enumerate(x)]
            return (attention.attn_fwd(*y, cu, ck)[0] * n64(dO)).sum()
        slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
        # the call's gradient along itself is its norm; its error against the exact one is bounded
        # by check_seq's terms: three roundings to bf16 of sums that cancel (p, ds, the result)
        tol = (6 * half(BF) if dt == BF else 2.0 ** -16) * np.linalg.norm(exact[i]) + 1e-6
        assert abs(slope - np.linalg.norm(n64(g))) <= tol


def test_attention_captured_and_on_another_stream():
    """A captured step of forward and backward, replayed on changed inputs and lengths."""
    D, N = 128, 520
    gen = torch.Generator().manual_seed(7)
    q, k, v, dO = (rand(gen, (N, 2, D), BF) for _ in range(4))
    cu = i32([0, 100, 300, 520])

    def step():
        o, lse = gdn.gdn_attn_fwd(q, k, v, cu)
        return (o, lse, *gdn.gdn_attn_bwd(q, k, v, o, lse, dO, cu))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    graph.replay()
    for a, b in zip(outs, first):
        assert torch.equal(a, b)
    cu.copy_(i32([0, 7, 400, 520]))
    for x in (q, k, v, dO):
        x.copy_(rand(gen, x.shape, BF))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, step()):
        assert torch.equal(a, b)
    # a stream that is given, with outputs and workspaces made for it
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        q.mul_(0.5)
    got = gdn.gdn_attn_fwd(q, k, v, cu, stream=side)
    side.synchronize()
    want = gdn.gdn_attn_fwd(q, k, v, cu)
    assert torch.equal(got[0], want[0])


def test_attention_argument_checks():
    q, k = torch.zeros(10, 4, 64, device="cuda", dtype=BF), torch.zeros(10, 2, 64, device="cuda", dtype=BF)
    cu = i32([0, 10])
    with pytest.raises(ValueError):
        gdn.gdn_attn_fwd(q, k, k.float(), cu)
    with pytest.raises(ValueError):
        gdn.gdn_attn_fwd(q, k, k[:9], cu)
    with pytest.raises(ValueError):
        gdn.gdn_attn_fwd(q, k, k, cu.long())
    with pytest.raises(ValueError):
        gdn.gdn_attn_fwd(q, k, k, None, cu)
    with pytest.raises(ValueError):
        gdn.gdn_attn_fwd(q, k, k, cu, i32([0, 5, 10]))
    with pytest.raises(ValueError):
        gdn.gdn_attn_fwd(q, k, k, cu, o=q.float())
    with pytest.raises(ValueError):
        gdn.gdn_attn_fwd(q.cpu(), k, k, cu)
    with pytest.raises(ValueError):
        gdn.gdn_attn_fwd(q[:1].expand(10, 4, 64), k, k, cu)
    with pytest.raises(gdn.GDNError):
        gdn.gdn_attn_fwd(q, k[:5], k[:5], cu)  # one set of offsets, two lengths
    with pytest.raises(gdn.GDNError):
        gdn.gdn_attn_fwd(q, k, k, i32([0, 4, 10]),
                         ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(gdn.GDNError):
        gdn.gdn_attn_fwd(q[:, :3], k, k, cu)
    empty = gdn.gdn_attn_fwd(q[:0], k[:0], k[:0], cu * 0)
    assert empty[0].shape == (0, 4, 64)


# --------------------------------------------------------------------------- the 8-bit cache

def filled(gen, pages, P, Hk, D):
    """Codes and scales of earlier steps: every code but NaN, scales over 30 powers of two."""
    codes = torch.randint(0, 254, (pages, P, Hk, D), generator=gen).to(torch.uint8)
    codes += (codes >= 127).to(torch.uint8)
    scale = torch.randint(-20, 10, (pages, P // 16, Hk), generator=gen)
    return codes.cuda().view(F8), torch.pow(2.0, scale.double()).float().cuda()


def step_of(ctx, new, P, extra=3, seed=0):
    gen = torch.Generator().manual_seed(seed)
    counts = [-(-(c + n) // P) for c, n in zip(ctx, new)]
    pages = sum(counts) + extra
    perm = torch.randperm(pages, generator=gen).numpy()
    table = np.full((len(ctx), max(max(counts), 1)), 10 ** 9)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = perm[at:at + c]
        at += c
    return table, pages, np.cumsum([0] + list(new))


def same(name, got, want):
    assert np.array_equal(got, want), f"{name}: {np.argwhere(got != want)[:5]}"


def u8(x):
    return x.view(torch.uint8).cpu().numpy()


def check_cache(ctx, new, Hk, D, P, dt, seed=0, tail=3, make=None):
    gen = torch.Generator().manual_seed(seed)
    table, pages, cu = step_of(ctx, new, P, seed=seed)
    N = int(cu[-1]) + tail
    kv = rand(gen, (N, 2 * Hk, D)) * torch.exp(3 * rand(gen, (N, 2 * Hk, 1)))
    kv = kv.to(dt)
    if make is not None:
        make(kv)
    k, v = kv[:, :Hk], kv[:, Hk:]
    caches = [filled(gen, pages, P, Hk, D) for _ in range(2)]
    before = [(u8(c).copy(), n64(s)) for c, s in caches]
    args = (caches[0][0], caches[1][0], caches[0][1], caches[1][1], i32(table))
    word = gdn.status_word()
    gdn.gdn_cache_write8(k, v, *args, i32(ctx), i32(cu), status=word)
    whole = np.cumsum([0] + [c + n for c, n in zip(ctx, new)])
    n = int(whole[-1]) + tail
    outs = [torch.full((n, Hk, D), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    gdn.gdn_cache_read8(*args, i32(whole), k=outs[0], v=outs[1], status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_OK
    for x, (codes, scale), (c0, s0), out in zip((k, v), caches, before, outs):
        rc, rs = attention.cache_write8(n64(x), c0, s0, table, ctx, cu)
        same("codes", u8(codes), rc)  # rows and scales that no token went to among them
        same("scales", n64(scale), rs)
        back = attention.cache_read8(rc, rs, table, whole, n)
        got = n64(out)
        assert (got[whole[-1]:] == 7).all()
        # e4m3 times a power of two is exact in bf16 and fp32, but for 256 x 2^120 = 2^128, to which
        # numbers from 248 x 2^120 on are rounded: past the largest finite number, infinity
        want = n64(torch.from_numpy(back[:whole[-1]]).to(dt))
        np.testing.assert_array_equal(got[:whole[-1]], want)


CACHE = [  # ctx, new, Hk, page
    ([0], [1], 1, 16), ([15], [1], 2, 16), ([15, 16, 17, 0], [2, 1, 40, 0], 3, 48),
    ([0, 5, 31, 100, 0], [100, 0, 1, 33, 16], 2, 32), ([7] * 70, [i % 3 for i in range(70)], 2, 16),
    ([i * 3 % 50 for i in range(700)], [1] * 700, 1, 16), ([3, 0, 77], [500, 1, 300], 8, 64),
]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CACHE, ids=[f"B{len(c[0])}_N{sum(c[1])}_h{c[2]}_p{c[3]}"
                                             for c in CACHE])
def test_cache_written_and_read_back(case, dt, D):
    ctx, new, Hk, P = case
    check_cache(ctx, new, Hk, D, P, dt, seed=len(ctx) + D)


@pytest.mark.parametrize("dt", [BF, F32])
def test_cache_of_extreme_and_non_finite_numbers(dt):
    """Largest and smallest numbers, zeros, infinities and NaN, alone and among others."""
    def make(kv):
        kv[0:16] = 0.0
        kv[16:32] *= 2.0 ** 120
        kv[32:48] *= 2.0 ** -120
        kv[48:64, :, ::3] = float("inf")
        kv[50, :, 1::3] = float("nan")
        kv[64:80] = float("-inf")
        kv[80] = torch.finfo(kv.dtype).max
        kv[81] = torch.finfo(kv.dtype).tiny
        kv[96:112, :, 0] = 448.0 * 2.0 ** 7
        kv[112:128, :, 0] = 449.0 * 2.0 ** 7
        kv[100, :, 1:] = 2.0 ** -30
    check_cache([0, 20], [130, 40], 2, 64, 16, dt, seed=8, make=make)


def test_cache_tokens_without_a_page_are_left_out():
    gen = torch.Generator().manual_seed(9)
    P, Hk, D = 16, 2, 64
    ctx, new = [10, -4, 0], [40, 20, 10]
    table, pages, cu = step_of([10, 0, 0], new, P, seed=9)
    table[0, 2], table[1, 1] = pages, -1
    table = table[:, :3]                       # request 0's last tokens are past the table
    k, v = rand(gen, (70, Hk, D), BF), rand(gen, (70, Hk, D), BF)
    (kc, ks), (vc, vs) = filled(gen, pages, P, Hk, D), filled(gen, pages, P, Hk, D)
    rc, rs = attention.cache_write8(n64(k), u8(kc).copy(), n64(ks), table, ctx, cu)
    word = gdn.status_word()
    gdn.gdn_cache_write8(k, v, kc, vc, ks, vs, i32(table), i32(ctx), i32(cu), status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_ERR_INVALID_ARG
    same("codes", u8(kc), rc)
    same("scales", n64(ks), rs)
    whole = np.cumsum([0, 50, 20, 10])
    back, _ = gdn.gdn_cache_read8(kc, vc, ks, vs, i32(table), i32(whole), n_tokens=80, status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_ERR_INVALID_ARG
    np.testing.assert_array_equal(n64(back), attention.cache_read8(rc, rs, table, whole, 80))


@pytest.mark.parametrize("cu", [[0, 30, 20, 60], [0, 10, 20, 90], [-7, 10, 20, 60], [5, 5, 5, 5]])
def test_cache_offsets_that_are_not_ordered_write_nothing_outside(cu):
    """Bad offsets are recorded; pages of no request stay as they are."""
    gen = torch.Generator().manual_seed(10)
    P, Hk, D = 16, 1, 64
    table, pages, _ = step_of([0, 0, 0], [96, 96, 96], P, seed=10)
    k = rand(gen, (60, Hk, D), BF)
    (kc, ks), (vc, vs) = filled(gen, pages, P, Hk, D), filled(gen, pages, P, Hk, D)
    before = u8(kc).copy()
    word = gdn.status_word()
    gdn.gdn_cache_write8(k, k, kc, vc, ks, vs, i32(table), i32([0, 0, 0]), i32(cu), status=word)
    fine = cu == sorted(cu) and cu[0] >= 0 and cu[-1] <= 60
    assert gdn.gdn_check_device_status(word) == (gdn.GDN_OK if fine else gdn.GDN_ERR_INVALID_ARG)
    unused = sorted(set(range(pages)) - set(table.ravel().tolist()))
    assert (u8(kc)[unused] == before[unused]).all()
    out = torch.full((60, Hk, D), 7.0, dtype=BF, device="cuda")
    gdn.gdn_cache_read8(kc, vc, ks, vs, i32(table), i32(cu), k=out, v=out.clone(), status=word)
    if fine:
        assert (out == 7).all() and (u8(kc) == before).all()


def test_cache_past_2_32_bytes():
    """The last pages of a cache of 4.5 GB: written, read back and attended to."""
    P, Hk, D, pages = 128, 8, 256, 18000
    gen = torch.Generator().manual_seed(25)
    kc, vc = (torch.empty((pages, P, Hk, D), dtype=F8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, P // 16, Hk), device="cuda") for _ in range(2))
    table, ctx, cu = np.array([[pages - 1, 3], [pages - 2, pages - 5]]), [0, 0], [0, 150, 350]
    k, v = rand(gen, (350, Hk, D), BF), rand(gen, (350, Hk, D), BF)
    gdn.gdn_cache_write8(k, v, kc, vc, ks, vs, i32(table), i32(ctx), i32(cu))
    back = gdn.gdn_cache_read8(kc, vc, ks, vs, i32(table), i32(cu), n_tokens=350)
    small = np.array([[0, 1], [2, 3]])
    args = []
    for x in (k, v):
        zero = np.zeros((4, P, Hk, D), np.uint8), np.zeros((4, P // 16, Hk))
        args.append(attention.cache_write8(n64(x), *zero, small, ctx, cu))
    for x, c in zip(back, args):
        np.testing.assert_array_equal(n64(x), attention.cache_read8(*c, small, cu, 350))
    q = rand(gen, (2, 16, D), BF)
    o, lse = gdn.gdn_attn_decode8(q, kc, vc, ks, vs, i32(table), i32([150, 200]))
    near = [torch.from_numpy(c[0]).cuda().view(F8) for c in args]
    sc = [torch.from_numpy(c[1]).float().cuda() for c in args]
    want = gdn.gdn_attn_decode8(q, *near, *sc, i32(small), i32([150, 200]))
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


# ------------------------------------------------------------------ decode over the 8-bit cache

def dec_inputs(lens, Hq, Hk, D, P, dt, seed=0, spread=2.0, q_scale=1.0):
    """Shuffled pages; rows past each length and unused pages hold NaN codes, scales of unused
    blocks NaN, unused table entries a page far outside the cache."""
    gen = torch.Generator().manual_seed(seed)
    table, pages, _ = step_of([0] * len(lens), lens, P, seed=seed)
    caches = []
    for _ in range(2):
        codes = (100 * rand(gen, (pages, P, Hk, D))).clamp(-448, 448).to(F8)
        exp = (spread * rand(gen, (pages, P // 16, Hk))).round() - 7
        scale = torch.pow(2.0, exp.double()).float()
        dead = np.ones((pages, P), bool)
        for b, n in enumerate(lens):
            for j in range(n):
                dead[table[b, j // P], j % P] = False
        codes.view(torch.uint8)[torch.from_numpy(dead).cuda()] = 0x7f
        scale[torch.from_numpy(dead.reshape(pages, -1, 16).all(2)).cuda()] = float("nan")
        caches.append((codes, scale))
    q = (q_scale * rand(gen, (len(lens), Hq, D))).to(dt)
    return q, caches[0][0], caches[1][0], caches[0][1], caches[1][1], i32(table), i32(lens)


def check_dec(q, kc, vc, ks, vs, table, lens, o, lse, scale=None):
    """Score: q in f16 terms (2^-11 of what is below 2^-27 of the row's largest is all that bf16
    loses; fp32: 2^-22 of q), D products on tensor cores, two factors; as check_seq's else.  The
    weights are one f16 number (2^-11) or two (2^-22) down to 2^-34 of the largest weight times the
    largest scale of V (a quarter of it is where f16's steps stop shrinking: 2^-24 / 2^9, rounded
    to half, 4 below the largest scale, and 2^4 above the smallest reference)."""
    dt, D = q.dtype, q.shape[-1]
    sc = scale or D ** -0.5
    kv, vv = (attention.values(u8(c), np.nan_to_num(n64(s))) for c, s in ((kc, ks), (vc, vs)))
    table, lens = table.cpu().numpy(), lens.cpu().numpy()
    ro, rl = decode.attn_decode(n64(q), kv, vv, table, lens, sc)
    bo, bl = np.zeros(ro.shape), np.zeros(rl.shape)
    P, G = kc.shape[1], q.shape[1] // kc.shape[2]
    one, two = (2.0 ** -11, 2.0 ** -27) if dt == BF else (2.0 ** -22, 2.0 ** -22)
    for b, n in enumerate(lens):
        ids = table[b, :-(-n // P)]
        ids = ids[(ids >= 0) & (ids < len(kv))]
        rows = np.concatenate([np.arange(P) + i * P for i in range(-(-n // P))
                               if 0 <= table[b, i] < len(kv)]) if n else []
        live = [r for r in range(len(rows)) if rows[r] < n]
        if not live:
            continue
        k, v = kv[ids].reshape(-1, *kv.shape[2:])[live], vv[ids].reshape(-1, *vv.shape[2:])[live]
        top_v = np.nanmax(np.where(np.isfinite(n64(vs)[ids]), n64(vs)[ids], 0), axis=(0, 1))
        for h in range(q.shape[1]):
            x, y = k[:, h // G], n64(q[b, h])
            s = x @ y * sc
            S = np.abs(x) @ np.abs(y) * sc * ((D + 8) * T + two)
            e = S + 4 * U * (np.abs(s) + np.abs(s).max() + 1) + 2.0 ** -21
            w = np.exp(s - rl[b, h])
            m = np.exp(s.max() - rl[b, h])  # the largest weight
            m_steps = (len(live) + 16) * T
            tiny = 2.0 ** -34 * m * 2.0 ** 4 * top_v[h // G] * 448 * len(live)
            bo[b, h] = (w * (e + e.max() + one + m_steps)) @ np.abs(v[:, h // G]) + tiny
            bl[b, h] = e.max() + (len(live) + 16) * U + 4 * U * (abs(rl[b, h]) + 1)
    within("o", o, ro, (half(dt) * np.abs(ro) + bo) * (1 + half(dt)))
    live = np.isfinite(rl)
    assert np.isneginf(n64(lse)[~live]).all() and (n64(o)[~live] == 0).all()
    within("lse", np.where(live, n64(lse), 0), np.where(live, rl, 0), bl)


DEC = [  # lens, Hq, Hk, D, page, dtype
    ([1], 1, 1, 64, 16, BF), ([1], 1, 1, 64, 16, F32),
    ([0, 1, 15, 16, 17, 63, 64, 65], 8, 2, 128, 16, BF),
    ([0, 1, 15, 16, 17, 63, 64, 65], 8, 2, 128, 16, F32),
    ([31, 32, 33, 0, 0, 47, 48, 49], 16, 2, 256, 48, BF),
    ([31, 32, 33, 0, 0, 47, 48, 49], 6, 2, 256, 48, F32),
    ([127, 128, 129, 255, 257, 1000, 3], 4, 4, 64, 32, BF),
    ([127, 128, 129, 255, 257, 1000, 3], 4, 4, 64, 32, F32),
    ([5000], 16, 1, 128, 64, BF), ([5000], 12, 1, 128, 64, F32), ([9011], 8, 1, 256, 16, BF),
    ([9011], 3, 1, 64, 16, F32), ([700, 1, 9001, 0, 40, 333], 24, 8, 128, 16, BF),
    ([0, 0, 0], 8, 2, 128, 16, BF), (list(range(1, 200, 3)), 10, 2, 128, 16, BF),
    ([2] * 700, 8, 1, 64, 16, BF), ([1500], 8, 1, 256, 16, F32),
    ([300, 0, 17, 1100], 9, 1, 64, 16, BF), ([300, 0, 17, 1100], 32, 2, 256, 16, BF),
    ([300, 0, 17, 700], 17, 1, 128, 16, F32), ([300, 0, 17, 700], 24, 2, 256, 16, F32),
    ([300, 0, 17, 700], 40, 1, 64, 16, F32), ([2500], 13, 1, 256, 48, BF),
    ([2000, 300], 20, 1, 128, 128, BF),
]


@pytest.mark.parametrize("case", DEC, ids=[
    f"B{len(c[0])}_max{max(c[0])}_h{c[1]}x{c[2]}_d{c[3]}_p{c[4]}_{'bf16' if c[5] == BF else 'f32'}"
    for c in DEC])
def test_decode8_matches_definition(case):
    lens, Hq, Hk, D, P, dt = case
    inp = dec_inputs(lens, Hq, Hk, D, P, dt, seed=len(lens) + D)
    word = gdn.status_word()
    o, lse = gdn.gdn_attn_decode8(*inp, status=word)
    check_dec(*inp, o, lse)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_OK
    again = gdn.gdn_attn_decode8(*inp)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode8_fp32_error_on_the_whole(D):
    """Root mean square over o.  Scores (of about 1): q's two terms 2^-22, at random; sums of 64
    columns 4 cuts of 2^-24 on average.  Weights: exp 2^-22, two terms 2^-22; o's sums 4 cuts.  In
    quadrature (sums of cuts in full): sqrt(3 (2^-22)^2 + (2^-22)^2 + (2^-22)^2) < 2^-20."""
    lens = [517, 131, 9, 300]
    inp = dec_inputs(lens, 16, 2, D, 16, F32, seed=D + 5, spread=0.5)
    o, _ = gdn.gdn_attn_decode8(*inp)
    q, kc, vc, ks, vs, table, n = inp
    kv, vv = (attention.values(u8(c), np.nan_to_num(n64(s))) for c, s in ((kc, ks), (vc, vs)))
    ref, _ = decode.attn_decode(n64(q), np.nan_to_num(kv), np.nan_to_num(vv), table.cpu().numpy(),
                                n.cpu().numpy(), D ** -0.5)
    assert np.linalg.norm(n64(o) - ref) <= 2.0 ** -20 * np.linalg.norm(ref)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode8_large_scores_far_scales_and_given_scale(dt, D):
    """Scores and V's scales that move over many powers of two from block to block."""
    inp = dec_inputs([700, 33], 4, 2, D, 16, dt, seed=11, spread=6.0, q_scale=5.0)
    o, lse = gdn.gdn_attn_decode8(*inp, scale=0.11)
    check_dec(*inp, o, lse, scale=float(np.float32(0.11)))


@pytest.mark.parametrize("dt", [BF, F32])
def test_decode8_queries_of_any_size(dt):
    """Rows of zeros, tiny and huge queries: the row's factor brings them into f16."""
    q, kc, vc, ks, vs, table, lens = dec_inputs([60, 200], 4, 1, 64, 16, dt, seed=12, spread=0.0)
    q[0, 0] = 0
    q[0, 1] *= 2.0 ** -60
    q[0, 2] *= 2.0 ** 10
    q[1, 3, ::2] *= 2.0 ** -30
    o, lse = gdn.gdn_attn_decode8(q, kc, vc, ks, vs, table, lens)
    check_dec(q, kc, vc, ks, vs, table, lens, o, lse)


def test_decode8_bad_pages_and_lengths_are_left_out():
    q, kc, vc, ks, vs, table, lens = dec_inputs([90, 130, 33, 20], 8, 2, 128, 16, BF, seed=13)
    kc.view(torch.uint8)[kc.view(torch.uint8) & 127 == 127] = 0x20
    vc.view(torch.uint8)[vc.view(torch.uint8) & 127 == 127] = 0x20
    ks.nan_to_num_(0.5)
    vs.nan_to_num_(0.5)
    table[0, 2], table[1, 0] = -1, kc.shape[0]
    table[3, 2:] = 0
    lens[2], lens[3] = -5, 10 ** 6
    word = gdn.status_word()
    o, lse = gdn.gdn_attn_decode8(q, kc, vc, ks, vs, table, lens, status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_ERR_INVALID_ARG
    lens[2], lens[3] = 0, table.shape[1] * 16
    check_dec(q, kc, vc, ks, vs, table, lens, o, lse)


# ------------------------------------------------------------------------- all of them together

def test_a_conversation_over_the_8_bit_cache():
    """Prompts, single tokens and a second prompt behind the cached context, as a server runs them:
    slots, norm and rotation, cache, attention.  Each attention against the definition over the
    values that the cache holds."""
    Hq, Hk, D, P, blocks, pages, rows = 4, 2, 128, 16, 12, 30, 192
    gen = torch.Generator().manual_seed(14)
    one = torch.ones(D, device="cuda")
    inv = torch.tensor([1e4 ** (-i / 32) for i in range(32)], device="cuda")
    kc, vc = (torch.zeros((pages, P, Hk, D), dtype=F8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, 1, Hk), device="cuda") for _ in range(2))
    table = torch.full((3, blocks), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=gen).int().cuda()
    ctx = i32([0, 0, 0])
    word = gdn.status_word()
    for new in ([50, 20, 1], [1, 1, 1], [1, 0, 1], [60, 33, 5], [1, 1, 1]):
        qkv = rand(gen, (rows, Hq + 2 * Hk, D), BF)
        seq, cu, pos, _, used = gdn.gdn_slot_map(ctx, i32(new), free, table, page_size=P,
                                                 pages=pages, n_tokens=rows, status=word)
        free = free[used.item():].contiguous()
        q, k = gdn.gdn_qk_norm_rope_fwd(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], one, one, inv, pos)
        v = qkv[:, Hq + Hk:]
        gdn.gdn_cache_write8(k, v, kc, vc, ks, vs, table, ctx, cu, status=word)
        if max(new) == 1:
            live = [b for b in range(3) if new[b]]
            at = cu[:-1].long()[live]
            o, lse = gdn.gdn_attn_decode8(q[at], kc, vc, ks, vs, table[live], seq[live],
                                          status=word)
            check_dec(q[at], kc, vc, ks, vs, table[live], seq[live], o, lse)
        else:
            ck = torch.nn.functional.pad(seq.cumsum(0), (1, 0)).int()
            K, V = gdn.gdn_cache_read8(kc, vc, ks, vs, table, ck, n_tokens=int(ck[-1]), status=word)
            o, lse = gdn.gdn_attn_fwd(q, K, V, cu, ck, status=word)
            n = int(cu[-1])
            ro, rl = attention.attn_fwd(n64(q), n64(K), n64(V), cu.tolist(), ck.tolist())
            b = sums(q, K, V, torch.zeros_like(q), rl, torch.zeros_like(q), cu.tolist(),
                     ck.tolist(), True, None)
            within("o", n64(o)[:n], ro[:n], (half(BF) * np.abs(ro) + b["o"])[:n])
        ctx = seq.clone()
    assert gdn.gdn_check_device_status(word) == gdn.GDN_OK


def test_a_training_step_of_the_attention_layer():
    """Norm and rotation, attention, and back: the gradients of the projection's slices against the
    chain of the definitions."""
    Hq, Hk, D, N = 4, 2, 64, 150
    gen = torch.Generator().manual_seed(15)
    qkv = rand(gen, (N, Hq + 2 * Hk, D), F32)
    wq, wk = 1 + 0.1 * rand(gen, (D,)), 1 + 0.1 * rand(gen, (D,))
    inv = torch.tensor([1e4 ** (-i / 16) for i in range(16)], device="cuda")
    cu, pos = [0, 60, 61, 150], torch.cat([torch.arange(n) for n in (60, 1, 89)]).int().cuda()
    q0, k0, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    q, k = gdn.gdn_qk_norm_rope_fwd(q0, k0, wq, wk, inv, pos)
    o, lse = gdn.gdn_attn_fwd(q, k, v, i32(cu))
    dO = rand(gen, o.shape)
    dq, dk, dv = gdn.gdn_attn_bwd(q, k, v, o, lse, dO, i32(cu))
    dq0, dk0, _, _ = gdn.gdn_qk_norm_rope_bwd(q0, k0, wq, wk, inv, pos, dq, dk)
    p, w, f = pos.cpu().numpy(), (n64(wq), n64(wk)), n64(inv)
    eq, ek = (decode.norm_rope_fwd(n64(x), y, p, f) for x, y in zip((q0, k0), w))
    eo, el = attention.attn_fwd(eq, ek, n64(v), cu, cu)
    gq, gk, gv = attention.attn_bwd(eq, ek, n64(v), eo, el, n64(dO), cu, cu)
    rq, _ = decode.norm_rope_bwd(n64(q0), w[0], p, f, gq)
    rk, _ = decode.norm_rope_bwd(n64(k0), w[1], p, f, gk)
    # fp32 throughout: chains of sums of 64 to 300 terms, 2^-24 each and 2^-21 of the exponentials
    for name, x, ref in (("o", o, eo), ("dq", dq0, rq), ("dk", dk0, rk), ("dv", dv, gv)):
        assert np.linalg.norm(n64(x) - ref) <= 2.0 ** -16 * np.linalg.norm(ref), name
