"""GPU tests of the decode-step calls at places where a definition is easily missed: softmax weights
that a short type cannot hold, infinite values, fp32 accuracy in the norm, an epsilon of zero or
above the rows' size, weight gradients that lose or double a token, and steps with fewer token rows
or narrower tables than their requests need.  Bounds are counted as in test_decode_gpu.py."""
import numpy as np
import pytest
import torch

import chunked_state_scan_gated_gb300 as gdn
from oracle import decode
from test_decode_gpu import (BF, F32, U, angle_err, attn_inputs, check_attn, check_slots, half, i32,
                             n64, rand, rope_inputs, slot_inputs, terms, within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load_library()


# ------------------------------------------------------------------------------ attention

@pytest.mark.parametrize("n", [2, 64, 640])
@pytest.mark.parametrize("D,Hq", [(64, 8), (64, 16), (128, 5), (128, 16), (256, 8), (256, 13)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_weights_are_not_held_in_the_cache_type(dt, D, Hq, n):
    """Even keys score 0 with v = 1, odd ones -a (exact in q's type, another a per head) with
    v = -1: o = tanh(a / 2).  The weight exp(-a) lies between the type's numbers, its rounding would
    be the same for every odd key, and o is small, so that nothing hides it.  Errors relative to 1 =
    sum |p v|: bf16 weights held as two terms 2^-15; exp 2^-21, in o and in the sum; the scale's and
    the difference's roundings 3 U of a < 1 / 2; n + 16 additions of 2^-22 at most; o's own."""
    q, kc, vc, table, lens = attn_inputs([n], Hq, 1, D, 16, dt, seed=30)
    a = (3 + 7 * torch.arange(Hq, device="cuda")) * 2.0 ** -9
    q.zero_()
    q[0, :, 0] = a.to(dt)
    assert torch.equal(q[0, :, 0].float(), a)
    ids = table[0, :-(-n // 16)].long()
    odd = (torch.arange(16, device="cuda") % 2).view(1, 16, 1)
    kc[ids] = torch.zeros(1, dtype=dt, device="cuda")
    kc[ids, :, :, 0] = -odd.to(dt)
    vc[ids] = (1 - 2 * odd).to(dt)[..., None]
    o, lse = gdn.gdn_attn_decode(q, kc, vc, table, lens, scale=1.0)
    p = np.exp(-n64(a))
    ref = np.repeat(((1 - p) / (1 + p))[:, None], D, 1)
    e = 2.0 ** -20 + 6 * U + (n + 16) * 2.0 ** -22
    within("o", o[0], ref, half(dt) * np.abs(ref)
           + (e + (2.0 ** -15 if dt == BF else 0.0)) * (1 + half(dt)))
    rl = np.log((1 + p) * n / 2)
    within("lse", lse[0], rl, e + 4 * U * np.abs(rl))


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 16), (256, 3), (256, 16)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_infinite_and_largest_values(dt, D, Hq, n):
    """Equal scores: an infinite value of a live row comes through as it is (weight 1, whose second
    term is zero), and two opposite ones are NaN; the other columns do not change.  A key of score
    -inf has no weight, however large its (finite) value."""
    q, kc, vc, table, lens = attn_inputs([n], Hq, 1, D, 16, dt, seed=31)
    ids = table[0, :-(-n // 16)].long()
    q.fill_(1.0)
    kc[ids] = 0.5
    vc[ids] = 3.0
    vc[ids[0], 0, 0, 3], vc[ids[-1], (n - 1) % 16, 0, 9] = float("inf"), -float("inf")
    vc[ids[0], 0, 0, 17] = float("inf")
    vc[ids[-1], (n - 1) % 16, 0, 17] = -float("inf")
    o, _ = gdn.gdn_attn_decode(q, kc, vc, table, lens)
    assert (o[0, :, 3] == float("inf")).all() and (o[0, :, 9] == -float("inf")).all()
    # one token: the second assignment stands alone
    assert (o[0, :, 17] == -float("inf")).all() if n == 1 else torch.isnan(o[0, :, 17]).all()
    rest = [d for d in range(D) if d not in (3, 9, 17)]
    within("o", o[0][:, rest], np.full((Hq, D - 3), 3.0),
           3 * (half(dt) + (n + 16) * 2.0 ** -22 + 2.0 ** -20))
    if n > 1:
        vc[ids] = 3.0
        kc[ids[1], 4] = -float("inf")
        vc[ids[1], 4] = torch.finfo(dt).max
        o, _ = gdn.gdn_attn_decode(q, kc, vc, table, lens)
        within("o", o[0], np.full((Hq, D), 3.0),
               3 * (half(dt) + (n + 16) * 2.0 ** -22 + 2.0 ** -20))


@pytest.mark.parametrize("D,Hq", [(64, 2), (64, 9), (128, 8), (128, 16), (256, 8), (256, 11)])
def test_attention_fp32_of_the_largest_numbers(D, Hq):
    """fp32 keys and values up to the type's largest are as exact as others: one key, whose weight is
    1, gives v; 8 keys of that size on queries that bring the scores back to 2 .. 16 (one product
    each, queries of 4 bits) weigh as they should: both splits cut off leave 2^-21 of an operand,
    scores 2^-21 and 3 U of the difference, exp 2^-21, in the weight and in the sum; o has its
    values' 2^-21 and 16 additions of 2^-22."""
    q, kc, vc, table, lens = attn_inputs([8], Hq, 1, D, 16, F32, seed=35)
    top = torch.finfo(F32).max
    page = table[0, 0].long()
    gen = torch.Generator().manual_seed(36)
    v = (0.5 + 0.5 * torch.rand((8, D), generator=gen)).cuda()
    vc[page, :8, 0] = v * top
    vc[page, 0, 0, 0] = -top
    o, _ = gdn.gdn_attn_decode(q, kc, vc, table, i32([1]))
    ref = n64(vc[page, 0, 0])[None].repeat(Hq, 0)
    within("o", o[0], ref, np.abs(ref) * (half(F32) + 2.0 ** -21))
    q.zero_()
    kc[page, :8] = 0.0
    row, at = torch.arange(8, device="cuda"), torch.arange(8, device="cuda") * 7
    kc[page, row, 0, at] = v[:, 0] * top
    q[0][:, at] = 2.0 ** -125 * (1 + torch.randint(0, 8, (Hq, 8), generator=gen) / 8).cuda()
    vc[page, :8, 0] = v
    o, lse = gdn.gdn_attn_decode(q, kc, vc, table, lens, scale=1.0)
    ro, rl = decode.attn_decode(n64(q), n64(kc), n64(vc), table.cpu().numpy(), [8], 1.0)
    e = 2 * (16 * (2.0 ** -21 + 3 * U) + 2.0 ** -21) + 2.0 ** -21 + 16 * 2.0 ** -22
    within("o", o, ro, e * np.abs(ro) + half(F32) * np.abs(ro))
    within("lse", lse, rl, e + 4 * U * np.abs(rl))


FP32 = [([65], 8, 1, 64), ([3000], 8, 2, 64), ([3000], 12, 1, 64), ([65], 8, 1, 128),
        ([5000, 70], 4, 2, 128), ([3000], 40, 2, 128), ([65], 8, 1, 256), ([5000, 70], 6, 2, 256),
        ([3000], 16, 1, 256), ([700, 1, 90], 26, 2, 256)]


@pytest.mark.parametrize("lens,Hq,Hk,D", FP32)
def test_attention_fp32_accuracy_in_the_norm(lens, Hq, Hk, D):
    """Two-term splits leave 2^-23 of an operand, a product 2^-22, a score (its terms' errors of
    random sign, sum |q k| scale up to 0.64 sqrt(D)) less than 2^-20, and a weight as much beside
    exp's 2^-21: relative errors of o that average out over keys and columns, 2^-19 in the norm
    with a factor to spare.  A tf32 product without its small terms is off by 2^-11."""
    inp = attn_inputs(lens, Hq, Hk, D, 16, F32, seed=32)
    o, lse = gdn.gdn_attn_decode(*inp)
    ro, rl = decode.attn_decode(*[n64(x) for x in inp[:3]], inp[3].cpu().numpy(),
                                inp[4].cpu().numpy())
    for b in range(len(lens)):
        for h in range(Hq):
            err = np.linalg.norm(n64(o[b, h]) - ro[b, h]) / np.linalg.norm(ro[b, h])
            assert err <= 2.0 ** -19, (b, h, err)
    assert np.abs(n64(lse) - rl).max() <= 2.0 ** -18


# ------------------------------------------------------------------ norm + rotation

# A lane adds the rows of its warp's groups one after another: at most 2 tokens of 9 groups and a
# part of a token's in the cases here; then 2 or 4 lanes, 8 warps; the CTAs' partials in fp64.
CHAIN = 64


def norm_bounds(x, w, f, inter, eps, angle):
    """(|n| of each rotated pair, its relative error) as check_rows of test_decode_gpu.py."""
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w
    return terms(n, inter, 2 * len(f)), 20 * U + angle


EPS = [(3, 3, 1, 64, 32, BF), (50, 5, 2, 64, 64, F32), (7, 1, 3, 128, 0, BF), (300, 7, 5, 128, 64, F32),
       (40, 3, 1, 256, 64, BF), (21, 9, 2, 80, 32, F32), (9, 1, 1, 8, 0, F32)]


@pytest.mark.parametrize("eps", [0.0, 0.1, 30.0])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("case", EPS, ids=["x".join(map(str, c[:5])) + (
    "_bf16" if c[5] == BF else "_f32") for c in EPS])
def test_rope_epsilon(case, inter, eps):
    """Forward and backward with an epsilon of zero (rows are not zero; the warp's places past the
    last head are) and with some that change the result."""
    N, Hq, Hk, D, R, dt = case
    q, k, _, wq, wk, f, _ = rope_inputs(N, Hq, Hk, D, R, dt, seed=33)
    gen = torch.Generator().manual_seed(34)
    dyq, dyk = rand(gen, (N, Hq, D), dt), rand(gen, (N, Hk, D), dt)
    eps32 = float(np.float32(eps))
    t = np.arange(N)
    yq, yk = gdn.gdn_qk_norm_rope_fwd(q, k, wq, wk, f, interleaved=inter, eps=eps)
    dq, dk, dwq, dwk = gdn.gdn_qk_norm_rope_bwd(q, k, wq, wk, f, None, dyq, dyk, interleaved=inter,
                                                eps=eps)
    ang = angle_err(t, n64(f))
    for name, x, w, y, dy, dx, dw in (("q", q, wq, yq, dyq, dq, dwq), ("k", k, wk, yk, dyk, dk, dwk)):
        x, w, dy = n64(x), n64(w), n64(dy)
        ref = decode.norm_rope_fwd(x, w, t, n64(f), inter, eps=eps32)
        A, e = norm_bounds(x, w, f, inter, eps32, ang)
        within(name, y, ref, half(dt) * np.abs(ref) + A * e * (1 + half(dt)))
        rdx, rdw = decode.norm_rope_bwd(x, w, t, n64(f), dy, inter, eps=eps32)
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps32)
        A, xr = terms(dy, inter, R), np.abs(x * r)
        e = 40 * U + ang
        tol = e * r * (A * np.abs(w) + xr * np.mean(A * np.abs(w) * xr, -1, keepdims=True))
        within("d" + name, dx, rdx, half(dt) * np.abs(rdx) + tol * (1 + half(dt)))
        tol = ((e + (CHAIN + 16) * U) * A * xr).sum((0, 1))
        within("dw" + name, dw, rdw, tol + U * np.abs(rdw))


TOKENS = [(4001, 17, 3, 128, 64, BF), (3001, 13, 5, 64, 64, BF), (2500, 12, 1, 256, 64, BF),
          (3003, 16, 9, 64, 32, F32), (2433, 3, 1, 64, 0, F32), (300, 1, 1, 128, 16, BF)]
TOKEN_IDS = ["x".join(map(str, c[:5])) for c in TOKENS]


@pytest.mark.parametrize("case", TOKENS, ids=TOKEN_IDS)
def test_rope_weight_gradient_counts_every_row_once(case):
    """Elements of size 1 with eps = 3: x r = x / 2 exactly (rsqrt: 2 units of 2^-23 at most).
    dy = x or 2 x without rotation: every row adds 1/2 or 1 to every column, so sums of small
    halves, exact in fp32 but for rsqrt's error: a row lost or counted twice is 1/2 at least."""
    N, Hq, Hk, D, _, dt = case
    gen = torch.Generator().manual_seed(N)
    w, none = torch.ones(D, device="cuda"), torch.empty(0, device="cuda")
    x = [torch.randint(0, 2, (N, H, D), generator=gen).mul(2).sub(1).to(dt).cuda() for H in (Hq, Hk)]
    m = [torch.randint(1, 3, (N, H, D), generator=gen).to(dt).cuda() for H in (Hq, Hk)]
    got = gdn.gdn_qk_norm_rope_bwd(*x, w, w, none, None, x[0] * m[0], x[1] * m[1], eps=3.0)[2:]
    for dw, y in zip(got, m):
        want = n64(y).sum((0, 1)) / 2
        tol = want.max() * (2.0 ** -22 + CHAIN * U)
        assert tol < 0.5
        within("dw", dw, want, tol)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("case", TOKENS, ids=TOKEN_IDS)
def test_rope_weight_gradient_to_its_own_roundings(case, inter):
    N, Hq, Hk, D, R, dt = case
    q, k, _, wq, wk, f, _ = rope_inputs(N, Hq, Hk, D, R, dt, seed=N + 1)
    gen = torch.Generator().manual_seed(N)
    dyq, dyk = rand(gen, (N, Hq, D), dt), rand(gen, (N, Hk, D), dt)
    _, _, dwq, dwk = gdn.gdn_qk_norm_rope_bwd(q, k, wq, wk, f, None, dyq, dyk, interleaved=inter)
    t = np.arange(N)
    for dw, x, w, dy in ((dwq, q, wq, dyq), (dwk, k, wk, dyk)):
        x, dy = n64(x), n64(dy)
        _, ref = decode.norm_rope_bwd(x, n64(w), t, n64(f), dy, inter)
        xr = np.abs(x) / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-6)
        tol = ((40 * U + angle_err(t, n64(f)) + (CHAIN + 16) * U) * terms(dy, inter, R) * xr)
        tol = tol.sum((0, 1)) + U * np.abs(ref)
        assert np.median(tol) < 0.02 * np.sqrt(np.mean(ref * ref))  # it would notice
        within("dw", dw, ref, tol)


# ------------------------------------------------------------------------------- slot map

def stale(table, pages, seed=0):
    """The table with its unused entries holding pages of other requests."""
    other = torch.from_numpy(np.random.default_rng(seed).integers(0, pages, tuple(table.shape)))
    return torch.where(table < 0, other.int().cuda(), table)


def check_step_is_whole(ctx, new, free, table, P, pages, n_tokens, ok):
    """Against the definition, and by itself: every length counts only tokens that have a row, every
    page that a length reaches was held before or is one of the first `used` free ones, none twice."""
    before = table.cpu().numpy()
    check_slots(ctx, new, free, table.clone(), P, pages, n_tokens, ok=ok)
    seq, cu, _, slots, used = (x.tolist() for x in gdn.gdn_slot_map(
        ctx, new, free, table, page_size=P, pages=pages, n_tokens=n_tokens))
    cap = table.shape[1] * P
    given, after = free.tolist()[:used[0]], table.cpu().numpy()
    assert len(given) == used[0] and cu[-1] <= n_tokens
    for b, c in enumerate(ctx.tolist()):
        assert min(c, cap) <= seq[b] <= min(c + cu[b + 1] - cu[b], cap)
        held = min(-(-c // P), table.shape[1])
        assert (after[b, :held] == before[b, :held]).all()
        fresh = after[b, held:-(-seq[b] // P)].tolist()
        assert fresh == given[:len(fresh)]
        del given[:len(fresh)]
    assert not given  # every page that was taken is in a table


@pytest.mark.parametrize("n_tokens", [0, 1, 6, 7, 29, 30, 31, 35, 41, 49, 50, 51, 59, 60, 61])
def test_slot_map_with_fewer_token_rows_than_tokens(n_tokens):
    c, w, free, table, pages = slot_inputs([10, 3, 40], [30, 20, 10], 8, 10, seed=1)
    check_step_is_whole(c, w, free, stale(table, pages), 8, pages, n_tokens, n_tokens >= 60)


@pytest.mark.parametrize("n_tokens", [0, 100, 767, 768, 769, 1023, 1024, 1025, 2000, 2047, 2100])
def test_slot_map_of_many_requests_cut_at_the_last_row(n_tokens):
    """2100 tokens of 700 requests: the cut falls on any of several blocks of requests and rows."""
    ctx, new = [(7 * b) % 50 for b in range(700)], [(b * 5) % 7 for b in range(700)]
    c, w, free, table, pages = slot_inputs(ctx, new, 4, 16, seed=2)
    assert sum(new) == 2100
    check_step_is_whole(c, w, free, stale(table, pages), 4, pages, n_tokens, n_tokens >= 2100)


@pytest.mark.parametrize("blocks", [0, 1, 2, 5, 6, 7, 8])
@pytest.mark.parametrize("n_tokens", [64, 45])
def test_slot_map_takes_no_page_past_the_table(blocks, n_tokens):
    """A request that its row of the table cannot hold takes no page that it has no entry for."""
    c, w, free, table, pages = slot_inputs([10, 40, 3, 0], [30, 15, 10, 5], 8, 8, seed=5)
    table = stale(table, pages)[:, :blocks].contiguous()
    check_step_is_whole(c, w, free, table, 8, pages, n_tokens, n_tokens == 64 and blocks >= 7)


def test_slot_map_arrays_side_by_side_in_one_block():
    """Arrays of one int32 block that touch and do not overlap, empty ones anywhere."""
    c, w, free, table, pages = slot_inputs([10, 3, 40], [30, 20, 10], 8, 10, seed=6)
    want = gdn.gdn_slot_map(c, w, free, table.clone(), page_size=8, pages=pages, n_tokens=64)
    sizes = [3, 3, free.numel(), table.numel(), 3, 4, 64, 64, 1]
    parts = list(torch.empty(sum(sizes), dtype=torch.int32, device="cuda").split(sizes))
    for p, x in zip(parts, (c, w, free, table.view(-1))):
        p.copy_(x)
    ctx, new, fr, tb, seq, cu, pos, slots, used = parts
    kw = dict(page_size=8, pages=pages, n_tokens=64)
    got = gdn.gdn_slot_map(ctx, new, fr, tb.view(3, 10), seq_len=seq, cu_seqlens=cu, positions=pos,
                           slots=slots, used=used, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    new.zero_()
    got = gdn.gdn_slot_map(ctx, new, fr, tb.view(3, 10), seq_len=seq, cu_seqlens=cu,
                           positions=used[:0], slots=used[:0], used=used, page_size=8, pages=pages,
                           n_tokens=0)
    assert torch.equal(got[0], ctx) and used.tolist() == [0] and not cu.any()
    with pytest.raises(gdn.GDNError):
        gdn.gdn_slot_map(ctx, new, fr, tb.view(3, 10), seq_len=seq, cu_seqlens=cu, positions=pos,
                         slots=slots, used=cu[3:], **kw)


def test_dropped_tokens_bring_no_other_request_into_the_attention():
    """Rows of the cache that the step does not write hold NaN; the tables' unused entries name
    such pages.  The attention over seq_len is over the rows that were written."""
    Hq, Hk, D, P, rows = 4, 2, 128, 16, 41
    c, w, free, table, pages = slot_inputs([0, 0, 0], [20, 30, 10], P, 4, seed=3)
    table = stale(table, pages)
    gen = torch.Generator().manual_seed(4)
    qkv, one = rand(gen, (rows, Hq + 2 * Hk, D), BF), torch.ones(D, device="cuda")
    kc, vc = (torch.full((pages, P, Hk, D), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    word = gdn.status_word()
    seq, cu, pos, slots, _ = gdn.gdn_slot_map(c, w, free, table, page_size=P, pages=pages,
                                              n_tokens=rows, status=word)
    q = gdn.gdn_qk_norm_rope_cache(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], one, one,
                                   torch.ones(8, device="cuda"), pos, slots, kc, vc, status=word)
    o, lse = gdn.gdn_attn_decode(q[:3].contiguous(), kc, vc, table, seq, status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_ERR_INVALID_ARG
    assert seq.tolist() == [20, 21, 0] and cu.tolist() == [0, 20, 41, 41]
    assert torch.isfinite(o).all() and torch.isfinite(lse[:2]).all()
    check_attn(q[:3].contiguous(), kc, vc, table, seq, o, lse)
