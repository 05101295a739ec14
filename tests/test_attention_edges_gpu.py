"""GPU tests of the full-attention calls and of the 8-bit cache at places where a definition is easily
missed: offsets out of order, blocks whose scale is far above the others', groups of query heads that a
tile holds whole, in part or twice over, fp32 accuracy in the norm.  Bounds are counted as in
test_attention_gpu.py."""
import numpy as np
import pytest
import torch

import chunked_state_scan_gated_gb300 as gdn
from oracle import attention, decode
from test_attention_gpu import (BF, F8, F32, U, check_cache, check_dec, check_seq, dec_inputs,
                                filled, i32, n64, rand, same, step_of, u8)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load_library()


# ------------------------------------------------------------------ attention over packed rows

GROUPS = [(16, 1), (32, 2), (48, 1), (6, 1), (12, 2), (24, 1), (5, 1)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hk", GROUPS)
def test_attention_of_groups_of_any_size(Hq, Hk, D):
    """A forward tile holds the largest power of two of a key head's query heads, up to 16: groups of
    16 and of several 16, and groups of which it holds a part; at ends of tiles of 8, 16 and 128 tokens,
    over the prompt and over a longer context."""
    lens = [7, 8, 9, 15, 16, 17, 129]
    check_seq(lens, None, Hq, Hk, D, BF, True, seed=Hq + D)
    check_seq(lens, [50, 8, 300, 15, 700, 9, 400], Hq, Hk, D, BF, True, seed=Hq + D + 1)
    check_seq([33, 2], [20, 140], Hq, Hk, D, BF, False, seed=Hq + D + 2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hk", GROUPS)
def test_attention_of_groups_of_any_size_with_divided_keys(Hq, Hk, D):
    """The same where the keys of every tile are divided and joined."""
    check_seq([5, 3, 17], [6000, 2500, 900], Hq, Hk, D, BF, True, seed=Hq + D + 3)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cu,ck,fine", [([0, 0], [0, 70], True), ([0, 3], [0, 70], False),
                                        ([0, 0], [-1, 70], False), ([0, 0], [0, 71], False),
                                        ([0, 0, 0], [0, 30, 70], True),
                                        ([0, 0, 1], [0, 30, 70], False)])
def test_attention_gradients_without_queries_check_their_offsets(cu, ck, fine, dt):
    k = torch.randn(70, 2, 64, device="cuda").to(dt)
    q, lse = torch.empty((0, 4, 64), dtype=dt, device="cuda"), torch.empty((0, 4), device="cuda")
    word = gdn.status_word()
    out = [torch.full_like(k, 7.0) for _ in range(2)]
    gdn.gdn_attn_bwd(q, k, k, q, lse, q, i32(cu), i32(ck), dk=out[0], dv=out[1], status=word)
    assert gdn.gdn_check_device_status(word) == (gdn.GDN_OK if fine else gdn.GDN_ERR_INVALID_ARG)
    assert not out[0].any() and not out[1].any()


# A rounding to fp32 is off by 0.425 U of the value in the root mean square (uniform within half a
# step, mantissas spread over their logarithm): STEP U^2.  A sum of n terms of random sign that is
# rounded at each is off by n STEP U^2 of its square at most (where the first terms are the largest;
# half of that where all are alike).
STEP = 0.425 ** 2


def fp32_errors(D, n, run):
    """Bounds (relative, in the norm) of o over n keys and of dq, dk, dv for q, k, v, dO of standard
    normal numbers: errors of a weight, in quadrature, with the sums', times 1.25.  Scores are of about
    1, sums of D products in two halves: STEP D / 4.  Forward: scaled and subtracted at 5 at most, ex2
    2^-22, n keys in two halves.  Backward: rounded at 8 (the lse of 1400 keys) once as a sum, once times
    log2(e), whose own error is 0.22 U; dP as the scores; gradients summed in runs of `run` rows."""
    score = STEP * D / 4
    o = score + STEP * (1 + 25) + 16 + STEP * n / 2
    p = score + 2 * STEP * 64 + (0.22 * 8) ** 2 + 16
    ds = p + score + 1
    return {k: 1.25 * U * x ** 0.5 for k, x in (("o", o), ("dq", ds + STEP * run),
                                                ("dk", ds + STEP * run), ("dv", p + STEP * run))}


def norm_within(name, x, ref, bound):
    err = np.linalg.norm(n64(x) - ref) / np.linalg.norm(ref)
    print(f"{name}: {err:.3g}, bound {bound:.3g}")
    assert err <= bound, (name, err, bound)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_fp32_error_on_the_whole(D):
    """1400 tokens, 16 query heads to a key head, so many key heads that no key tile's query heads are
    divided: 22,400 rows to a sum, which only runs of 16 blocks of 64 keep this accurate (in one run
    45 U and more).  One key head and its query heads against the definition."""
    n, Hk, G = 1400, 28, 16
    gen = torch.Generator(device="cuda").manual_seed(D)
    q, k, v, dO = (torch.randn((n, h, D), generator=gen, device="cuda")
                   for h in (Hk * G, Hk, Hk, Hk * G))
    o, lse = gdn.gdn_attn_fwd(q, k, v)
    dq, dk, dv = gdn.gdn_attn_bwd(q, k, v, o, lse, dO)
    at, hk = slice(9 * G, 10 * G), slice(9, 10)
    x = [n64(t) for t in (q[:, at], k[:, hk], v[:, hk])]
    bound = fp32_errors(D, n, 1024)
    norm_within("o", o[:, at], attention.attn_fwd(*x, [0, n], [0, n])[0], bound["o"])
    refs = attention.attn_bwd(*x, n64(o[:, at]), n64(lse[:, at]), n64(dO[:, at]), [0, n], [0, n])
    for name, got, ref in zip(("dq", "dk", "dv"), (dq[:, at], dk[:, hk], dv[:, hk]), refs):
        norm_within(name, got, ref, bound[name])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_fp32_error_over_a_long_context(D):
    """64 queries behind 12,224 keys, so many heads that no tile's keys are divided."""
    n, Hk, G = 12288, 19, 4
    gen = torch.Generator(device="cuda").manual_seed(D + 1)
    q = torch.randn((64, Hk * G, D), generator=gen, device="cuda")
    k, v = (torch.randn((n, Hk, D), generator=gen, device="cuda") for _ in range(2))
    o, _ = gdn.gdn_attn_fwd(q, k, v, i32([0, 64]), i32([0, n]))
    x = [n64(t) for t in (q[:, 8:12], k[:, 2:3], v[:, 2:3])]
    norm_within("o", o[:, 8:12], attention.attn_fwd(*x, [0, 64], [0, n])[0],
                fp32_errors(D, n, 1024)["o"])


# --------------------------------------------------------------------------- the 8-bit cache

def check_cut(cu, ctx, N, D, dt, P=16, Hk=2, seed=0, room=None):
    """Codes, scales and rows read back are those of the offsets as they count; `room` tokens (None: N)
    at most to a request."""
    gen = torch.Generator().manual_seed(seed)
    B = len(ctx)
    table, pages, _ = step_of([0] * B, [(room or N) + max(max(ctx), 0)] * B, P, seed=seed)
    caches = [filled(gen, pages, P, Hk, D) for _ in range(2)]
    before = [(u8(c).copy(), n64(s)) for c, s in caches]
    k, v = rand(gen, (N, Hk, D), dt), rand(gen, (N, Hk, D), dt)
    args = (caches[0][0], caches[1][0], caches[0][1], caches[1][1], i32(table))
    word = gdn.status_word()
    gdn.gdn_cache_write8(k, v, *args, i32(ctx), i32(cu), status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_ERR_INVALID_ARG
    outs = [torch.full((N, Hk, D), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    gdn.gdn_cache_read8(*args, i32(cu), k=outs[0], v=outs[1], status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_ERR_INVALID_ARG
    for x, (codes, scale), (c0, s0), out in zip((k, v), caches, before, outs):
        rc, rs = attention.cache_write8(n64(x), c0, s0, table, ctx, cu)
        same("codes", u8(codes), rc)
        same("scales", n64(scale), rs)
        want = attention.cache_read8(rc, rs, table, cu, N)
        np.testing.assert_array_equal(n64(out), np.where(np.isnan(want), 7.0, want))


@pytest.mark.parametrize("dt,D", [(BF, 64), (F32, 128), (BF, 256)])
@pytest.mark.parametrize("cu,ctx", [
    ([0, 30, 20, 60], [0, 0, 0]), ([0, 30, 20, 60], [5, 3, 33]), ([-7, 10, 20, 60], [0, 20, 1]),
    ([0, 10, 20, 90], [0, 0, 40]), ([9, 3, 50, 50], [1, 2, 3]), ([70, 10, 20, 30], [0, 0, 0]),
    ([0, 60, -2 ** 31, 2 ** 31 - 1], [7, 0, 0]), ([-9, -5, -1, 5], [0, 0, 0]),
])
def test_cache_offsets_out_of_order_are_cut(cu, ctx, dt, D):
    check_cut(cu, ctx, 60, D, dt)


def test_cache_offsets_out_of_order_among_many_requests():
    """More requests than a CTA has threads, the one bad offset far from most rows."""
    cu = list(range(701))
    cu[500] = 100
    check_cut(cu, [i % 20 for i in range(700)], 700, 64, BF, Hk=1)
    cu[500], cu[3] = 500, 650
    check_cut(cu, [i % 20 for i in range(700)], 700, 64, BF, Hk=1)


@pytest.mark.parametrize("dt,D", [(BF, 64), (F32, 64), (BF, 256)])
def test_cache_of_very_many_requests(dt, D):
    """So many that a CTA takes several runs of rows; the offsets in order, and not."""
    B = 6000
    new = [(0, 1, 2, 1, 5, 3, 1)[i % 7] for i in range(B)]
    ctx = [i * 7 % 40 for i in range(B)]
    check_cache(ctx, new, 1, D, 16, dt, seed=D)
    if D == 64:
        cu = np.cumsum([0] + new).tolist()
        cu[4000], cu[90], cu[5999] = cu[3993], cu[97], cu[5990]
        check_cut(cu, ctx, cu[-1], D, dt, Hk=1, room=40)


# ------------------------------------------------------------------ decode over the 8-bit cache

@pytest.mark.parametrize("place", [0, 7, 18])
@pytest.mark.parametrize("D,Hq,up", [(64, 16, 16), (128, 8, 24), (128, 32, 40), (256, 16, 30),
                                     (256, 32, 20)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_decode8_blocks_count_by_their_weight_whatever_their_scale(dt, D, Hq, up, place):
    """One block of V is 2^up larger than the others.  Odd heads see it alone (scores of about 60),
    even ones do not (-60), wherever it is.  Root mean square over each head's o: fp32 as in
    test_decode8_fp32_error_on_the_whole, 2^-20.  bf16: o's own rounding 2^-8 at most, weights 2^-11
    and scores 2^-19 far below it: 1.1 2^-8."""
    lens = [300, 517]
    q, kc, vc, ks, vs, table, n = dec_inputs(lens, Hq, 2, D, 16, dt, seed=D + place, spread=0.0)
    q.abs_()
    q[:, 1::2] *= -1
    for b in range(2):
        page = int(table[b, place])
        rows = min(16, lens[b] - 16 * place)
        kc[page, :rows] = torch.tensor(-1.0).to(F8)
        ks[page] = 60 / (0.8 * D ** 0.5)
        vs[page] *= 2.0 ** up
    o, lse = gdn.gdn_attn_decode8(q, kc, vc, ks, vs, table, n)
    kv, vv = (attention.values(u8(c), np.nan_to_num(n64(s))) for c, s in ((kc, ks), (vc, vs)))
    ref, rl = decode.attn_decode(n64(q), np.nan_to_num(kv), np.nan_to_num(vv), table.cpu().numpy(),
                                 n.cpu().numpy(), D ** -0.5)
    assert (np.abs(ref[:, 1::2]).max() > 2.0 ** (up - 6)) and np.abs(ref[:, ::2]).max() < 8
    err = np.linalg.norm(n64(o) - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
    assert err.max() <= (1.1 * 2.0 ** -8 if dt == BF else 2.0 ** -20), err
    assert np.abs(n64(lse) - rl).max() <= 2.0 ** -15 + 2.0 ** -19 * np.abs(rl).max()


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_decode8_scales_at_the_ends_of_their_range(dt):
    """V's scales of 2^-100, 2^100 and 0 (a block never written) beside each other; a context of
    zeros."""
    inp = dec_inputs([200, 60, 33], 8, 2, 64, 16, dt, seed=40, spread=0.0)
    vs, table = inp[4], inp[5]
    vs[table[0, :12].long()] = 2.0 ** -100
    for i, scale in enumerate((2.0 ** -100, 2.0 ** 100, 0.0)):
        vs[table[1, i].long()] = scale
    vs[table[2, :3].long()] = 0.0
    o, lse = gdn.gdn_attn_decode8(*inp)
    check_dec(*inp, o, lse)
    assert (o[0] != 0).any() and (o[2] == 0).all()
