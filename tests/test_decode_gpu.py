"""GPU parity of the decode-step calls against their fp64 definitions (oracle/decode.py; the core's
token recurrence for gdn_step), element by element.

Bounds.  `half(dtype)` = finfo.eps / 2 is one rounding to the output type; U = 2^-24 one fp32
rounding.  Each test adds to it the roundings of its call, relative to the sum of the absolute
values of the terms that are added (so cancellation is accounted for); the counts are written
beside each."""
import numpy as np
import pytest
import torch

import chunked_state_scan_gated_gb300 as gdn
import oracle
from oracle import decode

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


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
    x = n64(x)
    assert x.shape == ref.shape
    assert np.isfinite(x).all(), f"{name}: non-finite values"
    over = np.abs(x - ref) - bound
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, f"{name}{at}: {x[at]} against {ref[at]}, bound {np.broadcast_to(bound, x.shape)[at]}"


# ------------------------------------------------------------------------------ attention

def attn_inputs(lens, Hq, Hk, D, P, dt, seed=0, extra=3, qk_scale=1.0):
    """Shuffled pages; rows past each length and unused pages hold NaN, unused table entries a
    page far outside the cache."""
    gen = torch.Generator().manual_seed(seed)
    counts = [-(-n // P) for n in lens]
    pages, blocks = sum(counts) + extra, max(max(counts), 1) + 1
    perm = torch.randperm(pages, generator=gen).numpy()
    table = np.full((len(lens), blocks), 10 ** 9)
    dead = np.ones((pages, P), bool)
    at = 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        table[b, :c] = perm[at:at + c]
        for j in range(n):
            dead[table[b, j // P], j % P] = False
        at += c
    kc, vc = rand(gen, (pages, P, Hk, D), dt), rand(gen, (pages, P, Hk, D), dt)
    kc[torch.from_numpy(dead).cuda()] = float("nan")
    vc[torch.from_numpy(dead).cuda()] = float("nan")
    q = (qk_scale * rand(gen, (len(lens), Hq, D))).to(dt)
    return q, kc, vc, i32(table), i32(lens)


def check_attn(q, kc, vc, table, lens, o, lse, scale=None):
    """o = sum p v / l.  Score: D products, summed in at most D + 8 roundings of U, on tensor
    cores in steps that may each lose 2^-22 of the running magnitude: S = (D + 8) 2^-22 of
    sum |q k| scale.  exp: argument rounding U |s - m| (at most the score spread, bounded by 2 max
    |s|) and 2^-21 of its own.  The weights' error is then at most w = 2 S + 2 U (2 max|s| + 2) +
    2^-21, plus half a bf16 step where they are rounded for the product; sums over n keys, each
    of n + 16 roundings at most.  o also has its own rounding; lse the same without the weights'."""
    dt, D = q.dtype, q.shape[-1]
    ro, rl = decode.attn_decode(n64(q), n64(kc), n64(vc), table.cpu().numpy(), lens.cpu().numpy(),
                                scale)
    absv, S, top = np.zeros(ro.shape), np.zeros(rl.shape), np.zeros(rl.shape)
    sc = scale or D ** -0.5
    P, G = kc.shape[1], q.shape[1] // kc.shape[2]
    for b in range(len(ro)):
        n = int(lens[b])
        ids = table[b, :-(-n // P)].long()
        ok = (ids >= 0) & (ids < kc.shape[0])
        rows = ok.repeat_interleave(P)[:n]
        k = n64(kc[ids.clamp(0, kc.shape[0] - 1)].flatten(0, 1)[:n][rows])
        v = n64(vc[ids.clamp(0, kc.shape[0] - 1)].flatten(0, 1)[:n][rows])
        if not len(k):
            continue
        for h in range(q.shape[1]):
            s = k[:, h // G] @ n64(q[b, h]) * sc
            w = np.exp(s - rl[b, h])
            absv[b, h] = w @ np.abs(v[:, h // G])
            S[b, h] = (np.abs(k[:, h // G]) @ np.abs(n64(q[b, h]))).max() * sc * (D + 8) * 2.0 ** -22
            top[b, h] = np.abs(s).max()
    n = n64(lens)[:, None]
    w = 2 * S + 2 * U * (2 * top + 2) + 2.0 ** -21 + (n + 16) * U
    wo = w + (half(BF) if dt == BF else 0.0)
    within("o", o, ro, half(dt) * np.abs(ro) + wo[..., None] * absv * (1 + half(dt)))
    live = np.isfinite(rl)
    got = n64(lse)
    assert np.isneginf(got[~live]).all() and (n64(o)[~live] == 0).all()
    within("lse", torch.from_numpy(np.where(live, got, 0)), np.where(live, rl, 0),
           w + 4 * U * (np.abs(np.where(live, rl, 0)) + 1))


ATTN = [  # lens, Hq, Hk, D, page, dtype
    ([1], 1, 1, 64, 16, BF), ([1], 1, 1, 64, 16, F32),
    ([0, 1, 15, 16, 17, 63, 64, 65], 8, 2, 128, 16, BF),
    ([0, 1, 15, 16, 17, 63, 64, 65], 8, 2, 128, 16, F32),
    ([31, 32, 33, 0, 0, 47, 48, 49], 16, 2, 256, 48, BF),
    ([31, 32, 33, 0, 0, 47, 48, 49], 6, 2, 256, 48, F32),
    ([127, 128, 129, 255, 257, 1000, 3], 4, 4, 64, 32, BF),
    ([127, 128, 129, 255, 257, 1000, 3], 4, 4, 64, 32, F32),
    ([5000], 16, 1, 128, 64, BF), ([5000], 12, 1, 128, 64, F32),
    ([20011], 8, 1, 256, 16, BF), ([20011], 3, 1, 64, 16, F32),
    ([700, 1, 9001, 0, 40, 333], 24, 8, 128, 16, BF),
    ([700, 1, 2001, 0, 40, 333], 12, 4, 64, 128, BF),
    ([0, 0, 0], 8, 2, 128, 16, BF), ([0], 8, 2, 256, 16, F32),
    (list(range(1, 200, 3)), 10, 2, 128, 16, BF),
    ([2] * 700, 8, 1, 64, 16, BF),
    # parts joined: 11 and 24 by one warp per head, hundreds shared; many requests per lane
    ([700], 8, 1, 256, 16, BF), ([1500], 8, 1, 256, 16, BF), ([1500], 8, 1, 256, 16, F32),
    ([60011], 2, 1, 64, 64, BF), ([i % 7 for i in range(3000)], 2, 1, 64, 16, BF),
    ([(i * 37) % 301 for i in range(1111)], 2, 1, 64, 16, F32),
    # more than 8 query heads to a key head: 16 to a pass, the last pass not full
    ([300, 0, 17, 1100], 9, 1, 64, 16, BF), ([300, 0, 17, 1100], 32, 2, 256, 16, BF),
    ([300, 0, 17, 1100], 20, 1, 128, 32, BF), ([3000], 48, 2, 128, 16, BF),
    ([300, 0, 17, 700], 17, 1, 128, 16, F32), ([300, 0, 17, 700], 24, 2, 256, 16, F32),
    ([300, 0, 17, 700], 40, 1, 64, 16, F32), ([2500], 13, 1, 256, 48, BF),
]


@pytest.mark.parametrize("case", ATTN, ids=[
    f"B{len(c[0])}_max{max(c[0])}_h{c[1]}x{c[2]}_d{c[3]}_p{c[4]}_{'bf16' if c[5] == BF else 'f32'}"
    for c in ATTN])
def test_attention_matches_definition(case):
    lens, Hq, Hk, D, P, dt = case
    inp = attn_inputs(lens, Hq, Hk, D, P, dt, seed=len(lens) + D)
    word = gdn.status_word()
    o, lse = gdn.gdn_attn_decode(*inp, status=word)
    check_attn(*inp, o, lse)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_OK
    again = gdn.gdn_attn_decode(*inp)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])  # deterministic


@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_large_scores_and_given_scale(dt):
    inp = attn_inputs([300, 7], 8, 2, 128, 16, dt, seed=9, qk_scale=20.0)
    o, lse = gdn.gdn_attn_decode(*inp, scale=0.11)
    check_attn(*inp, o, lse, scale=float(np.float32(0.11)))


@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_equal_lowest_scores(dt):
    """Scores that are all the type's lowest finite product still weigh equally; a row of -inf
    scores among finite ones has no weight."""
    q, kc, vc, table, lens = attn_inputs([40], 2, 1, 64, 16, dt, seed=3)
    ids = table[0, :3].long()
    q.fill_(1.0)
    kc[ids] = -1e30
    o, lse = gdn.gdn_attn_decode(q, kc, vc, table, lens)
    v = n64(vc[ids].flatten(0, 1)[:40, 0])
    within("o", o[0], np.repeat(v.mean(0)[None], 2, 0),
           half(dt) * np.abs(v.mean(0)) + (60 * U + 2.0 ** -21 + (half(BF) if dt == BF else 0))
           * np.abs(v).mean(0) * (1 + half(dt)))
    kc[ids[1]] = -float("inf")
    o, _ = gdn.gdn_attn_decode(q, kc, vc, table, lens)
    v = np.concatenate([v[:16], v[32:]])
    within("o", o[0], np.repeat(v.mean(0)[None], 2, 0),
           half(dt) * np.abs(v.mean(0)) + (60 * U + 2.0 ** -21 + (half(BF) if dt == BF else 0))
           * np.abs(v).mean(0) * (1 + half(dt)))


def test_attention_shared_pages_and_strided_queries():
    """Two requests on the same pages (a shared prefix), q a slice of a fused projection."""
    q, kc, vc, table, lens = attn_inputs([90, 61, 20], 8, 2, 128, 16, BF, seed=4)
    table[1, :4] = table[0, :4]
    qkv = torch.randn(3, 12, 128, device="cuda").to(BF)
    q = qkv[:, :8]
    o, lse = gdn.gdn_attn_decode(q, kc, vc, table, lens)
    check_attn(q, kc, vc, table, lens, o, lse)
    same = gdn.gdn_attn_decode(q.contiguous(), kc, vc, table, lens)
    assert torch.equal(o, same[0])


@pytest.mark.parametrize("dt,D", [(BF, 128), (F32, 64)])
def test_attention_bad_pages_and_lengths_are_left_out(dt, D):
    q, kc, vc, table, lens = attn_inputs([90, 130, 33, 20], 8, 2, D, 16, dt, seed=5)
    kc.nan_to_num_(0.25)
    vc.nan_to_num_(0.25)
    table[0, 2], table[1, 0], table[2, :] = -1, kc.shape[0], -5
    lens[3] = -4
    word = gdn.status_word()
    o, lse = gdn.gdn_attn_decode(q, kc, vc, table, lens, status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_ERR_INVALID_ARG
    assert gdn.gdn_check_device_status(word) == gdn.GDN_OK
    check_attn(q, kc, vc, table, lens.clamp(min=0), o, lse)
    lens[3] = 10 ** 6  # clamped to the table's width, whose entries past its pages are bad
    o, lse = gdn.gdn_attn_decode(q, kc, vc, table, lens, status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_ERR_INVALID_ARG
    check_attn(q, kc, vc, table, lens.clamp(max=table.shape[1] * 16), o, lse)


@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_offsets_past_32_bits(dt):
    """Pages behind 2^32 elements of the cache."""
    P, Hk, D = 64, 8, 256
    pages = (1 << 32) // (P * Hk * D) + 4
    kc, vc = (torch.empty(pages, P, Hk, D, dtype=dt, device="cuda") for _ in range(2))
    ids = torch.tensor([pages - 1, 0, pages - 2], device="cuda")
    gen = torch.Generator().manual_seed(6)
    small = [rand(gen, (3, P, Hk, D), dt) for _ in range(2)]
    kc[ids], vc[ids] = small
    q, lens = rand(gen, (1, 16, D), dt), i32([150])
    o, lse = gdn.gdn_attn_decode(q, kc, vc, ids.int()[None], lens)
    check_attn(q, *small, i32([[0, 1, 2]]), lens, o, lse)
    del kc, vc
    torch.cuda.empty_cache()


def test_attention_graph_replay_and_streams():
    """A captured call replayed with other lengths, beside calls on another stream."""
    q, kc, vc, table, lens = attn_inputs([900, 1500, 3], 8, 2, 128, 16, BF, seed=7)
    other = attn_inputs([2222], 16, 2, 256, 16, BF, seed=8)
    ref_other = gdn.gdn_attn_decode(*other)
    gdn.gdn_attn_decode(q, kc, vc, table, lens)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        o, lse = gdn.gdn_attn_decode(q, kc, vc, table, lens)
    for new in ([900, 1500, 3], [1, 1499, 0], [900, 17, 2]):
        lens.copy_(i32(new))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = [gdn.gdn_attn_decode(*other) for _ in range(3)]
        g.replay()
        torch.cuda.synchronize()
        check_attn(q, kc, vc, table, lens, o, lse)
        for x in got:
            assert torch.equal(x[0], ref_other[0]) and torch.equal(x[1], ref_other[1])


@pytest.mark.parametrize("dt", [BF, F32])
def test_attention_scores_that_rise_and_fall_slowly(dt):
    """The running maximum creeps up by less than a factor 2^8 of weight from tile to tile, then
    falls."""
    q, kc, vc, table, lens = attn_inputs([2000], 2, 1, 64, 16, dt, seed=14)
    ramp = 6 * torch.sin(torch.linspace(0, 3, 2000, device="cuda"))
    ids = table[0, :125].long()
    q.fill_(1.0)
    kc[ids] = (ramp.view(125, 16, 1, 1) + 0.1 * torch.randn(125, 16, 1, 64, device="cuda")).to(dt)
    o, lse = gdn.gdn_attn_decode(q, kc, vc, table, lens)
    check_attn(q, kc, vc, table, lens, o, lse)


def test_attention_without_lse_and_into_given_outputs():
    inp = attn_inputs([300, 0, 5], 8, 2, 128, 16, BF, seed=15)
    o, lse = gdn.gdn_attn_decode(*inp)
    mine, ws = torch.empty_like(o), torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    got = gdn.gdn_attn_decode(*inp, o=mine, want_lse=False, ws=ws)
    assert got[0] is mine and got[1] is None and torch.equal(mine, o)
    with pytest.raises(gdn.GDNError):
        gdn.gdn_attn_decode(*inp, ws=ws[:512])


def test_binding_refuses_wrong_types_and_shapes():
    q, kc, vc, table, lens = attn_inputs([30, 5], 8, 2, 128, 16, BF, seed=16)
    for bad in ((q.float(), kc, vc, table, lens), (q, kc, vc[:-1], table, lens),
                (q, kc, vc, table.long(), lens), (q, kc, vc, table, lens[:1]),
                (q, kc, vc, table.t(), lens), (q.transpose(0, 1), kc, vc, table, lens),
                (q, kc.transpose(1, 2), vc, table, lens)):
        with pytest.raises(ValueError):
            gdn.gdn_attn_decode(*bad)
    d, state = step_inputs(2, 1, 2, 128, 128, BF, 4)
    for kw in (dict(slots=torch.zeros(2, dtype=torch.int64, device="cuda")),
               dict(slots=i32([0])), dict(state=state.bfloat16()), dict(state=state[:, :1])):
        with pytest.raises(ValueError):
            gdn.gdn_step(**(d | dict(state=state) | kw))
    with pytest.raises(gdn.GDNError):
        gdn.gdn_step(**d, state=state[:1])  # no slots, fewer states than rows


def test_calls_captured_behind_copies_memsets_and_other_streams():
    """Each call as the first kernel behind a memset, a device copy and a join of two streams, in
    a captured graph: they are launched behind what comes before them, whatever that is."""
    q, kc, vc, table, lens = attn_inputs([500, 70], 8, 2, 128, 16, BF, seed=17)
    d, state = step_inputs(2, 2, 4, 128, 128, BF, 2, seed=18)
    rq, rk, _, wq, wk, f, _ = rope_inputs(300, 4, 2, 128, 64, BF, seed=19)
    dyq, dyk = torch.randn(300, 4, 128, device="cuda").to(BF), torch.ones(300, 2, 128, device="cuda").to(BF)
    want_o = gdn.gdn_attn_decode(q, kc, vc, table, lens)[0]
    keep = state.clone()
    want_s = gdn.gdn_step(**d, state=keep)
    want_g = gdn.gdn_qk_norm_rope_bwd(rq, rk, wq, wk, f, None, dyq, dyk)
    lens2, state2, dyq2 = torch.empty_like(lens), torch.empty_like(state), torch.empty_like(dyq)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        lens2.zero_()
        empty = gdn.gdn_attn_decode(q, kc, vc, table, lens2)[0]
        lens2.copy_(lens)
        got_o = gdn.gdn_attn_decode(q, kc, vc, table, lens2)[0]
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            state2.copy_(state)
            dyq2.copy_(dyq)
        busy = torch.ones(1000, device="cuda") + 1
        main.wait_stream(side)
        got_s = gdn.gdn_step(**d, state=state2)
        got_g = gdn.gdn_qk_norm_rope_bwd(rq, rk, wq, wk, f, None, dyq2, dyk)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert (empty == 0).all() and torch.equal(got_o, want_o) and torch.equal(got_s, want_s)
        assert torch.equal(state2, keep) and all(torch.equal(a, b) for a, b in zip(got_g, want_g))
        assert (busy == 2).all()


def test_calls_on_a_given_stream():
    """`stream` runs the call there, allocations included; many calls in a row keep their outputs."""
    inp = attn_inputs([700, 90], 8, 2, 128, 16, BF, seed=23)
    want = gdn.gdn_attn_decode(*inp)
    rq, rk, _, wq, wk, f, _ = rope_inputs(200, 4, 2, 128, 64, BF, seed=24)
    dy = torch.randn(200, 4, 128, device="cuda").to(BF), torch.ones(200, 2, 128, device="cuda").to(BF)
    grads = gdn.gdn_qk_norm_rope_bwd(rq, rk, wq, wk, f, None, *dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [(gdn.gdn_attn_decode(*inp, stream=side),
            gdn.gdn_qk_norm_rope_bwd(rq, rk, wq, wk, f, None, *dy, stream=side))
           for _ in range(20)]
    filler = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(20)]
    torch.cuda.synchronize()
    for a, g in got:
        assert all(torch.equal(x, y) for x, y in zip(a + g, want + grads))
    assert all((x == 7).all() for x in filler)


def test_attention_empty_batch():
    q, kc, vc, table, lens = attn_inputs([5], 8, 2, 128, 16, BF)
    o, lse = gdn.gdn_attn_decode(q[:0], kc, vc, table[:0], lens[:0])
    assert o.shape == (0, 8, 128) and lse.shape == (0, 8)


# ------------------------------------------------------------------ norm + rotation

def rope_inputs(N, Hq, Hk, D, R, dt, far=0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    qkv = rand(gen, (N, Hq + 2 * Hk, D), dt)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    wq, wk = 1 + 0.1 * rand(gen, (D,)), 1 + 0.1 * rand(gen, (D,))
    f = torch.tensor([1e6 ** (-2 * i / max(R, 1)) for i in range(R // 2)], device="cuda")
    pos = torch.randint(0, far, (N,), generator=gen).int().cuda() if far else None
    return q, k, v, wq, wk, f, pos


def positions(pos, N, T=0):
    return pos.cpu().numpy() if pos is not None else np.arange(N) % (T or max(N, 1))


def terms(a, inter, R):
    """|a1| + |a2| of every pair (|a| where nothing is rotated)."""
    y = np.abs(a)
    i, j = decode._pairs(R, inter)
    y[..., i], y[..., j] = (y[..., i] + y[..., j],) * 2
    return y


def angle_err(t, f):
    """Error of cos and sin: the fraction's rounding, the dropped part of the product, and two
    units in the last place of the function."""
    err = np.zeros(len(t)) if len(f) == 0 else \
        2 * np.pi * (2.0 ** -23 + np.abs(t) * f.max() * 2.0 ** -50) + 2.0 ** -22
    return err[:, None, None]


def check_rows(name, y, x, w, t, f, inter, dt, scale=1.0):
    """n = x r w: 13 additions in the mean (halved by the root), 8 more roundings: 16 U of |n|;
    the rotation two products and a sum of such, with the angle's error."""
    x, w, f = n64(x), n64(w), n64(f)
    ref = decode.norm_rope_fwd(x, w, t, f, inter, rope_scale=scale)
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-6) * w
    A = terms(n, inter, 2 * len(f)) * max(scale, 1.0)
    within(name, y, ref, half(dt) * np.abs(ref) + A * (20 * U + angle_err(t, f)) * (1 + half(dt)))


ROPE = [  # N, Hq, Hk, D, R, dtype, far
    (1, 1, 1, 64, 64, BF, 0), (1, 16, 2, 256, 64, BF, 100), (7, 4, 2, 128, 128, BF, 0),
    (33, 6, 3, 80, 32, BF, 5000), (300, 8, 1, 256, 256, BF, 2 ** 20), (5, 3, 1, 8, 0, BF, 0),
    (129, 5, 5, 128, 16, BF, 2 ** 31 - 1), (1000, 16, 4, 64, 32, BF, 0),
    (1, 2, 1, 16, 16, F32, 0), (50, 4, 2, 128, 64, F32, 2 ** 20), (17, 1, 1, 256, 256, F32, 7),
    (200, 3, 3, 72, 48, F32, 2 ** 31 - 1), (65, 8, 2, 248, 240, F32, 0),
    # several tokens and kinds per warp
    (4001, 17, 3, 128, 64, BF, 0), (3001, 13, 5, 64, 64, BF, 9000), (2500, 12, 1, 256, 64, BF, 0),
    (3003, 16, 9, 64, 32, F32, 70000),
]
ROPE_IDS = [f"N{c[0]}_h{c[1]}x{c[2]}_d{c[3]}_r{c[4]}_{'bf16' if c[5] == BF else 'f32'}_p{c[6]}"
            for c in ROPE]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("case", ROPE, ids=ROPE_IDS)
def test_rope_forward_matches_definition(case, inter):
    N, Hq, Hk, D, R, dt, far = case
    q, k, _, wq, wk, f, pos = rope_inputs(*case, seed=N)
    scale = 1.25 if N % 2 else 1.0
    yq, yk = gdn.gdn_qk_norm_rope_fwd(q, k, wq, wk, f, pos, interleaved=inter, rope_scale=scale)
    t = positions(pos, N)
    check_rows("q", yq, q, wq, t, f, inter, dt, scale)
    check_rows("k", yk, k, wk, t, f, inter, dt, scale)


def check_grads(name, dx, dw, x, w, t, f, inter, dy, dt, scale=1.0):
    """dn: two products and a sum with the angle's error; g, the mean (13 additions) and
    the last difference: 40 U of |g| + |x r| mean|g x r| at most, times r.  dw: a lane adds its
    rows in order, 8 warps and the CTAs' partials after that (fp64): n + 16 roundings at
    most over the n rows."""
    x, w, f, dy = n64(x), n64(w), n64(f), n64(dy)
    rdx, rdw = decode.norm_rope_bwd(x, w, t, f, dy, inter, rope_scale=scale)
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-6)
    A = terms(dy, inter, 2 * len(f)) * max(scale, 1.0)
    e = 40 * U + angle_err(t, f)
    xr, g = np.abs(x * r), A * np.abs(w)
    tol = e * r * (g + xr * np.mean(g * xr, -1, keepdims=True))
    within(f"d{name}", dx, rdx, half(dt) * np.abs(rdx) + tol * (1 + half(dt)))
    rows = x.shape[0] * x.shape[1]
    tol = ((e + (rows + 16) * U) * A * xr).sum((0, 1))
    within(f"dw{name}", dw, rdw, tol + U * np.abs(rdw))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("case", ROPE, ids=ROPE_IDS)
def test_rope_backward_matches_definition(case, inter):
    N, Hq, Hk, D, R, dt, far = case
    q, k, _, wq, wk, f, pos = rope_inputs(*case, seed=N + 1)
    gen = torch.Generator().manual_seed(N)
    dyq, dyk = rand(gen, (N, Hq, D), dt), rand(gen, (N, Hk, D), dt)
    scale = 1.25 if N % 2 else 1.0
    kw = dict(interleaved=inter, rope_scale=scale)
    dq, dk, dwq, dwk = gdn.gdn_qk_norm_rope_bwd(q, k, wq, wk, f, pos, dyq, dyk, **kw)
    t = positions(pos, N)
    check_grads("q", dq, dwq, q, wq, t, f, inter, dyq, dt, scale)
    check_grads("k", dk, dwk, k, wk, t, f, inter, dyk, dt, scale)
    again = gdn.gdn_qk_norm_rope_bwd(q, k, wq, wk, f, pos, dyq, dyk, **kw)
    for a, b in zip((dq, dk, dwq, dwk), again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient_matches_differences_of_the_kernel(inter):
    """<dx, d> and <dw, d> against central differences of the fp32 forward along random d:
    outputs of size 1 carry 20 U each, the loss sums 4 * 6 * 32 of them with random signs
    (taken as all the same sign), over a step of 2 h; the third derivative's term is h^2."""
    N, Hq, Hk, D, R = 4, 4, 2, 32, 16
    q, k, _, wq, wk, f, pos = rope_inputs(N, Hq, Hk, D, R, F32, 1000, seed=5)
    gen = torch.Generator().manual_seed(6)
    dyq, dyk, eq, ek = (rand(gen, s) for s in ((N, Hq, D), (N, Hk, D)) * 2)
    ew, ev = rand(gen, (D,)), rand(gen, (D,))
    dq, dk, dwq, dwk = gdn.gdn_qk_norm_rope_bwd(q, k, wq, wk, f, pos, dyq, dyk, interleaved=inter)

    def loss(h):
        yq, yk = gdn.gdn_qk_norm_rope_fwd(q + h * eq, k + h * ek, wq + h * ew, wk + h * ev, f,
                                          pos, interleaved=inter)
        return float((yq.double() * dyq.double()).sum() + (yk.double() * dyk.double()).sum())

    h = 2.0 ** -9
    diff = (loss(h) - loss(-h)) / (2 * h)
    want = sum(float((a.double() * b.double()).sum())
               for a, b in ((dq, eq), (dk, ek), (dwq, ew), (dwk, ev)))
    size = float(dyq.abs().sum() + dyk.abs().sum())
    assert abs(diff - want) <= size * 4 * (20 * U / h + 30 * h * h)


def test_rope_positions_of_batch_rows_and_contiguous_inputs():
    """positions = None: t = n % T of q [B, T, H, D]; the bits of given positions."""
    gen = torch.Generator().manual_seed(7)
    q, k = rand(gen, (3, 21, 4, 64), BF), rand(gen, (3, 21, 2, 64), BF)
    w, f = torch.ones(64, device="cuda"), torch.tensor([0.7 ** i for i in range(16)], device="cuda")
    a = gdn.gdn_qk_norm_rope_fwd(q, k, w, w, f)
    pos = torch.arange(21, dtype=torch.int32, device="cuda").repeat(3, 1)
    b = gdn.gdn_qk_norm_rope_fwd(q, k, w, w, f, pos)
    c = gdn.gdn_qk_norm_rope_fwd(q.view(63, 4, 64), k.view(63, 2, 64), w, w, f, pos)
    d = gdn.gdn_qk_norm_rope_fwd(q, k, w, w, f, pos - 5)  # negative positions turn back
    for i in range(2):
        assert torch.equal(a[i], b[i]) and torch.equal(a[i].flatten(0, 1), c[i])
        check_rows("d", d[i].flatten(0, 1), (q, k)[i].flatten(0, 1), w,
                   (pos - 5).reshape(-1).cpu().numpy(), f, False, BF)


def test_rope_of_one_token_without_leading_sizes():
    gen = torch.Generator().manual_seed(8)
    q, k, w = rand(gen, (4, 64), BF), rand(gen, (2, 64), BF), torch.ones(64, device="cuda")
    f, pos = torch.ones(8, device="cuda"), torch.full((1,), 9, dtype=torch.int32, device="cuda")
    for p in (None, pos):
        a = gdn.gdn_qk_norm_rope_fwd(q, k, w, w, f, p)
        b = gdn.gdn_qk_norm_rope_fwd(q[None], k[None], w, w, f, p)
        for x, y in zip(a, b):
            assert torch.equal(x, y[0])


def test_attention_refuses_one_query_row_expanded():
    q, kc, vc, table, lens = attn_inputs([30, 5], 8, 2, 128, 16, BF, seed=16)
    with pytest.raises(ValueError):
        gdn.gdn_attn_decode(q[:1].expand(2, 8, 128), kc, vc, table, lens)


def test_rope_zero_rows_and_one_kind_of_heads():
    """A zero row normalises to zero (and its gradient stays finite); Hk = 0, Hq = 0 and N = 0."""
    w, f = torch.ones(64, device="cuda"), torch.ones(8, device="cuda")
    q, none = torch.zeros(3, 2, 64, device="cuda"), torch.zeros(3, 0, 64, device="cuda")
    y, e = gdn.gdn_qk_norm_rope_fwd(q, none, w, w, f)
    assert (y == 0).all() and e.shape == (3, 0, 64)
    x = torch.randn(700, 5, 64, device="cuda")
    a = gdn.gdn_qk_norm_rope_fwd(x, x[:, :0], w, w, f)[0]
    b = gdn.gdn_qk_norm_rope_fwd(x[:, :0], x, w, w, f)[1]
    assert torch.equal(a, b)
    ga = gdn.gdn_qk_norm_rope_bwd(x, x[:, :0], w, w, f, None, x, x[:, :0].contiguous())
    gb = gdn.gdn_qk_norm_rope_bwd(x[:, :0], x, w, w, f, None, x[:, :0].contiguous(), x)
    assert torch.equal(ga[0], gb[1]) and torch.equal(ga[2], gb[3])
    dq, _, dw, _ = gdn.gdn_qk_norm_rope_bwd(q, none, w, w, f, None, torch.ones_like(q), none)
    check_grads("q", dq, dw, q, w, np.arange(3), f, False, torch.ones_like(q), F32)
    z = q[:0]
    assert gdn.gdn_qk_norm_rope_fwd(z, z, w, w, f)[0].shape == (0, 2, 64)
    out = gdn.gdn_qk_norm_rope_bwd(z, z, w, w, f, None, z, z)
    assert (out[2] == 0).all() and (out[3] == 0).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_cache_writes_its_slots_only(dt, inter):
    N, Hq, Hk, D, R = 37, 4, 2, 128, 64
    q, k, v, wq, wk, f, pos = rope_inputs(N, Hq, Hk, D, R, dt, 9000, seed=8)
    yq, yk = gdn.gdn_qk_norm_rope_fwd(q, k, wq, wk, f, pos, interleaved=inter)
    slots = torch.randperm(64, generator=torch.Generator().manual_seed(1))[:N].int().cuda()
    slots[3], slots[N - 1], slots[5], slots[6] = -1, -1, 64, -7  # padding, then bad ones
    kc = torch.full((4, 16, Hk, D), 3.0, dtype=dt, device="cuda")
    vc = torch.full((4, 16, Hk, D), 5.0, dtype=dt, device="cuda")
    rk, rv = kc.view(-1, Hk, D).clone(), vc.view(-1, Hk, D).clone()
    keep = (slots >= 0) & (slots < 64)
    rk[slots[keep].long()], rv[slots[keep].long()] = yk[keep], v[keep]
    word = gdn.status_word()
    out = gdn.gdn_qk_norm_rope_cache(q, k, v, wq, wk, f, pos, slots, kc, vc, interleaved=inter,
                                     status=word)
    assert torch.equal(out, yq)
    assert torch.equal(kc.view(-1, Hk, D), rk) and torch.equal(vc.view(-1, Hk, D), rv)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_ERR_INVALID_ARG
    slots[5], slots[6] = -1, -1
    gdn.gdn_qk_norm_rope_cache(q, k, v, wq, wk, f, pos, slots, kc, vc, status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_OK


# ------------------------------------------------------------------------------- gdn_step

def step_inputs(B, Hqk, H, dk, dv, dt, pool, seed=0, slow=True):
    gen = torch.Generator().manual_seed(seed)
    d = dict(q=rand(gen, (B, 1, Hqk, dk), dt), k=rand(gen, (B, 1, Hqk, dk), dt),
             v=rand(gen, (B, 1, H, dv), dt), a=rand(gen, (B, 1, H), dt),
             b=rand(gen, (B, 1, H), dt),
             A_log=(1 + 15 * torch.rand(H, generator=gen)).log().cuda(),
             dt_bias=(-6.0 if slow else 0.0) + 0.1 * rand(gen, (H,)))
    state = rand(gen, (pool, H, dk, dv))
    return d, state


def check_step(d, S0, S1, o, rows, l2norm=True):
    """Against the oracle's recurrence for one token.  S' = alpha S + beta k (v - alpha S^T k):
    dk additions for S^T k, about 16 roundings more, alpha off by (16 + 4 |g|) U of itself;
    o: dk additions more, relative to the sum of |q| |terms of S'|."""
    n = {k: n64(x) for k, x in d.items()}
    ro, rS = oracle.fwd(n["q"], n["k"], n["v"], n["a"], n["b"], n["A_log"], n["dt_bias"],
                        h0=n64(S0), l2norm=l2norm)
    q, k, dt = n["q"][:, 0], n["k"][:, 0], d["q"].dtype
    dk, r = q.shape[-1], S0.shape[1] // q.shape[1]
    if l2norm:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + 1e-6)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + 1e-6)
    q, k = np.abs(np.repeat(q, r, 1)) * dk ** -0.5, np.abs(np.repeat(k, r, 1))
    g = np.exp(n["A_log"]) * np.logaddexp(0, n["a"][:, 0] + n["dt_bias"])
    al, be = np.exp(-g)[..., None, None], (1 / (1 + np.exp(-n["b"][:, 0])))[..., None, None]
    S = np.abs(n64(S0))
    mag = al * S + be * k[..., None] * (np.abs(n["v"][:, 0])[..., None, :]
                                        + al * (k[..., None] * S).sum(-2, keepdims=True))
    e = (2 * dk + 40 + 4 * g[..., None, None]) * U
    within("state", S1[rows], rS[rows], e[rows] * mag[rows])
    within("o", o[rows], ro[rows],
           half(dt) * np.abs(ro[rows])
           + (e * (q[..., None] * mag).sum(-2, keepdims=True))[rows, :, 0][:, None] * (1 + half(dt)))


STEP = [  # B, Hqk, H, dk, dv, dtype
    (1, 16, 32, 128, 128, BF), (1, 1, 1, 128, 128, BF), (7, 2, 6, 128, 128, BF),
    (65, 4, 4, 128, 128, BF), (1, 4, 8, 16, 16, F32), (5, 2, 4, 128, 128, F32),
    (3, 1, 3, 80, 48, F32), (4, 2, 2, 16, 128, F32), (4, 2, 2, 112, 16, F32),
    (2, 1, 2, 64, 96, F32),
]


@pytest.mark.parametrize("l2norm", [True, False])
@pytest.mark.parametrize("case", STEP, ids=["x".join(map(str, c[:5])) + (
    "_bf16" if c[5] == BF else "_f32") for c in STEP])
def test_step_matches_recurrence(case, l2norm):
    B, Hqk, H, dk, dv, dt = case
    pool = B + 3
    d, state = step_inputs(*case, pool, seed=B + dk)
    if not l2norm:  # keys of unit size keep the recurrence stable
        d["q"], d["k"] = d["q"] / dk ** 0.5, d["k"] / dk ** 0.5
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(B))[:B].int().cuda()
    before = state.clone()
    word = gdn.status_word()
    o = gdn.gdn_step(**d, state=state, slots=slots, l2norm=l2norm, status=word)
    at = slots.long()
    check_step(d, before[at], state[at], o, np.arange(B), l2norm)
    rest = torch.ones(pool, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(state[rest], before[rest])
    assert gdn.gdn_check_device_status(word) == gdn.GDN_OK
    # no slots: row b, the same bits
    alone = before[at].clone()
    assert torch.equal(gdn.gdn_step(**d, state=alone, l2norm=l2norm), o)
    assert torch.equal(alone, state[at])


def test_step_fast_decay_and_zero_rows():
    d, state = step_inputs(3, 2, 4, 128, 128, BF, 3, seed=11, slow=False)
    d["q"][1], d["k"][1] = 0, 0
    before = state.clone()
    o = gdn.gdn_step(**d, state=state)
    check_step(d, before, state, o, np.arange(3))


def test_step_padded_bad_and_repeated_slots():
    """-1 is a padded row; a slot out of range or given again is left out and recorded; the first
    row keeps a repeated slot."""
    d, state = step_inputs(6, 2, 4, 128, 128, BF, 8, seed=12)
    before, word = state.clone(), gdn.status_word()
    o = gdn.gdn_step(**d, state=state, slots=i32([5, -1, 2, -1, 0, 7]), status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_OK
    assert (o[[1, 3]] == 0).all()
    at = torch.tensor([5, 0, 2, 0, 0, 7])
    check_step(d, before[at], state[at], o, np.array([0, 2, 4, 5]))
    assert torch.equal(state[[1, 3, 4, 6]], before[[1, 3, 4, 6]])
    good = (o.clone(), state.clone())
    state.copy_(before)
    o = gdn.gdn_step(**d, state=state, slots=i32([5, 8, 2, 5, 0, 7]), status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_ERR_INVALID_ARG
    assert torch.equal(o, good[0]) and torch.equal(state, good[1])
    state.copy_(before)
    o = gdn.gdn_step(**d, state=state, slots=i32([5, -9, 2, 2, 0, 7]), status=word)
    assert gdn.gdn_check_device_status(word) == gdn.GDN_ERR_INVALID_ARG
    assert torch.equal(o, good[0]) and torch.equal(state, good[1])
    assert gdn.gdn_step(**{k: (x[:0] if x.dim() > 1 else x) for k, x in d.items()},
                        state=state, slots=i32([])).shape == (0, 1, 4, 128)


def test_step_offsets_past_32_bits():
    """States behind 2^31 elements of the pool."""
    d, small = step_inputs(3, 2, 32, 128, 128, BF, 3, seed=22)
    pool = torch.empty((1 << 32) // (32 * 128 * 128) + 3, 32, 128, 128, device="cuda")
    at = torch.tensor([pool.shape[0] - 1, 0, pool.shape[0] - 2], device="cuda")
    pool[at] = small
    o = gdn.gdn_step(**d, state=pool, slots=at.int())
    assert torch.equal(o, gdn.gdn_step(**d, state=small)) and torch.equal(pool[at], small)
    del pool
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt,tol", [(BF, 1e-2), (F32, 1e-5)])
def test_steps_continue_a_prefill(dt, tol):
    """gdn_fwd over T tokens, then one gdn_step per token, against gdn_fwd over all of them (the
    bars of the core's own parity)."""
    B, T, n, Hqk, H = 2, 70, 5, 2, 4
    gen = torch.Generator().manual_seed(13)
    q, k = rand(gen, (B, T + n, Hqk, 128), dt), rand(gen, (B, T + n, Hqk, 128), dt)
    v, a, b = rand(gen, (B, T + n, H, 128), dt), rand(gen, (B, T + n, H), dt), \
        rand(gen, (B, T + n, H), dt)
    A_log, bias = torch.zeros(H, device="cuda"), torch.full((H,), -4.0, device="cuda")
    o_all, h_all = gdn.gdn_fwd(q, k, v, a, b, A_log, bias)
    head = [x[:, :T].contiguous() for x in (q, k, v, a, b)]
    _, state = gdn.gdn_fwd(*head, A_log, bias)
    for t in range(T, T + n):
        o = gdn.gdn_step(*[x[:, t:t + 1].contiguous() for x in (q, k, v, a, b)], A_log, bias,
                         state)
        err = (o.double() - o_all[:, t:t + 1].double()).norm() / o_all[:, t:t + 1].double().norm()
        assert err <= tol
    assert (state.double() - h_all.double()).norm() / h_all.double().norm() <= tol


# ------------------------------------------------------------------------------- slot map

def slot_inputs(ctx, new, P, blocks, free_extra=3, seed=0):
    rng = np.random.default_rng(seed)
    held = [-(-max(c, 0) // P) for c in ctx]
    want = sum(-(-(max(c, 0) + max(n, 0)) // P) - h for c, n, h in zip(ctx, new, held))
    pages = sum(held) + want + free_extra + 1
    perm = rng.permutation(pages)
    table = np.full((len(ctx), blocks), -1)
    at = 0
    for b, c in enumerate(held):
        m = min(c, blocks)
        table[b, :m] = perm[at:at + m]
        at += c
    return i32(ctx), i32(new), i32(perm[at:]), i32(table), pages


def check_slots(ctx, new, free, table, P, pages, n_tokens, ok=True):
    ref = decode.slot_map(ctx.tolist(), new.tolist(), free.tolist(), table.cpu().numpy(), P, pages,
                          n_tokens)
    word = gdn.status_word()
    seq, cu, pos, slots, used = gdn.gdn_slot_map(ctx, new, free, table, page_size=P, pages=pages,
                                                 n_tokens=n_tokens, status=word)
    for name, x, r in (("seq_len", seq, ref[0]), ("cu", cu, ref[1]), ("positions", pos, ref[2]),
                       ("slots", slots, ref[3]), ("table", table, ref[4]),
                       ("used", used, np.array([ref[5]]))):
        np.testing.assert_array_equal(x.cpu().numpy(), r, err_msg=name)
    assert gdn.gdn_check_device_status(word) == (gdn.GDN_OK if ok else gdn.GDN_ERR_INVALID_ARG)


SLOTS = [  # ctx, new, page size, blocks, token rows
    ([0], [1], 16, 1, 1), ([0], [0], 16, 1, 5), ([], [], 16, 2, 3), ([15, 16, 17], [1, 1, 1], 16, 3, 8),
    ([0, 5, 0, 31], [33, 0, 64, 1], 16, 5, 98), ([3, 0, 8], [2, 0, 5], 4, 4, 9),
    ([7] * 300, [1] * 300, 8, 2, 300), (list(range(700)), [i % 3 for i in range(700)], 16, 50, 701),
    ([100, 0, 4000], [2000, 1500, 900], 24, 300, 5000), ([5, 0], [7, 3], 1, 14, 12),
    ([1000000], [4097], 256, 4000, 4097), ([0] * 9, [0] * 9, 16, 2, 0),
]


@pytest.mark.parametrize("case", SLOTS, ids=[f"B{len(c[0])}_n{sum(c[1])}_p{c[2]}" for c in SLOTS])
def test_slot_map_matches_definition(case):
    ctx, new, P, blocks, n = case
    c, w, free, table, pages = slot_inputs(ctx, new, P, blocks, seed=P)
    check_slots(c, w, free, table, P, pages, n)


def test_slot_map_faults_are_recorded_and_left_out():
    """Too few free pages, a table too narrow, bad pages, negative lengths, too few token rows."""
    c, w, free, table, pages = slot_inputs([10, 3, 40], [30, 20, 10], 8, 10, seed=1)
    check_slots(c, w, free[:4].clone(), table.clone(), 8, pages, 64, ok=False)
    check_slots(c, w, free, table[:, :6].contiguous(), 8, pages, 64, ok=False)
    bad = free.clone()
    bad[2] = pages
    check_slots(c, w, bad, table.clone(), 8, pages, 64, ok=False)
    broken = table.clone()
    broken[0, 1] = -1  # the page that request 0's next token falls on
    check_slots(c, w, free, broken, 8, pages, 64, ok=False)
    check_slots(c, w, free, table.clone(), 8, pages, 41, ok=False)
    c[1], w[2] = -5, -1
    check_slots(c, w, free, table.clone(), 8, pages, 64, ok=False)


# --------------------------------------------------------------------- a run of them together

@pytest.mark.parametrize("captured", [False, True])
def test_decode_steps_of_a_hybrid_model(captured):
    """Three requests served token by token through one attention layer and one GDN layer: slot
    map -> norm, rotation and cache rows -> attention over the cache, and gdn_step over the
    state pool; a prompt first, then one token each, with a padded row in the batch.  The
    attention of the last step is compared with the definition on all keys from the start."""
    Hq, Hk, D, P, pages, n = 4, 2, 128, 16, 40, 128
    gen = torch.Generator().manual_seed(21)
    kc, vc = (torch.full((pages, P, Hk, D), float("nan"), dtype=BF, device="cuda")
              for _ in range(2))
    table, free = i32(np.full((4, 8), -1)), i32(np.random.default_rng(2).permutation(pages))
    ctx = i32([0, 0, 0, 0])
    wq, wk = 1 + 0.1 * rand(gen, (D,)), 1 + 0.1 * rand(gen, (D,))
    f = torch.tensor([1e4 ** (-i / 32) for i in range(32)], device="cuda")
    state = torch.zeros(6, 4, 128, 128, device="cuda")
    slots_of = i32([4, 0, 3, -1])
    A_log, bias = torch.zeros(4, device="cuda"), torch.full((4,), -4.0, device="cuda")
    word = gdn.status_word()
    keys, vals = [[] for _ in range(4)], [[] for _ in range(4)]
    graph, held = None, None
    for step, new in enumerate([[37, 1, 20, 0]] + [[1, 1, 1, 0]] * 20):
        rows = n if step == 0 else 4
        qkv = rand(gen, (rows, Hq + 2 * Hk, D), BF)
        if step == 0 or not captured:
            xs = qkv
        elif held is None:
            xs = held = qkv.clone()
        else:
            xs = held.copy_(qkv)
        nw = i32(new)

        def run():
            seq, cu, pos, slots, used = gdn.gdn_slot_map(ctx, nw, free, table, page_size=P,
                                                         pages=pages, n_tokens=rows, status=word)
            q = gdn.gdn_qk_norm_rope_cache(xs[:, :Hq], xs[:, Hq:Hq + Hk], xs[:, Hq + Hk:], wq, wk,
                                           f, pos, slots, kc, vc, status=word)
            if rows > 4:
                return seq, cu, used, q, None, None
            o, lse = gdn.gdn_attn_decode(q, kc, vc, table, seq, status=word)
            g = [x.contiguous()[:, None] for x in (xs[:, :2], xs[:, 2:4], xs[:, 4:],
                                                   xs[:, 0, :4], xs[:, 1, :4])]
            oo = gdn.gdn_step(*g, A_log, bias, state, slots_of, status=word)
            return seq, cu, used, q, (o, lse), oo

        if captured and step >= 1:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                nw_kept = nw
                with torch.cuda.graph(graph):
                    out = run()
            nw_kept.copy_(nw)
            graph.replay()
        else:
            out = run()
        seq, cu, used, q, att, oo = out
        at = cu.tolist()
        k = decode.norm_rope_fwd(n64(qkv[:, Hq:Hq + Hk]), n64(wk),
                                 np.concatenate([np.arange(int(ctx[b]), int(ctx[b]) + m)
                                                 for b, m in enumerate(new)]
                                                + [np.zeros(rows - sum(new))]), n64(f))
        for b in range(4):
            keys[b].append(k[at[b]:at[b + 1]])
            vals[b].append(n64(qkv[at[b]:at[b + 1], Hq + Hk:]))
        took = int(used)
        free.copy_(torch.cat((free[took:], free[:took])))
        ctx.copy_(seq)
    assert ctx.tolist() == [57, 21, 40, 0]
    assert gdn.gdn_check_device_status(word) == gdn.GDN_OK
    o, lse = att
    assert (o[3] == 0).all() and torch.isneginf(lse[3]).all() and (oo[3] == 0).all()
    qn = n64(q)
    for b in range(3):
        kk, vv = np.concatenate(keys[b]), np.concatenate(vals[b])
        for h in range(Hq):
            s = kk[:, h // 2] @ qn[at[b], h] * D ** -0.5
            w = np.exp(s - s.max())
            w /= w.sum()
            # keys rounded to bf16 in the cache: each score moves by at most half a step of
            # sum |q k| scale, the weights by twice that; then the call's own roundings
            e = half(BF) * (np.abs(kk[:, h // 2]) @ np.abs(qn[at[b], h])).max() * D ** -0.5
            ref = w @ vv[:, h // 2]
            tol = half(BF) * np.abs(ref) + (np.expm1(2 * e) + half(BF) + 2.0 ** -12) \
                * (w @ np.abs(vv[:, h // 2])) * (1 + half(BF))
            assert (np.abs(n64(o[b, h]) - ref) <= tol).all()
    assert (state[[1, 2, 5]] == 0).all() and (state[[4, 0, 3]].abs().sum((1, 2, 3)) > 0).all()
