"""Pins of the fp64 oracle of the full-attention calls and of the 8-bit cache: torch's own
attention and float8 type, closed forms, central finite differences."""
import numpy as np
import pytest
import torch

from oracle import attention, decode


def rand(shape, seed=0):
    return np.random.RandomState(seed).randn(*shape)


@pytest.mark.parametrize("causal", [True, False])
def test_forward_matches_torch_per_sequence(causal):
    q, k, v = rand((30, 4, 16)), rand((30, 2, 16), 1), rand((30, 2, 16), 2)
    cu = [0, 7, 7, 20, 29]
    o, lse = attention.attn_fwd(q, k, v, cu, cu, causal)
    for a, b in zip(cu[:-1], cu[1:]):
        if a == b:
            continue
        qs, ks, vs = (torch.from_numpy(x[a:b]).transpose(0, 1) for x in (q, k, v))
        ref = torch.nn.functional.scaled_dot_product_attention(
            qs, ks.repeat_interleave(2, 0), vs.repeat_interleave(2, 0), is_causal=causal)
        np.testing.assert_allclose(o[a:b], ref.transpose(0, 1).numpy(), atol=1e-12)
    assert (o[29:] == 0).all() and np.isneginf(lse[29:]).all()


def test_queries_are_the_last_of_a_longer_context():
    """The last nq rows of a causal run over all keys; rows that see nothing when nq > nk."""
    q, k, v = rand((12, 2, 8)), rand((12, 1, 8), 1), rand((12, 1, 8), 2)
    whole = attention.attn_fwd(q, k, v, [0, 12], [0, 12])
    part = attention.attn_fwd(q[7:], k, v, [0, 5], [0, 12])
    for a, b in zip(whole, part):
        np.testing.assert_allclose(a[7:], b, atol=1e-12)
    o, lse = attention.attn_fwd(q, k[:4], v[:4], [0, 12], [0, 4])
    assert (o[:8] == 0).all() and np.isneginf(lse[:8]).all() and np.isfinite(lse[8:]).all()
    np.testing.assert_allclose(o[8], np.repeat(v[:1, 0], 2, 0))  # the first that sees one key


def test_equal_keys_give_the_mean_of_what_is_seen():
    v = rand((6, 1, 4))
    o, lse = attention.attn_fwd(rand((6, 1, 4), 1), np.zeros((6, 1, 4)), v, [0, 6], [0, 6])
    for i in range(6):
        np.testing.assert_allclose(o[i], v[:i + 1].mean(0))
        np.testing.assert_allclose(lse[i], np.log(i + 1), atol=1e-15)


@pytest.mark.parametrize("causal,lens,klens", [(True, [3, 5], [3, 5]), (True, [4, 3], [2, 7]),
                                               (False, [4, 3], [2, 7])])
def test_backward_matches_finite_differences(causal, lens, klens):
    cu, ck = np.cumsum([0] + lens), np.cumsum([0] + klens)
    x = [rand((cu[-1], 2, 4)), rand((ck[-1], 1, 4), 1), rand((ck[-1], 1, 4), 2)]
    dO = rand((cu[-1], 2, 4), 3)

    def loss():
        return (attention.attn_fwd(*x, cu, ck, causal, 0.6)[0] * dO).sum()

    o, lse = attention.attn_fwd(*x, cu, ck, causal, 0.6)
    grads = attention.attn_bwd(*x, o, lse, dO, cu, ck, causal, 0.6)
    for t, g in zip(x, grads):
        flat = t.reshape(-1)
        for i in range(flat.size):
            keep = flat[i]
            flat[i] = keep + 1e-5
            up = loss()
            flat[i] = keep - 1e-5
            down = loss()
            flat[i] = keep
            assert abs((up - down) / 2e-5 - g.reshape(-1)[i]) < 1e-8


def test_offsets_that_are_not_ordered_are_cut():
    got = attention.sequences([-3, 5, 2, 9, 40], [0, 5, 2, 9, 40], 12, 12)
    assert [(r.start, r.stop) for r, _ in got] == [(0, 5), (5, 5), (5, 9), (9, 12)]


def test_e4m3_table_and_rounding_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(attention.E4M3, codes.view(torch.float8_e4m3fn).double().numpy())
    x = torch.cat((torch.randn(4000, dtype=torch.float64) * 100, torch.linspace(-0.02, 0.02, 999),
                   torch.tensor([448.0, 447.0, 440.0, 432.0, -448.0, 0.0, -0.0]).double()))
    x = x.clamp(-448, 448)
    mid = (attention.E4M3[:126] + attention.E4M3[1:127]) / 2  # ties
    x = torch.cat((x, torch.from_numpy(mid))).float()
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(attention.e4m3_codes(x.double().numpy()), want)
    assert (attention.e4m3_codes([np.nan, np.inf, -np.inf]) & 127 == 127).all()


def test_block_scales():
    for top, s in [(0.0, 2.0 ** -100), (448.0, 1.0), (448.1, 2.0), (224.0, 0.5), (1.75, 2.0 ** -8),
                   (1.76, 2.0 ** -7), (3e38, 2.0 ** 120)]:
        assert attention.block_scale(top) == s


def test_write_token_by_token_gives_the_values_of_one_write():
    """Powers of two: growing a block's scale later rounds again only below e4m3's normal numbers."""
    P, Hk, D, n = 32, 2, 8, 50
    x = rand((n, Hk, D)) * np.exp(0.2 * np.arange(n))[:, None, None]
    table = np.array([[2, 0]])
    zero = np.zeros((3, P, Hk, D), np.uint8), np.zeros((3, P // 16, Hk))
    at_once = attention.cache_write8(x, *zero, table, [0], [0, n])
    step = zero
    for t in range(n):
        step = attention.cache_write8(x[t:t + 1], *step, table, [t], [0, 1])
    np.testing.assert_array_equal(step[1], at_once[1])
    a, b = (attention.cache_read8(*c, table, [0, n], n) for c in (at_once, step))
    tiny = np.repeat(at_once[1][[2, 0]].reshape(-1, Hk), 16, 0)[:n, :, None] * 2.0 ** -6
    assert (np.abs(a - b) <= np.where(np.abs(a) >= tiny, 0.0, tiny * 2.0 ** -3)).all()
    assert (np.abs(a - x) <= np.maximum(np.abs(x) * 2.0 ** -4, tiny * 2.0 ** -4)).all()


def test_decode_over_the_values_is_the_forward_of_one_query():
    P, Hk, D, n = 16, 2, 8, 21
    x, y = rand((n, Hk, D)), rand((n, Hk, D), 1)
    table = np.array([[1, 2]])
    zero = np.zeros((3, P, Hk, D), np.uint8), np.zeros((3, 1, Hk))
    kc, vc = (attention.cache_write8(z, *zero, table, [0], [0, n]) for z in (x, y))
    q = rand((1, 4, D), 2)
    got = decode.attn_decode(q, attention.values(*kc), attention.values(*vc), table, [n])
    k, v = (attention.cache_read8(*c, table, [0, n], n) for c in (kc, vc))
    for a, b in zip(got, attention.attn_fwd(q, k, v, [0, 1], [0, n])):
        np.testing.assert_allclose(a, b, atol=1e-12)


@pytest.mark.parametrize("bad,good", [([0, 30, 20, 60], [0, 30, 30, 60]), ([-7, 10, 20, 90], [0, 10, 20, 60]),
                                      ([70, 10, 20, 30], [60, 60, 60, 60])])
def test_cache_offsets_that_are_not_ordered_are_cut(bad, good):
    P, Hk, D = 16, 1, 4
    x, table = rand((60, Hk, D)), np.arange(15).reshape(3, 5)
    zero = np.zeros((15, P, Hk, D), np.uint8), np.zeros((15, 1, Hk))
    a, b = (attention.cache_write8(x, *zero, table, [3, 0, 20], cu) for cu in (bad, good))
    for y, z in zip(a, b):
        np.testing.assert_array_equal(y, z)
    np.testing.assert_array_equal(attention.cache_read8(*a, table, bad, 60),
                                  attention.cache_read8(*b, table, good, 60))
