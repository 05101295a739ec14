"""Pins of the decode-step oracle (oracle/decode.py) to things other than itself: closed forms,
torch library routines in fp64, complex rotations and finite differences."""
import numpy as np
import pytest
import torch

from oracle import decode


def test_attention_matches_torch_on_gathered_rows():
    rng = np.random.default_rng(1)
    B, Hq, Hk, D, P, pages = 3, 6, 2, 8, 4, 20
    q = rng.standard_normal((B, Hq, D))
    kc, vc = rng.standard_normal((2, pages, P, Hk, D))
    table = rng.permutation(pages)[:15].reshape(3, 5)
    lens = [0, 1, 19]
    o, lse = decode.attn_decode(q, kc, vc, table, lens)
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all()
    np.testing.assert_allclose(o[1], np.repeat(vc[table[1, 0], 0], 3, axis=0))  # one token: v
    n = lens[2]
    k = torch.from_numpy(kc[table[2]].reshape(-1, Hk, D)[:n]).transpose(0, 1)
    v = torch.from_numpy(vc[table[2]].reshape(-1, Hk, D)[:n]).transpose(0, 1)
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q[2])[:, None], k.repeat_interleave(3, 0), v.repeat_interleave(3, 0))
    np.testing.assert_allclose(o[2], ref[:, 0].numpy(), rtol=1e-12)
    s = torch.einsum("hd,hnd->hn", torch.from_numpy(q[2]), k.repeat_interleave(3, 0)) / D ** 0.5
    np.testing.assert_allclose(lse[2], torch.logsumexp(s, 1).numpy(), rtol=1e-12)


def test_attention_equal_keys_average_the_values():
    kc = np.ones((4, 4, 1, 8))
    vc = np.random.default_rng(2).standard_normal((4, 4, 1, 8))
    o, lse = decode.attn_decode(np.ones((1, 1, 8)), kc, vc, np.array([[2, 0, 3, 1]]), [14])
    rows = np.concatenate([vc[2, :, 0], vc[0, :, 0], vc[3, :, 0], vc[1, :2, 0]])
    np.testing.assert_allclose(o[0, 0], rows.mean(0))
    np.testing.assert_allclose(lse[0, 0], np.sqrt(8) + np.log(14))


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_a_complex_product(inter):
    rng = np.random.default_rng(3)
    n = rng.standard_normal((5, 2, 12))
    f = np.array([1.0, 0.3, 0.01])
    pos = np.array([0, 1, -7, 100, 12345])
    y = decode.rotate(n, pos, f, inter, rope_scale=1.5)
    z = 1.5 * np.exp(1j * pos[:, None] * f)[:, None]
    if inter:
        w = (n[..., 0:6:2] + 1j * n[..., 1:6:2]) * z
        got = y[..., 0:6:2] + 1j * y[..., 1:6:2]
    else:
        w = (n[..., :3] + 1j * n[..., 3:6]) * z
        got = y[..., :3] + 1j * y[..., 3:6]
    np.testing.assert_allclose(got, w, atol=1e-12)
    np.testing.assert_array_equal(y[..., 6:], n[..., 6:])
    np.testing.assert_array_equal(y[0, :, 6:], n[0, :, 6:])


def test_norm_matches_torch_rms_norm():
    rng = np.random.default_rng(4)
    x, w = rng.standard_normal((3, 2, 16)), rng.standard_normal(16)
    y = decode.norm_rope_fwd(x, w, [0, 0, 0], np.ones(4), eps=1e-6)
    ref = torch.nn.functional.rms_norm(torch.from_numpy(x), (16,), torch.from_numpy(w), eps=1e-6)
    np.testing.assert_allclose(y, ref.numpy(), rtol=1e-12)


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_backward_matches_finite_differences(inter):
    rng = np.random.default_rng(5)
    x, w, dy = rng.standard_normal((3, 2, 8)), rng.standard_normal(8), rng.standard_normal((3, 2, 8))
    f, pos = np.array([1.0, 0.1]), [0, 3, 1000]
    dx, dw = decode.norm_rope_bwd(x, w, pos, f, dy, inter, rope_scale=0.8)

    def loss(x_, w_):
        return np.sum(dy * decode.norm_rope_fwd(x_, w_, pos, f, inter, rope_scale=0.8))

    h = 1e-6
    for arr, grad, at in ((x, dx, 0), (w, dw, 1)):
        for i in np.ndindex(arr.shape):
            p, m = arr.copy(), arr.copy()
            p[i] += h
            m[i] -= h
            d = (loss(p, w) - loss(m, w)) if at == 0 else (loss(x, p) - loss(x, m))
            assert abs(d / (2 * h) - grad[i]) < 1e-7


def test_slot_map_worked_example():
    """Pages of 4.  Request 0 has 3 tokens (page 9) and gets 2: one more on page 9, one on the
    first free page.  Request 1 has none and gets none.  Request 2 has 8 (pages 5, 6) and gets 5:
    two free pages."""
    table = np.array([[9, -1, -1, -1], [-1] * 4, [5, 6, -1, -1]])
    seq, cu, pos, slots, table, used = decode.slot_map([3, 0, 8], [2, 0, 5], [2, 0, 7, 1], table,
                                                       4, 10, 9)
    assert seq.tolist() == [5, 0, 13] and cu.tolist() == [0, 2, 2, 7] and used == 3
    assert pos.tolist() == [3, 4, 8, 9, 10, 11, 12, 0, 0]
    assert slots.tolist() == [39, 8, 0, 1, 2, 3, 28, -1, -1]
    assert table.tolist() == [[9, 2, -1, -1], [-1] * 4, [5, 6, 0, 7]]
