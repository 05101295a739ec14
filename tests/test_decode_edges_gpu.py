"""GPU tests of the decode-step calls at places where a definition is easily missed: softmax weights
that a short type cannot hold, infinite values.  Bounds are counted as in test_decode_gpu.py."""
import numpy as np
import pytest
import torch

import chunked_state_scan_gated_gb300 as gdn
from test_decode_gpu import BF, F32, U, attn_inputs, half, n64, within

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
