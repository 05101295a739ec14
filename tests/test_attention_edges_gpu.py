"""GPU tests of the full-attention calls and of the 8-bit cache at places where a definition is easily
missed: offsets out of order.  Bounds are counted as in test_attention_gpu.py."""
import numpy as np
import pytest
import torch

import chunked_state_scan_gated_gb300 as gdn
from oracle import attention
from test_attention_gpu import BF, F8, F32, filled, i32, n64, rand, same, step_of, u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load_library()


# --------------------------------------------------------------------------- the 8-bit cache

def check_cut(cu, ctx, N, D, dt, P=16, Hk=2, seed=0):
    """Codes, scales and rows read back are those of the offsets as they count."""
    gen = torch.Generator().manual_seed(seed)
    B = len(ctx)
    table, pages, _ = step_of([0] * B, [N + max(max(ctx), 0)] * B, P, seed=seed)
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
