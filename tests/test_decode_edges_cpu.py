"""CPU tests of refusals that the decode-step calls owe at their edges: arrays of one call that lie on
one another, a scale that only overflows once it is in base 2.  Validation fails before any launch,
so the addresses are stand-ins."""
import ctypes
import itertools

import pytest

import chunked_state_scan_gated_gb300 as gdn
from chunked_state_scan_gated_gb300 import build as gbuild

A = 1 << 20
BAD = gdn.GDN_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load_library()


# int32 elements of each array of gdn_slot_map below
B, BLOCKS, FREE, ROWS = 3, 10, 20, 64
SIZES = {"ctx_len": B, "new_len": B, "free_pages": FREE, "block_table": B * BLOCKS, "seq_len": B,
         "cu_seqlens": B + 1, "positions": ROWS, "slots": ROWS, "used": 1}
INPUTS = ("ctx_len", "new_len", "free_pages")


@pytest.mark.parametrize("x,y", [p for p in itertools.combinations(SIZES, 2)
                                 if not set(p) <= set(INPUTS)])
def test_slot_map_arrays_that_overlap_are_refused(lib, x, y):
    """y begins on x's first element, on its last one, or ends on its first one."""
    p = gdn.SlotProblem(16, 0, B, BLOCKS, 100, FREE, ROWS)
    for shift in (0, SIZES[x] - 1, 1 - SIZES[y]):
        at = {k: A * (i + 1) for i, k in enumerate(SIZES)}
        at[y] = at[x] + 4 * shift
        assert lib.gdn_slot_map(p, *[at[k] for k in SIZES], None, None) == BAD, shift


@pytest.mark.parametrize("scale,status", [(2.3e38, gdn.GDN_OK), (2.4e38, BAD), (3.4e38, BAD),
                                          (-3.4e38, gdn.GDN_OK), (1e-45, gdn.GDN_OK)])
def test_attention_scale_has_to_be_finite_in_base_2(lib, scale, status):
    """exp(scale x) is taken as 2^(scale log2(e) x): an infinite factor makes 0 * inf of equal
    scores.  Below 0 the scale means the default."""
    p = gdn.AttnProblem(gdn.GDN_BF16, 128, 16, scale, 3, 8, 2, 100, 10, 0)
    n = ctypes.c_size_t(0)
    assert lib.gdn_attn_decode_workspace_size(p, ctypes.byref(n)) == status
