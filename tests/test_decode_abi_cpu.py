"""CPU checks of the decode-step calls: struct layouts against the header, and every refusal of
the host-side validation (no launch reaches CUDA)."""
import ctypes
import os
import subprocess

import pytest
import torch

import chunked_state_scan_gated_gb300 as gdn
from chunked_state_scan_gated_gb300 import build as gbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # a 256-byte aligned stand-in address; validation fails before any use
BAD, UNSUP, WS = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gdn.load_library()


def test_struct_layouts_match_the_header(tmp_path):
    structs = {"gdn_rope_problem": gdn.RopeProblem, "gdn_attn_problem": gdn.AttnProblem,
               "gdn_slot_problem": gdn.SlotProblem}
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "gdn.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'  printf("{name} size %zu\\n", sizeof({name}));')
        for f, _ in cls._fields_:
            lines.append(f'  printf("{name} {f} %zu\\n", offsetof({name}, {f}));')
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True,
                               text=True).stdout.splitlines():
        name, key, val = line.split()
        cls = structs[name]
        assert int(val) == (ctypes.sizeof(cls) if key == "size" else getattr(cls, key).offset)


# ----------------------------------------------------------------------------- gdn_step

STEP_ARGS = ["slots", "q", "k", "v", "a", "b", "A_log", "dt_bias", "state", "o", "status"]


def step(lib, over=None, prob=None, n_slots=9):
    p = gdn.Problem()
    lib.gdn_problem_init(ctypes.byref(p))
    p.B, p.T, p.Hqk, p.H, p.dk, p.dv = 2, 1, 16, 32, 128, 128
    for k, v in (prob or {}).items():
        setattr(p, k, v)
    args = dict.fromkeys(STEP_ARGS, A) | (over or {})
    return lib.gdn_step(p, n_slots, *[args[k] for k in STEP_ARGS], None)


@pytest.mark.parametrize("kw,status", [
    (dict(prob={"T": 2}), BAD), (dict(prob={"T": 0}), BAD), (dict(prob={"H": 24}), BAD),
    (dict(prob={"dtype": 5}), BAD), (dict(prob={"dk": 64}), UNSUP),
    (dict(prob={"chunk": 32}), UNSUP), (dict(n_slots=-1), BAD),
    (dict(n_slots=1 << 31), UNSUP), (dict(over={"slots": None}, n_slots=1), BAD),
    (dict(over={"slots": A + 2}), BAD), (dict(over={"status": A + 16}), BAD),
    (dict(prob={"B": 0}, over=dict.fromkeys(STEP_ARGS)), gdn.GDN_OK),
] + [(dict(over={k: x}), BAD) for k in STEP_ARGS[1:10] for x in (None, A + 8)])
def test_step_refusals(lib, kw, status):
    assert step(lib, **kw) == status


# ------------------------------------------------------------------- gdn_qk_norm_rope_*

def rope_problem(**kw):
    p = gdn.RopeProblem(gdn.GDN_BF16, 128, 64, 0, 10, 0, 4, 2, 0, 0, 0, 1e-6, 1.0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


FWD = ["q", "k", "wq", "wk", "inv_freq", "positions", "q_out", "k_out"]
BWD = FWD[:6] + ["dq_out", "dk_out", "dq", "dk", "dwq", "dwk"]


def rope_fwd(lib, p, **over):
    args = dict.fromkeys(FWD, A) | over
    return lib.gdn_qk_norm_rope_fwd(p, *[args[k] for k in FWD], None)


def rope_bwd(lib, p, ws=A, ws_bytes=1 << 40, **over):
    args = dict.fromkeys(BWD, A) | over
    return lib.gdn_qk_norm_rope_bwd(p, *[args[k] for k in BWD], ws, ws_bytes, None)


def rope_cache(lib, p, n_slots=64, **over):
    a = dict.fromkeys(["q", "k", "v", "wq", "wk", "inv_freq", "positions", "slots", "q_out",
                       "k_cache", "v_cache", "status"], A) | over
    return lib.gdn_qk_norm_rope_cache(
        p, a["q"], a["k"], a["v"], a["wq"], a["wk"], a["inv_freq"], a["positions"], n_slots,
        a["slots"], a["q_out"], a["k_cache"], a["v_cache"], a["status"], None)


@pytest.mark.parametrize("kw,status", [
    ({"dtype": 3}, BAD), ({"N": -1}, BAD), ({"T": -1}, BAD), ({"Hq": -1}, BAD),
    ({"Hq": 0, "Hk": 0}, BAD), ({"D": 0}, BAD), ({"R": -16}, BAD), ({"R": 144}, BAD),
    ({"eps": -1.0}, BAD), ({"eps": float("nan")}, BAD), ({"rope_scale": float("inf")}, BAD),
    ({"q_stride": 504}, BAD), ({"k_stride": 260}, BAD), ({"v_stride": 128}, BAD),
    ({"D": 100}, UNSUP), ({"D": 264, "R": 64}, UNSUP), ({"R": 40}, UNSUP),
    ({"N": 1 << 29}, UNSUP),
])
def test_rope_problem_refusals(lib, kw, status):
    p = rope_problem(**kw)
    n = ctypes.c_size_t(0)
    assert rope_fwd(lib, p) == status
    assert rope_bwd(lib, p) == status
    assert rope_cache(lib, p) == status
    assert lib.gdn_qk_norm_rope_bwd_workspace_size(p, ctypes.byref(n)) == status


def test_rope_pointer_refusals(lib):
    p = rope_problem()
    for k in FWD:
        assert rope_fwd(lib, p, **{k: A + (2 if k == "positions" else 8)}) == BAD
        if k != "positions":
            assert rope_fwd(lib, p, **{k: None}) == BAD
    for k in BWD:
        assert rope_bwd(lib, p, **{k: A + (2 if k == "positions" else 8)}) == BAD
    for k in ("v", "slots", "k_cache", "v_cache", "q_out"):
        assert rope_cache(lib, p, **{k: None}) == BAD
    assert rope_cache(lib, p, status=A + 4) == BAD
    assert rope_cache(lib, p, n_slots=-1) == BAD
    assert rope_cache(lib, p, n_slots=1 << 31) == UNSUP
    assert rope_fwd(lib, rope_problem(N=0), **dict.fromkeys(FWD)) == gdn.GDN_OK


def test_rope_workspace(lib):
    size = gdn.gdn_qk_norm_rope_bwd_workspace_size
    assert size(rope_problem(N=0)) == 0
    assert size(rope_problem(N=1 << 20)) == size(rope_problem(N=1 << 21)) > 0  # grid is capped
    p = rope_problem(N=1000)
    assert rope_bwd(lib, p, ws_bytes=size(p) - 4) == WS
    assert rope_bwd(lib, p, ws=None) == WS
    assert rope_bwd(lib, p, ws=A + 4) == WS
    assert lib.gdn_qk_norm_rope_bwd_workspace_size(p, None) == BAD


# --------------------------------------------------------------------- gdn_attn_decode

ATTN = ["q", "k_cache", "v_cache", "block_table", "seq_len", "o", "lse"]


def attn(lib, prob=None, ws=A, ws_bytes=1 << 40, status=A, **over):
    p = gdn.AttnProblem(gdn.GDN_BF16, 128, 16, 0.0, 3, 8, 2, 100, 10, 0)
    for k, v in (prob or {}).items():
        setattr(p, k, v)
    args = dict.fromkeys(ATTN, A) | over
    return lib.gdn_attn_decode(p, *[args[k] for k in ATTN], ws, ws_bytes, status, None)


@pytest.mark.parametrize("kw,status", [
    ({"dtype": 2}, BAD), ({"B": -1}, BAD), ({"Hq": 0}, BAD), ({"Hk": 0}, BAD), ({"Hk": 3}, BAD),
    ({"pages": -1}, BAD), ({"max_blocks": -1}, BAD), ({"page_size": 0}, BAD), ({"D": 0}, BAD),
    ({"scale": float("nan")}, BAD), ({"scale": float("inf")}, BAD), ({"q_stride": 1016}, BAD), ({"q_stride": 1028}, BAD),
    ({"D": 96}, UNSUP), ({"page_size": 24}, UNSUP), ({"pages": 1 << 27}, UNSUP),
    ({"max_blocks": 1 << 27}, UNSUP), ({"B": 1 << 28}, UNSUP),
])
def test_attn_problem_refusals(lib, kw, status):
    assert attn(lib, kw) == status
    p = gdn.AttnProblem(gdn.GDN_BF16, 128, 16, 0.0, 3, 8, 2, 100, 10, 0)
    for k, v in kw.items():
        setattr(p, k, v)
    n = ctypes.c_size_t(0)
    assert lib.gdn_attn_decode_workspace_size(p, ctypes.byref(n)) == status


def test_attn_pointer_refusals(lib):
    for k in ATTN:
        assert attn(lib, **{k: A + 2}) == BAD
        if k != "lse":
            assert attn(lib, **{k: None}) == BAD
    assert attn(lib, ws=A + 16) == BAD
    assert attn(lib, status=A + 16) == BAD
    assert attn(lib, ws=None) == WS
    assert attn(lib, ws_bytes=8) == WS
    assert attn(lib, {"B": 0}, **dict.fromkeys(ATTN)) == gdn.GDN_OK


# ------------------------------------------------------------------------ gdn_slot_map

SLOT = ["ctx_len", "new_len", "free_pages", "block_table", "seq_len", "cu_seqlens", "positions",
        "slots", "used", "status"]


def slot_map(lib, prob=None, **over):
    p = gdn.SlotProblem(16, 0, 3, 10, 100, 20, 64)
    for k, v in (prob or {}).items():
        setattr(p, k, v)
    args = dict.fromkeys(SLOT, A) | over
    return lib.gdn_slot_map(p, *[args[k] for k in SLOT], None)


@pytest.mark.parametrize("kw,status", [
    ({"page_size": 0}, BAD), ({"B": -1}, BAD), ({"max_blocks": -1}, BAD), ({"pages": -1}, BAD),
    ({"n_free": -1}, BAD), ({"n_tokens": -1}, BAD), ({"B": 1 << 31}, UNSUP),
    ({"pages": 1 << 27}, UNSUP), ({"max_blocks": 1 << 27}, UNSUP), ({"n_free": 1 << 31}, UNSUP),
    ({"n_tokens": 1 << 31}, UNSUP),
])
def test_slot_map_problem_refusals(lib, kw, status):
    assert slot_map(lib, kw) == status


def test_slot_map_pointer_refusals(lib):
    for k in SLOT:
        assert slot_map(lib, **{k: A + 2}) == BAD
        if k != "status":
            assert slot_map(lib, **{k: None}) == BAD


def test_slot_map_lengths_in_place_are_refused(lib):
    assert slot_map(lib, ctx_len=2 * A, seq_len=2 * A) == BAD
    assert slot_map(lib, new_len=2 * A, seq_len=2 * A) == BAD


def test_binding_refuses_host_tensors_and_wrong_layouts():
    """The binding's own checks, on the CPU: no address reaches the library."""
    q, k = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    w, f = torch.zeros(64), torch.zeros(8)
    with pytest.raises(ValueError):
        gdn.gdn_qk_norm_rope_fwd(q, k, w, w, f)
    with pytest.raises(ValueError):
        gdn.gdn_attn_decode(q, torch.zeros(2, 16, 2, 64), torch.zeros(2, 16, 2, 64),
                            torch.zeros(3, 1, dtype=torch.int32),
                            torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        gdn.gdn_step(torch.zeros(1, 2, 1, 16), q, q, q, q, w, w, torch.zeros(1, 1, 16, 16))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_slot_map(i, i, i, torch.zeros(2, 2, dtype=torch.int32), page_size=16, pages=4,
                         n_tokens=8)
    # evenly spaced tokens are accepted, anything else refused (the address check aside)
    x = torch.zeros(2, 3, 10, 64)
    assert gdn._rows("q", x[:, :, 2:6], -1, torch.float32, (2, 3, 4, 64))[1] == 640
    assert gdn._rows("q", x[:, :1, 2:6], -1, torch.float32, (2, 1, 4, 64))[1] == 1920
    for bad in (x[:, :2, 2:6], x[:, :, ::2], x[..., ::2], x.transpose(1, 2)):
        with pytest.raises(ValueError):
            gdn._rows("q", bad, -1, torch.float32, bad.shape)


def test_binding_refuses_an_expanded_token():
    """A stride of zero between tokens is no layout of the library's (its 0 means contiguous)."""
    x = torch.zeros(1, 4, 64)
    for bad in (x.expand(5, 4, 64), x.expand(2, 5, 4, 64), x[:, :2].expand(5, 2, 64),
                torch.zeros(1, 1, 4, 64).expand(6, 1, 4, 64), torch.zeros(5, 1, 64).expand(5, 4, 64)):
        with pytest.raises(ValueError):
            gdn._rows("q", bad, -1, torch.float32, bad.shape)
    assert gdn._rows("q", x, -1, torch.float32, (1, 4, 64))[1] == 0


def test_binding_takes_one_token_without_leading_sizes():
    q, k = torch.zeros(4, 64), torch.zeros(2, 64)
    p = gdn._rope_problem(q, k, None, -1, torch.zeros(8), None, False, 1e-6, 1.0)[0]
    assert (p.N, p.T, p.Hq, p.Hk, p.D, p.q_stride) == (1, 0, 4, 2, 64, 0)
