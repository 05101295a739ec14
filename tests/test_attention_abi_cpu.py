"""CPU checks of the full-attention and 8-bit cache calls: struct layouts against the header, and
every refusal of the host-side validation (no launch reaches CUDA)."""
import ctypes
import os
import subprocess

import pytest

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
    structs = {"gdn_attn_seq_problem": gdn.AttnSeqProblem, "gdn_cache8_problem": gdn.Cache8Problem}
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


# ------------------------------------------------------------------- gdn_attn_fwd / _bwd

FWD = ["q", "k", "v", "cu_q", "cu_k", "o", "lse"]
BWD = ["q", "k", "v", "o", "lse", "dO", "cu_q", "cu_k", "dq", "dk", "dv"]


def seq_problem(**kw):
    p = gdn.AttnSeqProblem(gdn.GDN_BF16, 128, 1, 0.0, 3, 40, 50, 8, 2, 0, 0, 0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def call(lib, p, bwd, ws=A, ws_bytes=1 << 40, status=None, **over):
    names = BWD if bwd else FWD
    args = dict.fromkeys(names, A) | over
    fn = lib.gdn_attn_bwd if bwd else lib.gdn_attn_fwd
    return fn(p, *[args[k] for k in names], ws, ws_bytes, status, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,status", [
    ({"dtype": 3}, BAD), ({"Nq": -1}, BAD), ({"Nk": -1}, BAD), ({"Hq": 0}, BAD), ({"Hk": 0}, BAD),
    ({"Hq": 9}, BAD), ({"D": 0}, BAD), ({"n_seqs": 0}, BAD), ({"n_seqs": -1}, BAD),
    ({"causal": 2}, BAD), ({"scale": float("nan")}, BAD), ({"scale": float("inf")}, BAD),
    ({"scale": 3e38}, BAD), ({"q_stride": 1016}, BAD), ({"k_stride": 260}, BAD),
    ({"v_stride": 128}, BAD), ({"q_stride": -1024}, BAD), ({"D": 96}, UNSUP), ({"D": 512}, UNSUP),
    ({"Nq": 1 << 29}, UNSUP), ({"Nk": 1 << 31}, UNSUP), ({"n_seqs": (1 << 20) + 1}, UNSUP),
    ({"q_stride": 1 << 31}, UNSUP), ({"Hq": 1 << 24, "Hk": 1 << 24}, UNSUP),
])
def test_seq_problem_refusals(lib, bwd, kw, status):
    p = seq_problem(**kw)
    assert call(lib, p, bwd) == status
    n = ctypes.c_size_t(0)
    size = lib.gdn_attn_bwd_workspace_size if bwd else lib.gdn_attn_fwd_workspace_size
    assert size(p, ctypes.byref(n)) == status


@pytest.mark.parametrize("bwd,kw,status", [
    (b, {k: x}, BAD) for b, names in ((False, FWD), (True, BWD)) for k in names
    for x in (None, A + 2) if not (x is None and k in ("cu_k", "cu_q", "lse"))
] + [
    (True, {"lse": None}, BAD), (False, {"lse": A + 8}, BAD),
    (False, {"cu_k": None}, BAD),                      # Nk differs from Nq
    (False, {"cu_q": None}, BAD), (False, {"cu_q": None, "cu_k": None}, BAD),  # 3 does not divide
    (False, {"ws": A + 64}, BAD), (True, {"status": A + 16}, BAD),
    (False, {"ws": None}, WS), (True, {"ws_bytes": 100}, WS), (False, {"ws_bytes": 100}, WS),
])
def test_seq_pointer_refusals(lib, bwd, kw, status):
    assert call(lib, seq_problem(), bwd, **kw) == status


def test_seq_calls_without_rows_do_nothing(lib):
    p = seq_problem(Nq=0, Nk=0, n_seqs=0)
    none = dict.fromkeys(BWD)
    assert call(lib, p, True, **none) == gdn.GDN_OK
    assert call(lib, p, False, **dict.fromkeys(FWD)) == gdn.GDN_OK
    assert lib.gdn_attn_fwd(None, *[A] * 8, 1 << 40, None, None) == BAD


# ------------------------------------------------------------------ gdn_cache_write8 / _read8

WRITE = ["k", "v", "block_table", "ctx_len", "cu_seqlens", "k_cache", "v_cache", "k_scale",
         "v_scale", "status"]
READ = ["k_cache", "v_cache", "k_scale", "v_scale", "block_table", "cu_seqlens", "k", "v", "status"]


def cache(lib, read=False, prob=None, **over):
    p = gdn.Cache8Problem(gdn.GDN_BF16, 128, 16, 0, 3, 40, 2, 9, 5, 0, 0)
    for k, v in (prob or {}).items():
        setattr(p, k, v)
    names = READ if read else WRITE
    args = dict.fromkeys(names, A) | over
    return (lib.gdn_cache_read8 if read else lib.gdn_cache_write8)(
        p, *[args[k] for k in names], None)


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("prob,status", [
    ({"dtype": 3}, BAD), ({"B": -1}, BAD), ({"N": -1}, BAD), ({"Hk": 0}, BAD), ({"pages": -1}, BAD),
    ({"max_blocks": -1}, BAD), ({"page_size": 0}, BAD), ({"D": 0}, BAD), ({"k_stride": 128}, BAD),
    ({"v_stride": 260}, BAD), ({"D": 96}, UNSUP), ({"page_size": 24}, UNSUP),
    ({"pages": 1 << 28}, UNSUP), ({"max_blocks": 1 << 28}, UNSUP), ({"N": 1 << 30}, UNSUP),
    ({"B": (1 << 20) + 1}, UNSUP), ({"Hk": 1 << 24}, UNSUP),
])
def test_cache8_problem_refusals(lib, read, prob, status):
    assert cache(lib, read, prob) == status


@pytest.mark.parametrize("read,kw", [
    (r, {k: x}) for r, names in ((False, WRITE), (True, READ)) for k in names
    for x in (None, A + 2) if not (x is None and k == "status")])
def test_cache8_pointer_refusals(lib, read, kw):
    assert cache(lib, read, **kw) == BAD


def test_cache8_calls_without_tokens_do_nothing(lib):
    for read, names in ((False, WRITE), (True, READ)):
        none = dict.fromkeys(names) | {"cu_seqlens": A}
        assert cache(lib, read, {"N": 0, "B": 0, "pages": 0}, **none) == gdn.GDN_OK
    assert lib.gdn_cache_read8(None, *[A] * 9, None) == BAD


# ---------------------------------------------------------------------------- gdn_attn_decode8

DEC = ["q", "k_cache", "v_cache", "k_scale", "v_scale", "block_table", "seq_len", "o", "lse"]


def dec(lib, prob=None, ws=A, ws_bytes=1 << 40, status=None, **over):
    p = gdn.AttnProblem(gdn.GDN_BF16, 128, 16, 0.0, 3, 8, 2, 9, 5, 0)
    for k, v in (prob or {}).items():
        setattr(p, k, v)
    args = dict.fromkeys(DEC, A) | over
    return lib.gdn_attn_decode8(p, *[args[k] for k in DEC], ws, ws_bytes, status, None)


@pytest.mark.parametrize("kw,status", [
    (dict(prob={"dtype": 3}), BAD), (dict(prob={"Hq": 9}), BAD), (dict(prob={"D": 80}), UNSUP),
    (dict(prob={"page_size": 24}), UNSUP), (dict(prob={"q_stride": 1000}), BAD),
    (dict(prob={"scale": float("inf")}), BAD), (dict(prob={"pages": 1 << 28}), UNSUP),
    (dict(ws=None), WS), (dict(ws_bytes=1000), WS), (dict(ws=A + 64), BAD),
    (dict(status=A + 16), BAD), (dict(lse=A + 8), BAD),
    (dict(prob={"B": 0}, **dict.fromkeys(DEC)), gdn.GDN_OK),
] + [({k: x}, BAD) for k in DEC[:8] for x in (None, A + 2)])
def test_decode8_refusals(lib, kw, status):
    assert dec(lib, **kw) == status


def test_decode8_workspace_depends_on_head_dim_and_type_alone(lib):
    def size(**kw):
        n = ctypes.c_size_t(0)
        p = gdn.AttnProblem(gdn.GDN_BF16, 128, 16, 0.0, 3, 8, 2, 9, 5, 0)
        for k, v in kw.items():
            setattr(p, k, v)
        assert lib.gdn_attn_decode8_workspace_size(p, ctypes.byref(n)) == gdn.GDN_OK
        return n.value
    assert size() == size(B=700, Hq=96, Hk=1, pages=1000, max_blocks=77, page_size=128)
