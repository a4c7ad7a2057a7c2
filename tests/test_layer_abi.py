"""Host-side checks of the layer operators' C ABI: struct layouts and
refusals before anything is launched.  No GPU is used."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

from gated_deltanet_linear_gdr_gb300 import _binding as B
from gated_deltanet_linear_gdr_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7f0000000000  # never dereferenced: the calls below stop at their checks


@pytest.fixture(scope="module")
def lib():
    return B.load_library(libbuild.build())


@pytest.mark.parametrize("cls,name", [(B.gdr_linattn_args, "gdr_linattn_args"), (B.gdr_norm_args, "gdr_norm_args")])
def test_struct_layout_matches_header(tmp_path, cls, name):
    fields = [f[0] for f in cls._fields_]
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gdr.h"\nint main(void) {\n'
                    f'  printf("size %zu\\n", sizeof({name}));\n' +
                    "".join(f'  printf("{f} %zu\\n", offsetof({name}, {f}));\n' for f in fields) + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                        check=True).stdout.splitlines())
    assert int(got["size"]) == ctypes.sizeof(cls)
    for f in fields:
        assert int(got[f]) == getattr(cls, f).offset, f


def linattn(**over):
    a = B.gdr_linattn_args()
    v = dict(batch=2, nv=4, nk=2, K=64, V=128, token_dtype=B.GDR_BF16, state_dtype=B.GDR_BF16, total_tokens=8, q=FAKE,
             q_seq_stride=128, q_head_stride=64, k=FAKE, k_seq_stride=128, k_head_stride=64, v=FAKE, v_seq_stride=512,
             v_head_stride=128, decay=FAKE, decay_stride=1, out=FAKE, out_seq_stride=512, out_head_stride=128, state=FAKE,
             state_slot_stride=4 * 64 * 128, state_head_stride=64 * 128, state_kdim_stride=128, state_vdim_stride=1,
             max_slots=4, slot_idx=FAKE, offsets=FAKE)
    v.update(over)
    for n, x in v.items():
        setattr(a, n, x)
    return a


INV, UNS = B.GDR_ERR_INVALID_ARG, B.GDR_ERR_UNSUPPORTED


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), INV), (dict(nv=0), INV), (dict(nk=3), INV), (dict(K=72), UNS), (dict(K=144), UNS), (dict(V=8), UNS),
    (dict(V=272), UNS), (dict(token_dtype=2), UNS), (dict(state_dtype=-1), UNS), (dict(total_tokens=-1), INV),
    (dict(total_tokens=1 << 31), UNS), (dict(batch=1 << 30), UNS), (dict(state=None), INV), (dict(slot_idx=None), INV),
    (dict(offsets=None), INV), (dict(decay=None), INV), (dict(decay_stride=-1), INV), (dict(max_slots=0), INV),
    (dict(state_vdim_stride=2), UNS), (dict(state_kdim_stride=0), INV), (dict(state_kdim_stride=129), UNS),
    (dict(state=FAKE + 8), UNS), (dict(q=None), INV), (dict(out=None), INV), (dict(v_seq_stride=-1), INV),
    (dict(out_seq_stride=0), INV), (dict(q=FAKE + 1), UNS), (dict(workspace=FAKE + 4), UNS), (dict(workspace_bytes=-1), INV)])
def test_linattn_rejects(lib, over, code):
    assert lib.gdr_linattn_fwd(ctypes.byref(linattn(**over)), None) == code
    assert lib.gdr_last_error().decode().startswith("gdr_linattn_fwd")


def test_linattn_null_and_empty(lib):
    assert lib.gdr_linattn_fwd(None, None) == INV
    assert lib.gdr_linattn_workspace_bytes(None) == INV
    assert lib.gdr_linattn_workspace_bytes(ctypes.byref(linattn(K=8))) == UNS
    assert lib.gdr_linattn_workspace_bytes(ctypes.byref(linattn(max_row_len=1))) == 0
    assert lib.gdr_linattn_fwd(ctypes.byref(linattn(batch=0, state=None)), None) == B.GDR_OK


def norm(**over):
    a = B.gdr_norm_args()
    v = dict(tokens=4, heads=2, D=64, eps=1e-6, residual_scale=1.0, has_post_norm=1, x=FAKE, x_seq_stride=128,
             x_head_stride=64, gate=FAKE, gate_seq_stride=128, gate_head_stride=64, gate_elem_stride=1, out=FAKE,
             out_seq_stride=128, out_head_stride=64)
    v.update(over)
    for n, x in v.items():
        setattr(a, n, x)
    return a


@pytest.mark.parametrize("over,code", [
    (dict(tokens=-1), INV), (dict(heads=0), INV), (dict(D=0), INV), (dict(D=16385), UNS), (dict(tokens=1 << 31), UNS),
    (dict(x_dtype=2), UNS), (dict(out_dtype=-1), UNS), (dict(activation=3), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(x=None), INV), (dict(x=None, residual=FAKE), INV),
    (dict(gate_first=1, has_post_norm=0), INV), (dict(gate_first=1, gate=None), INV), (dict(out=None), INV),
    (dict(gate_elem_stride=2), UNS), (dict(x_seq_stride=-1), INV), (dict(out_seq_stride=0), INV),
    (dict(out_head_stride=0), INV), (dict(x=FAKE + 2), UNS), (dict(post_weight=FAKE + 2), UNS)])
def test_norm_rejects(lib, over, code):
    assert lib.gdr_block_norm(ctypes.byref(norm(**over)), None) == code
    assert lib.gdr_last_error().decode().startswith("gdr_block_norm")


def test_norm_null_and_empty(lib):
    assert lib.gdr_block_norm(None, None) == INV
    assert lib.gdr_block_norm(ctypes.byref(norm(tokens=0)), None) == B.GDR_OK
