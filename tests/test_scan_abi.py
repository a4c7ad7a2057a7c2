"""Host-side checks of the C ABI of the state space operators and the
verification of drafts: struct layouts and refusals before anything is launched.  No GPU is used."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from gated_deltanet_linear_gdr_gb300 import _binding as B
from gated_deltanet_linear_gdr_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7f0000000000  # never dereferenced: the calls below stop at their checks
INV, UNS = B.GDR_ERR_INVALID_ARG, B.GDR_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return B.load_library(libbuild.build())


@pytest.mark.parametrize("cls", [B.gdr_short_conv_args, B.gdr_scan_args, B.gdr_accept_args])
def test_struct_layout_matches_header(tmp_path, cls):
    name, fields = cls.__name__, [f[0] for f in cls._fields_]
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


def _fill(cls, values, over):
    a = cls()
    for n, x in {**values, **over}.items():
        setattr(a, n, x)
    return a


def conv(**over):
    return _fill(B.gdr_short_conv_args, dict(
        batch=2, channels=64, width=4, token_dtype=B.GDR_BF16, state_dtype=B.GDR_F32, keep_state=1, total_tokens=8, x=FAKE,
        x_seq_stride=64, weight=FAKE, weight_chan_stride=4, weight_tap_stride=1, out=2 * FAKE, out_seq_stride=64, conv_state=FAKE,
        state_slot_stride=192, state_chan_stride=3, state_tap_stride=1, max_slots=4, slot_idx=FAKE, offsets=FAKE), over)


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), INV), (dict(total_tokens=-1), INV), (dict(total_tokens=1 << 31), UNS), (dict(channels=0), INV),
    (dict(batch=(1 << 27) + 1), UNS),
    (dict(channels=1 << 29), UNS), (dict(width=0), UNS), (dict(width=5), UNS), (dict(activation=2), INV), (dict(token_dtype=2), UNS),
    (dict(state_dtype=-1), UNS), (dict(slot_idx=None), INV), (dict(offsets=None), INV), (dict(weight=None), INV),
    (dict(max_slots=0), INV), (dict(weight_tap_stride=-1), INV), (dict(weight=FAKE + 2), UNS), (dict(bias=FAKE + 2), UNS),
    (dict(counts=FAKE, keep_state=0), INV), (dict(out=None, keep_state=0), INV), (dict(conv_state=None), INV),
    (dict(state_tap_stride=0), INV), (dict(conv_state=FAKE + 2), UNS), (dict(x=None), INV), (dict(x_seq_stride=-1), INV),
    (dict(x=FAKE + 1), UNS), (dict(out=FAKE + 1), UNS), (dict(out_seq_stride=63), INV), (dict(out=FAKE), INV),
    (dict(out=FAKE + 64), INV), (dict(out=FAKE + 2 * 7 * 64), INV), (dict(out=FAKE + 128, x_seq_stride=96, out_seq_stride=96), INV),
    (dict(out=FAKE + 128, x_seq_stride=128, out_seq_stride=96), INV), (dict(out=FAKE - 2, x_seq_stride=200, out_seq_stride=200), INV)])
def test_conv_rejects(lib, over, code):
    assert lib.gdr_short_conv(ctypes.byref(conv(**over)), None) == code
    assert lib.gdr_last_error().decode().startswith("gdr_short_conv")


def scan(**over):
    return _fill(B.gdr_scan_args, dict(
        batch=2, nv=4, nk=2, K=16, V=32, token_dtype=B.GDR_BF16, dt_dtype=B.GDR_BF16, state_dtype=B.GDR_F32, keep_state=1,
        total_tokens=8, x=FAKE, x_seq_stride=128, x_head_stride=32, dt=FAKE, dt_seq_stride=128, dt_head_stride=32, dt_elem_stride=1,
        B=FAKE, B_seq_stride=32, B_head_stride=16, C=FAKE, C_seq_stride=32, C_head_stride=16, A=FAKE, A_head_stride=512,
        A_kdim_stride=32, A_vdim_stride=1, out=FAKE, out_seq_stride=128, out_head_stride=32, state=FAKE, state_slot_stride=2048,
        state_head_stride=512, state_kdim_stride=32, state_vdim_stride=1, max_slots=4, slot_idx=FAKE, offsets=FAKE), over)


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), INV), (dict(nv=0), INV), (dict(nk=3), INV), (dict(K=0), UNS), (dict(K=129), UNS), (dict(V=0), UNS),
    (dict(V=1 << 23), UNS), (dict(token_dtype=2), UNS), (dict(dt_dtype=2), UNS), (dict(token_dtype=B.GDR_F32), UNS),
    (dict(state_dtype=-1), UNS), (dict(total_tokens=-1), INV), (dict(total_tokens=1 << 31), UNS), (dict(state=None), INV),
    (dict(total_tokens=(1 << 31) - 31), UNS), (dict(batch=(1 << 27) + 1), UNS),
    (dict(slot_idx=None), INV), (dict(offsets=None), INV), (dict(A=None), INV), (dict(max_slots=0), INV),
    (dict(state_vdim_stride=2), UNS), (dict(state_kdim_stride=0), INV), (dict(A_vdim_stride=-1), INV), (dict(D_head_stride=-1), INV),
    (dict(state=FAKE + 2), UNS), (dict(A=FAKE + 2), UNS), (dict(D=FAKE + 2), UNS), (dict(dt_bias=FAKE + 1), UNS),
    (dict(counts=FAKE, keep_state=0), INV), (dict(out=None, keep_state=0), INV), (dict(x=None), INV), (dict(dt=None), INV),
    (dict(B=None), INV), (dict(C=None), INV), (dict(z_seq_stride=-1), INV), (dict(dt_elem_stride=2), UNS),
    (dict(out_seq_stride=0), INV), (dict(out_head_stride=0), INV), (dict(z=FAKE + 1), UNS), (dict(workspace=FAKE + 4), UNS),
    (dict(workspace_bytes=-1), INV)])
def test_scan_rejects(lib, over, code):
    assert lib.gdr_selective_scan(ctypes.byref(scan(**over)), None) == code
    assert lib.gdr_last_error().decode().startswith("gdr_selective_scan")


def accept(**over):
    return _fill(B.gdr_accept_args, dict(
        batch=2, vocab=100, prob_dtype=B.GDR_F32, max_row_len=4, total_tokens=8, target=FAKE, target_seq_stride=100, draft=FAKE,
        draft_seq_stride=100, tokens=FAKE, offsets=FAKE, uniforms=FAKE, row_uniforms=FAKE, out_tokens=FAKE, out_seq_stride=4,
        counts=FAKE), over)


@pytest.mark.parametrize("over,code", [
    (dict(batch=-1), INV), (dict(vocab=0), INV), (dict(vocab=1 << 29), UNS), (dict(max_row_len=0), INV), (dict(prob_dtype=3), UNS),
    (dict(total_tokens=-1), INV), (dict(total_tokens=1 << 31), UNS), (dict(offsets=None), INV), (dict(row_uniforms=None), INV),
    (dict(out_tokens=None), INV), (dict(counts=None), INV), (dict(out_seq_stride=3), INV), (dict(target=None), INV),
    (dict(tokens=None), INV), (dict(uniforms=None), INV), (dict(target_seq_stride=-1), INV), (dict(draft_seq_stride=-1), INV),
    (dict(target=FAKE + 2), UNS), (dict(draft=FAKE + 2), UNS), (dict(batch=1 << 28), UNS)])
def test_accept_rejects(lib, over, code):
    assert lib.gdr_accept_drafts(ctypes.byref(accept(**over)), None) == code
    assert lib.gdr_last_error().decode().startswith("gdr_accept_drafts")


def test_null_and_empty(lib):
    for fn in (lib.gdr_short_conv, lib.gdr_selective_scan, lib.gdr_accept_drafts):
        assert fn(None, None) == INV
    assert lib.gdr_selective_scan_workspace_bytes(None) == INV
    assert lib.gdr_selective_scan_workspace_bytes(ctypes.byref(scan(K=200))) == UNS
    assert lib.gdr_selective_scan_workspace_bytes(ctypes.byref(scan(max_row_len=1))) == 0
    assert lib.gdr_short_conv(ctypes.byref(conv(batch=0, x=None)), None) == B.GDR_OK
    assert lib.gdr_selective_scan(ctypes.byref(scan(batch=0, state=None)), None) == B.GDR_OK
    assert lib.gdr_accept_drafts(ctypes.byref(accept(batch=0, counts=None)), None) == B.GDR_OK


@pytest.mark.parametrize("bad", [None, 3, [1.0], "x"])
def test_python_calls_take_tensors(bad):
    x, w, pool, i = torch.zeros(4, 8), torch.zeros(8, 4), torch.zeros(4, 8, 3), torch.zeros(5, dtype=torch.int32)
    h, a = torch.zeros(4, 1, 8), torch.zeros(1, 8, 8)
    calls = [(gdr.gdr_short_conv, [x, w, None, pool, i[:4], i], (0, 1, 3, 4, 5)),
             (gdr.gdr_selective_scan, [h, h, a, h, h, torch.zeros(4, 1, 8, 8), i[:4], i], range(8)),
             (lambda *t: gdr.gdr_accept_drafts(*t, max_row_len=2), [x, x, i[:4], i, x[:, 0], x[:, 0]], (0, 2, 3, 4, 5))]
    for fn, args, which in calls:
        for k in which:
            broken = list(args)
            broken[k] = bad
            # the tensors are of the host, which is refused too where it is seen first
            with pytest.raises((TypeError, ValueError), match="torch.Tensor|CUDA tensor"):
                fn(*broken)
        with pytest.raises(ValueError, match="CUDA tensor"):
            fn(*args)
