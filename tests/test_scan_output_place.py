"""Where the selective scan's output may lie: on none of its inputs' values but x's or z's own place.  No GPU is used."""
from __future__ import annotations

import ctypes

import pytest

from gated_deltanet_linear_gdr_gb300 import _binding as B
from tests.test_scan_abi import FAKE, INV, lib, scan  # noqa: F401

AWAY = dict(dt=2 * FAKE, B=2 * FAKE, C=2 * FAKE)
# x, z [8, 4, 32] and B, C [8, 2, 16] of bfloat16, out on x; a token has 256 bytes, a head 64


@pytest.mark.parametrize("over,on", [
    (dict(out=FAKE + 2), "x"), (dict(out=FAKE - 64), "x"), (dict(out=FAKE + 8 * 256 - 2), "x"), (dict(out_seq_stride=160), "x"),
    (dict(out_head_stride=40, out_seq_stride=160), "x"), (dict(x_seq_stride=0), "x"), (dict(x_head_stride=0), "x"),
    (dict(total_tokens=1, out=FAKE + 64), "x"), (dict(z=FAKE + 8), "z"), (dict(z=FAKE, z_head_stride=0), "z"),
    # between x's heads, one value too far
    (dict(x_seq_stride=256, x_head_stride=64, out_seq_stride=256, out_head_stride=64, out=FAKE + 62), "x"),
    (dict(dt=FAKE), "dt"), (dict(dt=FAKE + 8 * 256 - 2), "dt"), (dict(dt=FAKE + 2, dt_seq_stride=4, dt_head_stride=1, dt_elem_stride=0), "dt"),
    (dict(dt=FAKE - 4, dt_dtype=B.GDR_F32), "dt"), (dict(B=FAKE + 128), "B"), (dict(B=FAKE + 8 * 256 - 2, B_seq_stride=0), "B"),
    (dict(C=FAKE - 30), "C"), (dict(C=FAKE, x=3 * FAKE, C_head_stride=0), "C")])
def test_output_on_an_input_is_refused(lib, over, on):  # noqa: F811
    assert lib.gdr_selective_scan(ctypes.byref(scan(**{**AWAY, **over})), None) == INV
    assert lib.gdr_last_error().decode() == f"gdr_selective_scan: out lies on {on}"
