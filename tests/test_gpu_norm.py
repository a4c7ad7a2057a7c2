"""The fused block norms (gdr_gate_norm, gdr_residual_norm) against float64,
over widths, types, gates, strides and refusals."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from tests.layer_helpers import U16, U32, norm_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _randn(*shape, dtype=F32, seed=0, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def check(got, ref, D):
    """A row's statistics are sums of D float32 products (at most D + 8 roundings, of terms of one sign, or
    of differences from a mean that is good to D U32 of the largest entry), the gate's exponential and the
    products add under 32 roundings; with entries within a factor of 16 of the row's rms every value is good to
    32 (D + 40) U32 of itself plus of the row's rms, and the output's type rounds once."""
    err = (got.double() - ref).abs()
    rms = ref.pow(2).mean(-1, keepdim=True).sqrt()
    tol = 32 * (D + 40) * U32 * (ref.abs() + rms) + (U16 if got.dtype == BF16 else 0.0) * ref.abs() + 1e-30
    assert bool((err <= tol).all()), f"{float((err / tol).max()):.3g} x the bound"
    if ref.numel() >= 4096:  # independent roundings: far below the worst case
        rel = float((got.double() - ref).norm() / ref.norm())
        assert rel <= (U16 if got.dtype == BF16 else 2e-6), f"relative error {rel:.3g}"


@pytest.mark.parametrize("D", [1, 7, 64, 80, 128, 200, 256, 513, 1000, 1024, 2047, 2048, 4096, 8192, 16384])
@pytest.mark.parametrize("x,g,y", [(BF16, BF16, BF16), (F32, BF16, BF16), (F32, F32, F32), (BF16, F32, F32)])
@pytest.mark.parametrize("gate_first,centered", [(False, False), (True, True)])
def test_gate_norm(D, x, g, y, gate_first, centered):
    H = 3 if D <= 256 else 1
    a, z, w = _randn(5, H, D, dtype=x, std=2.0), _randn(5, H, D, dtype=g, seed=1), 1 + 0.1 * _randn(D, seed=2)
    got = gdr.gdr_gate_norm(a, z, w, out_dtype=y, gate_first=gate_first, centered=centered)
    assert got.dtype == y and got.shape == a.shape
    if D == 1 and centered:
        assert not got.any()
        return
    check(got, norm_ref(a, gate=z, act="silu", gate_first=gate_first, post=True, post_w=w, centered=centered)[1], D)


@pytest.mark.parametrize("act", [None, "silu", "sigmoid"])
def test_gate_norm_forms(act):
    a, z = _randn(9, 4, 128, dtype=BF16), _randn(9, 4, 128, dtype=BF16, seed=1)
    check(gdr.gdr_gate_norm(a, z, activation=act), norm_ref(a, gate=z, act=act, post=True)[1], 128)
    check(gdr.gdr_gate_norm(a, z[..., :1], activation=act), norm_ref(a, gate=z[..., :1], act=act, post=True)[1], 128)
    check(gdr.gdr_gate_norm(a, None), norm_ref(a, post=True)[1], 128)
    check(gdr.gdr_gate_norm(a[:, 0], z[:, 0], activation=act), norm_ref(a[:, 0], gate=z[:, 0], act=act, post=True)[1], 128)


@pytest.mark.parametrize("D", [7, 64, 256, 1000, 2047, 2048, 4096, 5000, 8192, 16384])
@pytest.mark.parametrize("x,h,y", [(BF16, BF16, BF16), (BF16, F32, BF16), (F32, F32, F32)])
@pytest.mark.parametrize("gate", ["none", "element", "token", "channel"])
def test_residual_norm(D, x, h, y, gate):
    T = 6
    block, res = _randn(T, D, dtype=x), _randn(T, D, dtype=h, seed=1, std=3.0)
    w, pw = 1 + 0.1 * _randn(D, seed=2), 1 + 0.1 * _randn(D, seed=3)
    shape = {"none": None, "element": (T, D), "token": (T, 1), "channel": (D,)}[gate]
    z = None if shape is None else _randn(*shape, dtype=x, seed=4)
    for post, centered, act in [(pw, False, "sigmoid"), (None, True, "silu")]:
        if D == 7 and centered:
            continue
        ro, out = gdr.gdr_residual_norm(block, res, w, post_weight=post, gate=z, activation=act if z is not None else None,
                                        residual_scale=0.7, centered=centered, out_dtype=y)
        rh, rout = norm_ref(block, gate=z, act=act, post=post is not None, post_w=post, residual=res, scale=0.7, pre=True,
                            pre_w=w, centered=centered)
        assert ro.dtype == h and out.dtype == y
        check(ro, rh, D)
        check(out, rout, D)


@pytest.mark.parametrize("D", [4097, 6001, 8191, 8193, 16383, 6168, 8200])
@pytest.mark.parametrize("x,h", [(BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("gate", ["element", "token"])
@pytest.mark.parametrize("centered", [False, True])
def test_wide_rows(D, x, h, gate, centered):
    block, res = _randn(3, D, dtype=x), _randn(3, D, dtype=h, seed=1)
    z = _randn(3, D if gate == "element" else 1, dtype=x, seed=2)
    w, pw = 1 + 0.1 * _randn(D, seed=3), 1 + 0.1 * _randn(D, seed=4)
    got_h, got = gdr.gdr_residual_norm(block, res, w, post_weight=pw, gate=z, activation="sigmoid", residual_scale=0.7,
                                       centered=centered, out_dtype=BF16)
    rh, rout = norm_ref(block, gate=z, act="sigmoid", post=True, post_w=pw, residual=res, scale=0.7, pre=True, pre_w=w,
                        centered=centered)
    check(got_h, rh, D)
    check(got, rout, D)


@pytest.mark.parametrize("D", [2, 66, 130, 510, 514, 2046, 2050, 4094, 4098, 8190, 8194, 16382])
@pytest.mark.parametrize("x,h", [(BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("gate", ["none", "element", "channel"])
def test_even_widths(D, x, h, gate):
    """Rows of pairs, among them views whose rows begin on an even element, and on an odd one."""
    T, w = 5, 1 + 0.1 * _randn(D, seed=3)
    for first in (0, 2, 1):
        block = _randn(T, D + 4, dtype=x)[:, first:first + D]
        res = _randn(T, D + 2, dtype=h, seed=1)[:, :D]
        z = {"none": None, "element": _randn(T, D, dtype=x, seed=2), "channel": _randn(D, dtype=x, seed=2)}[gate]
        act = None if z is None else "silu"
        got_h, got = gdr.gdr_residual_norm(block, res, w, post_weight=w, gate=z, activation=act, residual_scale=0.7,
                                           out_dtype=BF16)
        rh, rout = norm_ref(block, gate=z, act=act, post=True, post_w=w, residual=res, scale=0.7, pre=True, pre_w=w)
        check(got_h, rh, D)
        check(got, rout, D)


def test_residual_norm_first_of_a_stack_and_in_place():
    res, w = _randn(5, 512, dtype=BF16), 1 + 0.1 * _randn(512, seed=1)
    h, out = gdr.gdr_residual_norm(None, res, w)
    assert h is res
    check(out, norm_ref(None, residual=res, pre=True, pre_w=w)[1], 512)
    block = _randn(5, 512, dtype=BF16, seed=2)
    rh, rout = norm_ref(block, residual=res, pre=True, scale=0.25)
    keep = res.clone()
    h, out = gdr.gdr_residual_norm(block, res, None, residual_scale=0.25, residual_out=res)
    assert h is res and not torch.equal(res, keep)
    check(res, rh, 512)
    check(out, rout, 512)


def test_strides():
    """Views into packed projections, one element off 16 bytes, and heads before tokens."""
    big = _randn(9, 2 * 4 * 64 + 3, dtype=BF16)
    for shift in (0, 1, 3):
        a = big[:, shift:shift + 256].view(9, 4, 64)
        z = big[:, 256 + shift:512 + shift].view(9, 4, 64)
        out = torch.full((4, 9, 72), 5.0, dtype=BF16, device=DEV)
        o = out.transpose(0, 1)[..., :64]
        gdr.gdr_gate_norm(a, z, out=o)
        check(o, norm_ref(a, gate=z, act="silu", post=True)[1], 64)
        assert bool((out[..., 64:] == 5.0).all())


def test_hard_rows():
    """Zero rows, infinities, NaN and gates far out: as the formula has them, and only in their own rows."""
    a, z = _randn(6, 1, 128), _randn(6, 1, 128, seed=1)
    a[0] = 0
    a[1, 0, 5] = float("nan")
    a[2, 0, 7] = float("inf")
    z[3] = 1e4
    z[4] = -1e4
    got = gdr.gdr_gate_norm(a, z)
    ref = norm_ref(a, gate=z, act="silu", post=True)[1]
    assert not got[0].any() and bool(torch.isnan(got[1]).all())
    assert bool(torch.isnan(got[2, 0, 7])) and not got[2, 0, :7].any()
    for i in (3, 5):
        check(got[i], ref[i], 128)
    assert float(got[4].abs().max()) <= 1e-30
    h, out = gdr.gdr_residual_norm(a[:, 0], z[:, 0], None)
    assert bool(torch.isfinite(out[[0, 3, 4, 5]]).all())


def test_many_rows_and_nothing():
    a, z = _randn(70001, 1, 64, dtype=BF16), _randn(70001, 1, 64, dtype=BF16, seed=1)
    check(gdr.gdr_gate_norm(a, z), norm_ref(a, gate=z, act="silu", post=True)[1], 64)
    assert gdr.gdr_gate_norm(a[:0], z[:0]).shape == (0, 1, 64)


def test_refusals():
    a, z = _randn(4, 2, 64), _randn(4, 2, 64, seed=1)
    for call, kind in [(lambda: gdr.gdr_gate_norm(a.cpu(), z), ValueError), (lambda: gdr.gdr_gate_norm(a.half(), z), TypeError),
                       (lambda: gdr.gdr_gate_norm(a, z[:3]), ValueError), (lambda: gdr.gdr_gate_norm(a[0, 0], None), ValueError),
                       (lambda: gdr.gdr_gate_norm(a, z, torch.ones(63, device=DEV)), ValueError),
                       (lambda: gdr.gdr_gate_norm(a, z, torch.ones(64, device=DEV, dtype=BF16)), TypeError),
                       (lambda: gdr.gdr_gate_norm(a, z, activation="gelu"), ValueError),
                       (lambda: gdr.gdr_gate_norm(a, None, gate_first=True), ValueError),
                       (lambda: gdr.gdr_gate_norm(a, z, out=a[:2]), ValueError),
                       (lambda: gdr.gdr_gate_norm(a.transpose(1, 2), None), ValueError),
                       (lambda: gdr.gdr_residual_norm(a[:, 0], a, None), ValueError),
                       (lambda: gdr.gdr_residual_norm(a[:2, 0], a[:, 1], None), ValueError),
                       (lambda: gdr.gdr_residual_norm(None, a[:, 1], None, gate=a[:, 1]), ValueError),
                       (lambda: gdr.gdr_residual_norm(a[:, 0], a[:, 1], None, gate=a[0, 0, :5]), ValueError)]:
        with pytest.raises(kind):
            call()
    wide = torch.zeros(1, 16385, device=DEV)
    with pytest.raises(gdr.GdrError, match="16384"):
        gdr.gdr_gate_norm(wide, None)
    with pytest.raises(gdr.GdrError, match="eps"):
        gdr.gdr_gate_norm(a, z, eps=-1.0)
