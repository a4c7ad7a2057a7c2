"""Corners of the layer operators that a call meets seldom."""
from __future__ import annotations

import ctypes

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from gated_deltanet_linear_gdr_gb300 import _binding as B
from tests.layer_helpers import U16, U32, check_linattn, linattn_ref, norm_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def _randn(*shape, dtype=F32, seed=0, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


@pytest.mark.parametrize("K", [64, 128])
@pytest.mark.parametrize("pool", [BF16, F32])
def test_units_dealt_by_load(K, pool):
    """The first chunk's tokens arrive right behind the deal of the units, and nothing of the deal may lie where they
    do: the first tokens weigh most here (a state that never fades, keys of one sign), and calls repeat bit for bit."""
    lens, nv = [513, 640, 90, 700, 515], 48
    T = sum(lens)
    q, k = _randn(T, nv // 2, K, dtype=BF16), _randn(T, nv // 2, K, dtype=BF16, seed=1).abs()
    v, lam = _randn(T, nv, 64, dtype=BF16, seed=2), torch.ones(nv, device=DEV)
    off = torch.tensor([sum(lens[:i]) for i in range(6)], dtype=torch.int32, device=DEV)
    slot = torch.tensor([4, 0, 2, 1, 3], dtype=torch.int32, device=DEV)
    start = _randn(5, nv, K, 64, dtype=pool, seed=3)
    assert gdr.gdr_linattn_workspace_bytes(q, k, v, lam, start, slot, off, max_row_len=700) == 0
    first = None
    for _ in range(30):
        state = start.clone()
        out = gdr.gdr_linattn_fwd(q, k, v, lam, state, slot, off, max_row_len=700)
        if first is None:
            first = out, state
            check_linattn(out, state, linattn_ref(q, k, v, lam, start, slot, off), 700, True)
        assert torch.equal(out, first[0]) and torch.equal(state, first[1])
    assert gdr.gdr_get_status() == 0


@pytest.mark.parametrize("heads,D", [(3, 64), (2, 128), (1, 1024), (1, 4096), (2, 66), (1, 2047)])
@pytest.mark.parametrize("x_dtype,h_dtype", [(BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("with_out", [False, True])
def test_residual_out_without_a_residual(heads, D, x_dtype, h_dtype, post, with_out):
    """The C entry's residual_out is h, and h is u where there is no residual; rows past the last stay as they were."""
    T = 5
    x, gate, w = _randn(T, heads, D, dtype=x_dtype), _randn(T, heads, D, dtype=x_dtype, seed=1), 1 + 0.1 * _randn(D, seed=2)
    h = torch.full((T + 1, heads, D), 7.0, dtype=h_dtype, device=DEV)
    out = torch.full((T + 1, heads, D), 7.0, dtype=BF16, device=DEV)
    a = B.gdr_norm_args()
    types = {BF16: B.GDR_BF16, F32: B.GDR_F32}
    for n, value in dict(tokens=T, heads=heads, D=D, eps=1e-6, residual_scale=0.3, has_post_norm=post, has_pre_norm=True,
                         activation=1, x_dtype=types[x_dtype], gate_dtype=types[x_dtype], residual_dtype=types[h_dtype],
                         out_dtype=B.GDR_BF16, x=x.data_ptr(), gate=gate.data_ptr(), gate_elem_stride=1,
                         residual_out=h.data_ptr(), post_weight=w.data_ptr(), pre_weight=w.data_ptr()).items():
        setattr(a, n, value)
    for n in ("x", "gate", "residual_out") + (("out",) if with_out else ()):
        setattr(a, n + "_seq_stride", heads * D)
        setattr(a, n + "_head_stride", D)
    if with_out:
        a.out = out.data_ptr()
    assert B.load_library().gdr_block_norm(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == B.GDR_OK
    rh, rout = norm_ref(x, gate=gate, act="silu", post=post, post_w=w, pre=True, pre_w=w)
    for got, want in [(h, rh)] + ([(out, rout)] if with_out else []):
        rms = want.pow(2).mean(-1, keepdim=True).sqrt()  # a row's statistics: as in the tests of the norms
        tol = 32 * (D + 40) * U32 * (want.abs() + rms) + (U16 if got.dtype == BF16 else 0.0) * want.abs() + 1e-30
        assert bool(((got[:T].double() - want).abs() <= tol).all())
        assert bool((got[T:] == 7.0).all())
    if not with_out:
        assert bool((out == 7.0).all())


def _token(heads, dim, T, seed):
    """One token's values for all T, by a stride of 0."""
    return _randn(1, heads, dim, dtype=BF16, seed=seed).expand(T, heads, dim)


def _skipped(T, K, V, out, slot, max_row_len, flags):
    """A call of one row that is skipped: its output has to be cleared."""
    off = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    pool = _randn(1, 1, K, V, dtype=BF16)
    keep = pool.clone()
    gdr.gdr_get_status(clear=True)
    args = _token(1, K, T, 1), _token(1, K, T, 2), _token(1, V, T, 3), torch.ones(1, device=DEV), pool
    gdr.gdr_linattn_fwd(*args, torch.tensor([slot], dtype=torch.int32, device=DEV), off, out, max_row_len=max_row_len)
    assert gdr.status_names(gdr.gdr_get_status()) == flags
    assert torch.equal(pool, keep)


def test_a_skipped_row_of_more_than_2_to_the_31_outputs():
    T = 2 ** 24 + 5
    out = torch.full((T + 1, 1, 128), 7.0, dtype=BF16, device=DEV)
    _skipped(T, 128, 128, out[:T], -1, 0, [])
    assert not bool(out[:T].any()) and bool((out[T] == 7.0).all())


def test_a_row_far_past_its_bound():
    """The short form, whose rows are told apart by their length: zeros of 2^31 + 48 vectors, on top of one another."""
    T = 2 ** 27 + 3
    buf = torch.full((T * 8 + 136,), 7.0, dtype=BF16, device=DEV)
    _skipped(T, 64, 128, buf.as_strided((T, 1, 128), (8, 128, 1)), 0, 16, ["ROW_TOO_LONG"])
    end = (T - 1) * 8 + 128
    assert not bool(buf[:end].any()) and bool((buf[end:] == 7.0).all())


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("D,form", [(64, "gate"), (1024, "gate"), (66, "gate"), (2047, "gate"), (64, "row"), (1024, "residual"),
                                    (2047, "residual")])
def test_activations_in_float32(act, D, form):
    """Values of 1 and -1, whose norm is themselves, so that what a float32 output is off by is the activation's error:
    two units of the exponential, the sum's, the quotient's and the product's rounding, under 2^-21 altogether."""
    T = 64
    x = torch.where(_randn(T, D) > 0, 1.0, -1.0)
    g = torch.linspace(-80.0, 80.0, T * (1 if form == "row" else D), device=DEV).view(T, -1)
    if form == "residual":
        out = gdr.gdr_residual_norm(x, torch.zeros(T, D, device=DEV), None, gate=g, activation=act, out_dtype=BF16)[0]
    else:
        out = gdr.gdr_gate_norm(x, g, activation=act, eps=0.0)
    assert out.dtype == F32
    gd = g.double()
    want = x.double() * (gd / (1 + torch.exp(-gd)) if act == "silu" else 1 / (1 + torch.exp(-gd)))
    err = float(((out.double() - want).abs() / want.abs()).nan_to_num(0.0).max())
    assert err <= 2.0 ** -21, f"{err * 2 ** 21:.3g} x the bound"


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_activations_far_out(dtype):
    """Gates of infinity, NaN and past where the exponential overflows, as the formula has them."""
    inf = float("inf")
    g = torch.tensor([inf, -inf, float("nan"), 1e30, -1e30, 100.0, -100.0, 0.0], device=DEV).to(dtype)[:, None].expand(8, 64)
    x = torch.ones(8, 64, dtype=dtype, device=DEV)
    got = gdr.gdr_gate_norm(x, g.contiguous(), activation="sigmoid", eps=0.0)[:, 0].tolist()
    assert got[:2] == [1.0, 0.0] and got[2] != got[2] and got[3:6] == [1.0, 0.0, 1.0] and abs(got[6]) <= 1e-30 and got[7] == 0.5
    got = gdr.gdr_gate_norm(x, g.contiguous(), activation="silu", eps=0.0)[:, 0].double().tolist()
    assert got[0] == inf and got[1] != got[1] and got[2] != got[2] and got[3] >= 9e29 and got[4] == 0.0
    assert got[5] == 100.0 and abs(got[6]) <= 1e-30 and got[7] == 0.0
