"""The layer operators run on their tensors' device, whichever is current.
Device queries and launches are replaced by fakes: one GPU, or none, is enough."""
from __future__ import annotations

import contextlib
import ctypes

import pytest
import torch

import gated_deltanet_linear_gdr_gb300 as gdr
from gated_deltanet_linear_gdr_gb300 import _binding as B


class Devices:
    """A fake of the current device that notes what is launched where."""

    def __init__(self, monkeypatch, current=0):
        self.current, self.calls = current, []
        monkeypatch.setattr(B, "_current_device", lambda: self.current)
        monkeypatch.setattr(B, "_raw_stream", lambda i: 1000 + i)
        monkeypatch.setattr(B, "_stream", lambda d: 1000 + getattr(d, "index", d))
        monkeypatch.setattr(torch.cuda, "device", self.switch)

    @contextlib.contextmanager
    def switch(self, device):
        old, self.current = self.current, getattr(device, "index", device)
        yield
        self.current = old

    def entry(self, *args):
        self.calls.append((self.current, args[-1]))
        return 0


@pytest.mark.parametrize("device", [0, 1])
def test_direct_calls(monkeypatch, device):
    d = Devices(monkeypatch)
    assert B._launch(d.entry, b"", device) == 0
    assert d.calls == [(device, 1000 + device)] and d.current == 0


@pytest.mark.parametrize("device", [0, 1])
@pytest.mark.parametrize("stream", [None, 77])
def test_prepared_calls(monkeypatch, device, stream):
    d = Devices(monkeypatch)
    B.Prepared(d.entry, ctypes.c_int(), (), (), torch.device("cuda", device))(stream)
    assert d.calls == [(device, 1000 + device if stream is None else stream)] and d.current == 0


@pytest.mark.gpu
def test_every_entry_switches_to_its_tensors_device(monkeypatch):
    entered = []

    class Device(torch.cuda.device):
        def __init__(self, device):
            entered.append(getattr(device, "index", device))
            super().__init__(device)

    x = torch.randn(4, 64, device="cuda:0")
    y, z = gdr.gdr_gate_norm(x, x), gdr.gdr_residual_norm(x, x, None)[1]
    q, pool = x.view(4, 1, 64), torch.zeros(4, 1, 64, 64, device="cuda:0")
    rows = torch.arange(5, dtype=torch.int32, device="cuda:0")
    args = q, q, q, torch.ones(1, device="cuda:0"), pool, rows[:4], rows
    o = gdr.gdr_linattn_fwd(*args, max_row_len=1)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    assert torch.equal(gdr.gdr_gate_norm(x, x), y) and entered == [0]
    assert torch.equal(gdr.gdr_residual_norm(x, x, None)[1], z) and entered == [0, 0]
    pool.zero_()
    assert torch.equal(gdr.gdr_linattn_fwd(*args, max_row_len=1), o) and entered == [0, 0, 0]
    out = torch.empty_like(q)
    call = gdr.prepare_linattn_fwd(*args, out, max_row_len=1)
    pool.zero_()
    call()
    assert torch.equal(out, o) and entered == [0, 0, 0, 0]
