"""Every C call of a Buffer is made with the buffer's device current (the library launches on the current one)."""
import contextlib

import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    from combine_moe_layout_02_amd.build import LIB
    import os
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    import combine_moe_layout_02_amd
    return combine_moe_layout_02_amd


class _Library:
    """Notes the calls it gets, and which device was current at each."""

    def __init__(self):
        self.current, self.calls = torch.device("cuda", 0), []

    @contextlib.contextmanager
    def on(self, device):
        before, self.current = self.current, device
        yield
        self.current = before

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.current))
            return 0
        return call


@pytest.mark.parametrize("kw", [{}, dict(fp8=True), dict(mx4=True), dict(balance_slots=2), dict(mx4=True, balance_slots=2)],
                         ids=["bf16", "fp8", "mx4", "balanced", "mx4 balanced"])
def test_calls_are_made_on_the_buffers_device(moe, monkeypatch, kw):
    buf = moe.Buffer(S=4, H=128, K=2, E=8, R=2, device="cpu", **kw)
    buf.device, buf._index = torch.device("cuda", 3), 3
    lib = _Library()
    monkeypatch.setattr(moe, "_lib", lib)
    monkeypatch.setattr(torch.cuda, "device", lib.on)
    monkeypatch.setattr(moe, "_raw_current_device", lambda: lib.current.index)
    monkeypatch.setattr(moe, "_stream", lambda stream, device: 0)
    hidden, w, idx = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 2), torch.zeros(4, 2, dtype=torch.int32)
    buf.layout_call(idx, check=False)
    buf.dispatch_call(hidden, idx, w, check=False)
    buf.layout_dispatch_call(hidden, idx, w, check=False)
    buf.combine_call(torch.zeros(8, 128, dtype=torch.bfloat16), w, check=False)
    if not buf.mx4:
        buf.zero_padding_call()
    assert len(lib.calls) >= 4
    assert all(device == buf.device for _, device in lib.calls), lib.calls
    assert lib.current.index == 0
