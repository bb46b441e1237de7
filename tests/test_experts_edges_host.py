"""CPU-only checks of the expert products' handles: streams, devices and
sizes that the binding has to get right before any CUDA call."""
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def experts():
    import combine_moe_gate_warp_gb300 as pkg
    pkg.build()
    from combine_moe_gate_warp_gb300 import experts
    return experts


def on_gpu(monkeypatch, rows, index=0, current=0x111):
    """The handle as it would be on cuda:`index`, with that current stream."""
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: index, raising=False)
    rows.device = torch.device("cuda", index)
    return rows


def test_a_plans_rows_are_on_its_stream(experts, monkeypatch):
    """dispatch and combine run on the stream that the plan was built with,
    whatever the current one is: so do the products on its rows."""
    off, ws = torch.zeros(5, dtype=torch.int32), torch.zeros(8192, dtype=torch.uint8)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x111, raising=False)
    for handle in (0xABC, 0):  # a side stream, and the default stream beside a side stream
        plan = SimpleNamespace(layout=SimpleNamespace(offsets=off), r_max=8, ws=ws,
                               stream=SimpleNamespace(cuda_stream=handle))
        assert on_gpu(monkeypatch, experts.ExpertRows.of(plan))._stream() == handle
    # without a stream of its own a handle follows the current one
    assert on_gpu(monkeypatch, experts.ExpertRows(off, rows=8, device="cpu"))._stream() == 0x111
