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


def on_gpu(monkeypatch, rows, index=0, current=0x111, device=0):
    """The handle as it would be on cuda:`index`, with that current stream and device."""
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: device, raising=False)
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


def test_another_current_device_is_refused(experts, monkeypatch):
    """A launch goes to the current device: rows on another one are refused
    before the library is called, by the products and by status()."""
    def called(*args):
        raise AssertionError("the library was called")

    off = torch.tensor([0, 3, 8], dtype=torch.int32)
    for stream in (None, SimpleNamespace(cuda_stream=0xABC)):
        r = experts.ExpertRows(off, rows=8, device="cpu")
        r._lib = SimpleNamespace(moe_expert_linear=called, moe_expert_dgrad=called, moe_expert_wgrad=called,
                                 moe_act_backward=called)
        r.stream = stream
        on_gpu(monkeypatch, r, index=1, device=0)
        monkeypatch.setattr(experts, "_check", lambda *a: 16)
        monkeypatch.setattr(experts, "_check_rows", lambda *a: 16)
        monkeypatch.setattr(experts.ExpertRows, "_new", lambda self, shape, dtype=None: torch.empty(0))
        monkeypatch.setattr(experts.abi, "moe_get_status", called)
        bf = dict(dtype=torch.bfloat16)
        x, dy, w = torch.zeros(8, 32, **bf), torch.zeros(8, 64, **bf), torch.zeros(2, 64, 32, **bf)
        saved = experts.SavedLayer.empty(8, 64, "cpu")
        for call in (lambda: r.linear(x, w), lambda: r.dgrad(dy, w), lambda: r.wgrad(dy, x),
                     lambda: r.act_backward(dy, act="gelu", saved=saved), r.status):
            with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
                call()


def test_sizes_past_32_bits_are_refused(experts):
    """ctypes passes an integer's low 32 bits: sizes past them are refused
    before they could be taken for small ones."""
    off = torch.zeros(3, dtype=torch.int32)
    for rows in ((1 << 32) + 8, 1 << 31, -1):
        with pytest.raises(ValueError, match="rows"):
            experts.ExpertRows(off, rows=rows, device="cpu")
    assert experts.ExpertRows(off, rows=(1 << 31) - 1, device="cpu")._c.rows == (1 << 31) - 1
    r = experts.ExpertRows(off, rows=0, device="cpu")
    far, bf = (1 << 32) + 64, dict(dtype=torch.bfloat16)
    wide, x = torch.empty(0, far, **bf), torch.empty(0, 64, **bf)
    for w in (torch.empty(2, 0, far, **bf), torch.empty(2, far, 0, **bf)):
        for call in (r.linear, r.dgrad):
            with pytest.raises(ValueError, match="columns are too many"):
                call(wide, w)
    saved = experts.SavedLayer(torch.empty(0, far, dtype=torch.uint8), torch.empty(0, far // 32, dtype=torch.uint8))
    for call in (lambda: r.wgrad(wide, x, out=x), lambda: r.wgrad(x, wide, out=x),
                 lambda: r.act_backward(wide, act="silu", saved=saved, out=x)):
        with pytest.raises(ValueError, match="columns are too many"):
            call()


def test_cut_refusals(experts):
    L, abi = experts.abi.lib(), experts.abi
    import ctypes
    out = (ctypes.c_int32 * 3)(9, 9, 9)
    bad, uns = abi.MOE_ERR_INVALID_ARG, abi.MOE_ERR_UNSUPPORTED
    for args, want in (((3, 0, 8, 1, 64, 64, out), bad), ((-1, 0, 8, 1, 64, 64, out), bad),
                       ((0, 0, -1, 1, 64, 64, out), bad), ((0, 0, 8, 1, 64, 64, None), bad),
                       ((1, 1, 8, 1, 64, 64, out), bad), ((0, 0, 8, 0, 64, 64, out), uns),
                       ((0, 0, 8, 257, 64, 64, out), uns), ((2, 0, 1 << 30, 1, 64, 64, out), uns),
                       ((0, 0, 8, 1, 60, 64, out), uns), ((0, 0, 8, 1, 64, (1 << 20) + 8, out), uns)):
        assert L.moe_expert_cut(*args) == want, args
    r = experts.ExpertRows(torch.zeros(3, dtype=torch.int32), rows=0, device="cpu")
    assert r.cut("linear", 64, 64) == (0, 0, 0)  # nothing to cut
    with pytest.raises(ValueError):
        r.cut("product", 64, 64)
