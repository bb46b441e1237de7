"""CPU-only checks of the expert products' entry points: what the C ABI and
the binding refuse, before any CUDA call."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(1 << 20)
OFF = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def abi():
    import combine_moe_gate_warp_gb300 as pkg
    pkg.build()
    from combine_moe_gate_warp_gb300 import abi
    return abi


def rows(abi, n=64, E=4, offsets=1 << 20, ws=1 << 20):
    return ctypes.byref(abi.moe_rows(n, E, offsets, ws))


def linear(abi, G, **kw):
    a = dict(x=FAKE, xs=None, K=64, w=FAKE, ws=None, N=64, bias=None, act=0, res=None, y=FAKE, sv=None, ss=None)
    a.update(kw)
    return abi.lib().moe_expert_linear(G, *a.values(), None)


def test_rows_are_checked(abi):
    for G, want in ((None, abi.MOE_ERR_INVALID_ARG), (rows(abi, n=-1), abi.MOE_ERR_INVALID_ARG),
                    (rows(abi, ws=None), abi.MOE_ERR_INVALID_ARG), (rows(abi, ws=4), abi.MOE_ERR_INVALID_ARG),
                    (rows(abi, E=0), abi.MOE_ERR_UNSUPPORTED), (rows(abi, E=257), abi.MOE_ERR_UNSUPPORTED),
                    (rows(abi, n=1 << 30), abi.MOE_ERR_UNSUPPORTED),
                    (rows(abi, offsets=None), abi.MOE_ERR_INVALID_ARG)):  # one group: E == 1
        assert linear(abi, G) == want
        assert abi.lib().moe_expert_dgrad(G, FAKE, 64, FAKE, 64, 0, None, None, FAKE, None, None) == want
        assert abi.lib().moe_expert_wgrad(G, FAKE, 64, FAKE, 64, FAKE, None, 0, None) == want
        assert abi.lib().moe_act_backward(G, FAKE, 64, 1, FAKE, FAKE, FAKE, None, None) == want


def test_linear_refusals(abi):
    G = rows(abi)
    bad, uns = abi.MOE_ERR_INVALID_ARG, abi.MOE_ERR_UNSUPPORTED
    for kw, want in ((dict(K=0), uns), (dict(K=60), uns), (dict(N=4), uns), (dict(N=(1 << 20) + 8), uns),
                     (dict(act=4), bad), (dict(act=-1), bad), (dict(N=72, act=3), uns),
                     (dict(xs=FAKE), bad), (dict(ws=FAKE), bad), (dict(xs=FAKE, ws=FAKE, K=72), uns),
                     (dict(sv=FAKE), bad), (dict(ss=FAKE), bad), (dict(sv=FAKE, ss=FAKE, N=40), uns),
                     (dict(sv=FAKE, ss=FAKE, N=96, act=3), uns), (dict(x=None), bad), (dict(w=None), bad),
                     (dict(y=None), bad), (dict(x=OFF), bad), (dict(w=OFF), bad), (dict(bias=OFF), bad),
                     (dict(res=OFF), bad), (dict(y=OFF), bad), (dict(sv=OFF, ss=FAKE), bad)):
        assert linear(abi, G, **kw) == want, kw


def test_gradient_refusals(abi):
    G, L = rows(abi), abi.lib()
    bad, uns = abi.MOE_ERR_INVALID_ARG, abi.MOE_ERR_UNSUPPORTED

    def dgrad(dy=FAKE, N=64, w=FAKE, K=64, act=0, sv=None, ss=None, dx=FAKE, a=None):
        return L.moe_expert_dgrad(G, dy, N, w, K, act, sv, ss, dx, a, None)

    assert dgrad(N=12) == uns and dgrad(K=0) == uns and dgrad(act=9) == bad
    assert dgrad(dy=None) == bad and dgrad(w=None) == bad and dgrad(dx=OFF) == bad
    assert dgrad(sv=FAKE, ss=FAKE) == bad and dgrad(a=FAKE) == bad        # no activation: nothing saved
    assert dgrad(act=1) == bad and dgrad(act=1, sv=FAKE) == bad           # an activation: saved
    assert dgrad(act=1, sv=FAKE, ss=FAKE, K=40) == uns and dgrad(act=3, sv=FAKE, ss=FAKE, K=16) == uns

    def wgrad(dy=FAKE, N=64, x=FAKE, K=64, dw=FAKE, db=None):
        return L.moe_expert_wgrad(G, dy, N, x, K, dw, db, 0, None)

    assert wgrad(N=4) == uns and wgrad(K=20) == uns and wgrad(dw=None) == bad and wgrad(x=None) == bad
    assert wgrad(db=OFF) == bad and wgrad(dy=OFF) == bad

    def act(dy=FAKE, N=64, a=1, sv=FAKE, ss=FAKE, du=FAKE, out=None):
        return L.moe_act_backward(G, dy, N, a, sv, ss, du, out, None)

    assert act(a=0) == bad and act(a=4) == bad and act(N=48) == uns and act(N=32, a=3) == uns
    assert act(sv=None) == bad and act(du=None) == bad and act(dy=OFF) == bad and act(out=OFF) == bad


def test_no_rows_need_no_gpu(abi):
    """Nothing to do is not an error, and launches nothing."""
    G = rows(abi, n=0)
    assert linear(abi, G, x=None, y=None) == abi.MOE_OK
    assert abi.lib().moe_expert_dgrad(G, None, 64, FAKE, 64, 0, None, None, None, None, None) == abi.MOE_OK
    assert abi.lib().moe_act_backward(G, None, 64, 1, None, None, None, None, None) == abi.MOE_OK


def test_struct_and_constants_match_the_header(abi):
    hdr = open(os.path.join(ROOT, "include", "moe_experts.h")).read()
    body = re.sub(r"/\*.*?\*/", "", hdr[hdr.index("typedef struct moe_rows {"):hdr.index("} moe_rows;")], flags=re.S)
    assert [f for f, _ in abi.moe_rows._fields_] == re.findall(r"\*?(\w+)(?:,|;)", body)
    for name in ("NONE", "SILU", "GELU", "SWIGLU"):
        assert int(re.search(rf"#define MOE_ACT_{name} (\d)", hdr).group(1)) == getattr(abi, f"MOE_ACT_{name}")


def test_binding_refusals(abi):
    """The binding checks types, shapes and devices of what it is given; on a
    CPU-only machine the rows themselves live on the CPU and nothing is run."""
    from combine_moe_gate_warp_gb300 import ExpertFFN, ExpertRows, SavedLayer
    off = torch.tensor([0, 3, 3, 7], dtype=torch.int32)
    r = ExpertRows(off, rows=8, device="cpu")
    bf = dict(dtype=torch.bfloat16)
    x, w = torch.zeros(8, 32, **bf), torch.zeros(3, 64, 32, **bf)
    for kw, err, what in ((dict(x=x[:7]), ValueError, "x: expected shape"), (dict(x=x.float()), ValueError, "x: exp"),
                          (dict(x=torch.zeros(32, 8, **bf).T), ValueError, "contiguous"), (dict(x=3), TypeError, "x"),
                          (dict(w=w[0]), ValueError, r"\[E, N, K\]"), (dict(w=w[:2]), ValueError, "2 experts"),
                          (dict(act="relu"), ValueError, "swiglu"), (dict(bias=w), ValueError, "bias"),
                          (dict(residual=x), ValueError, "residual"), (dict(out=x), ValueError, "out"),
                          (dict(x_scales=torch.zeros(8, 2)), ValueError, "go together"),
                          (dict(saved=SavedLayer.empty(8, 96, "cpu")), ValueError, "saved.codes")):
        a = dict(x=x, w=w)
        a.update(kw)
        with pytest.raises(err, match=what):
            r.linear(a.pop("x"), a.pop("w"), **a)
    with pytest.raises(ValueError, match="CUDA device"):
        r.linear(x, w)
    dy = torch.zeros(8, 64, **bf)
    for call, what in ((lambda: r.dgrad(x, w), "dy"), (lambda: r.dgrad(dy, w, act="silu"), "go together"),
                       (lambda: r.dgrad(dy, w, a=x), "saved layer"),
                       (lambda: r.wgrad(dy, x, dtype=torch.float16), "bfloat16 or float32"),
                       (lambda: r.wgrad(dy[:3], x), "dy"), (lambda: r.wgrad(dy, x, out=w.float()), "out"),
                       (lambda: r.act_backward(dy, act="none", saved=SavedLayer.empty(8, 64, "cpu")), "none"),
                       (lambda: r.linear_backward(dy, x, w, act="gelu"), "go together"),
                       (lambda: SavedLayer.empty(8, 40, "cpu"), "multiple of 32"),
                       (lambda: ExpertFFN(r, w, torch.zeros(3, 32, 48, **bf)), "fit together"),
                       (lambda: ExpertFFN(r, w, torch.zeros(3, 32, 64, **bf), act="none"), "activation"),
                       (lambda: ExpertRows(off.long(), rows=8, device="cpu"), "int32"),
                       (lambda: ExpertRows(off[:1], rows=8, device="cpu"), "E in 1"),
                       (lambda: ExpertRows(off, rows=-1, device="cpu"), "rows"),
                       (lambda: ExpertRows(off, rows=8, device="cpu", ws=torch.zeros(100)), "workspace")):
        with pytest.raises(ValueError, match=what):
            call()


def test_quantize_weights():
    """e4m3 weights: the largest of a column is 448 * scale, every value is
    within half a step (2^-4 of it, or 2^-10 of the scale), zeros stay zeros."""
    from combine_moe_gate_warp_gb300 import quantize_weights
    w = torch.randn(3, 24, 32, generator=torch.Generator().manual_seed(1)).bfloat16()
    w[1, 5] = 0
    codes, scales = quantize_weights(w)
    assert codes.shape == w.shape and scales.shape == (3, 24, 2)
    v = codes.view(torch.float8_e4m3fn).double() * scales[..., :1].double()
    assert bool(((v - w.double()).abs() <= 2.0 ** -4 * w.double().abs() * (1 + 2.0 ** -20)
                 + 2.0 ** -10 * scales[..., :1].double()).all())
    assert bool((v[1, 5] == 0).all()) and scales[1, 5, 0] == 1 and scales[1, 5, 1] == 0
    assert torch.allclose(scales[..., 1].double(), v.sum(2), rtol=2.0 ** -23, atol=0)
    one, two = quantize_weights(w[0])
    assert torch.equal(one, codes[0]) and torch.equal(two, scales[0])
