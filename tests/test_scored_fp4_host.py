"""CPU-only checks of routing by scores and of rows in 4 bits: what the C ABI
and the binding refuse, before any CUDA call."""
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


def scoring(abi, **kw):
    a = dict(score=0, groups=4, top_groups=2, group_top=2, renorm=1, scale=1.0, bias_rate=0.0, bias=None, bias_next=None)
    return abi.moe_scoring(*{**a, **kw}.values())


def test_the_struct_is_the_header_s(abi):
    src = open(os.path.join(ROOT, "include", "moe_route.h")).read()
    body = re.search(r"typedef struct moe_scoring \{(.*?)\} moe_scoring;", src, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n for line in body.split(";") for n in re.findall(r"\*?(\w+)\s*(?:,|$)", line.strip())]
    assert names == [n for n, _ in abi.moe_scoring._fields_]
    assert ctypes.sizeof(abi.moe_scoring) == 48
    for name in ("SIGMOID", "SOFTMAX"):
        assert int(re.search(rf"#define MOE_SCORE_{name} (\d+)", src).group(1)) == getattr(abi, f"MOE_SCORE_{name}")
    for K in (32, 512, 544, 4096, 1 << 20):
        assert abi.fp4_pitch(K) == (K + 511) // 512 * 16 >= K // 32


def test_gate_refusals(abi):
    bad, uns, small = abi.MOE_ERR_INVALID_ARG, abi.MOE_ERR_UNSUPPORTED, abi.MOE_ERR_WORKSPACE_TOO_SMALL

    def gate(S=None, logits=FAKE, T=10, E=16, k=4, idx=FAKE, gates=FAKE, counts=FAKE, aux=FAKE, ent=FAKE, ws=FAKE,
             n=1 << 20):
        return abi.lib().moe_gate_scored(logits, T, E, k, scoring(abi) if S is None else S, idx, gates, counts, aux,
                                         ent, ws, n, None)

    for S, want in ((dict(score=2), bad), (dict(score=-1), bad), (dict(groups=0), uns), (dict(groups=3), uns),
                    (dict(groups=32), uns), (dict(top_groups=0), uns), (dict(top_groups=5), uns),
                    (dict(groups=16, top_groups=3, group_top=1), uns),   # three experts for four slots
                    (dict(groups=16, top_groups=8, group_top=2), uns),   # the two best of one
                    (dict(group_top=0), uns), (dict(group_top=3), uns), (dict(scale=float("nan")), bad),
                    (dict(scale=float("inf")), bad), (dict(bias_rate=float("nan")), bad), (dict(bias=OFF.value), bad),
                    (dict(bias_next=OFF.value), bad)):
        assert gate(scoring(abi, **S)) == want, S
        assert abi.lib().moe_gate_scored_backward(FAKE, FAKE, FAKE, 10, 16, 4, scoring(abi, **S), FAKE, FAKE, 1 << 20,
                                                  None) == want, S
    for kw, want in ((dict(T=-1), bad), (dict(E=0), uns), (dict(E=300), uns), (dict(k=0), uns), (dict(k=17), uns),
                     (dict(T=1 << 29), uns), (dict(logits=None), bad), (dict(idx=None), bad), (dict(gates=None), bad),
                     (dict(counts=None), bad), (dict(ws=None), bad), (dict(logits=OFF), bad), (dict(idx=OFF), bad),
                     (dict(gates=OFF), bad), (dict(ws=OFF), bad), (dict(n=100), small)):
        assert gate(**kw) == want, kw
    assert abi.lib().moe_gate_scored(FAKE, 10, 16, 4, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 20, None) == bad

    def back(logits=FAKE, idx=FAKE, d=FAKE, T=10, E=16, k=4, out=FAKE, ws=FAKE, n=1 << 20):
        return abi.lib().moe_gate_scored_backward(logits, idx, d, T, E, k, scoring(abi), out, ws, n, None)

    for kw, want in ((dict(T=-1), bad), (dict(E=0), uns), (dict(k=17), uns), (dict(logits=None), bad),
                     (dict(idx=OFF), bad), (dict(d=None), bad), (dict(out=OFF), bad), (dict(ws=None), bad),
                     (dict(n=100), small)):
        assert back(**kw) == want, kw


def test_fp4_refusals(abi):
    bad, uns = abi.MOE_ERR_INVALID_ARG, abi.MOE_ERR_UNSUPPORTED
    L = abi.lib()
    G = ctypes.byref(abi.moe_rows(64, 4, 1 << 20, 1 << 20))
    for K in (0, 16, 40, (1 << 20) + 32, -32):
        assert L.moe_quantize_fp4(G, FAKE, K, FAKE, FAKE, None) == uns
        assert L.moe_dequantize_fp4(G, FAKE, FAKE, K, FAKE, None) == uns
    for a in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (OFF, FAKE, FAKE), (FAKE, OFF, FAKE),
              (FAKE, FAKE, OFF)):
        assert L.moe_quantize_fp4(G, a[0], 64, a[1], a[2], None) == bad
        assert L.moe_dequantize_fp4(G, a[0], a[1], 64, a[2], None) == bad
    for rows in (abi.moe_rows(-1, 4, 1 << 20, 1 << 20), abi.moe_rows(8, 4, None, 1 << 20),
                 abi.moe_rows(8, 4, 1 << 20, None)):
        assert L.moe_quantize_fp4(ctypes.byref(rows), FAKE, 64, FAKE, FAKE, None) == bad
    lay = abi.moe_layout(T=10, E=4, k=2, P=1, r_max=20, ws=1 << 20, offsets=1 << 20, dst_row=1 << 20)

    def dispatch(x=FAKE, T=10, H=64, codes=FAKE, scales=FAKE):
        return L.moe_dispatch_fp4(x, T, H, ctypes.byref(lay), codes, scales, None)

    for kw, want in ((dict(T=11), bad), (dict(H=0), uns), (dict(H=48), uns), (dict(H=(1 << 20) + 32), uns),
                     (dict(x=None), bad), (dict(codes=None), bad), (dict(scales=None), bad), (dict(x=OFF), bad),
                     (dict(codes=OFF), bad), (dict(scales=OFF), bad)):
        assert dispatch(**kw) == want, kw


def test_the_binding_refuses(abi):
    from combine_moe_gate_warp_gb300 import ExpertRows, Fp4Rows, RouteShape, Scoring
    with pytest.raises(ValueError, match="score"):
        Scoring("tanh")
    for kw in (dict(groups=0), dict(groups=257), dict(groups=(1 << 32) + 1), dict(top_groups=0), dict(group_top=-1)):
        with pytest.raises(ValueError, match="to 256"):
            Scoring(**kw)
    with pytest.raises(ValueError, match="CUDA"):
        abi.moe_gate_scored(torch.zeros(4, 8), 2, Scoring(), None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        abi.moe_gate_scored_backward(torch.zeros(4, 8), None, None, Scoring(), None, None)
    with pytest.raises(ValueError, match="CUDA"):
        abi.moe_dispatch_fp4(torch.zeros(4, 32), 4, 32, None, None, None)
    assert RouteShape(T=1, H=32, E=1, k=1, P=1).scoring is None
    r = ExpertRows(rows=4, device="cpu")
    u8 = dict(dtype=torch.uint8)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = Fp4Rows(torch.zeros(4, 32, **u8), torch.zeros(4, 16, **u8))
    for bad in (torch.zeros(4, 64), x[:3], x[:, :32], x.T.contiguous().T):
        with pytest.raises((ValueError, MemoryError)):
            r.quantize_fp4(bad, out=q)
    with pytest.raises(ValueError, match="multiple of 32"):
        r.quantize_fp4(torch.zeros(4, 48, dtype=torch.bfloat16))
    for bad in (Fp4Rows(q.codes[:3], q.scales), Fp4Rows(q.codes, q.scales[:, :8]), Fp4Rows(q.codes.int(), q.scales)):
        with pytest.raises(ValueError):
            r.dequantize_fp4(bad)
    with pytest.raises(TypeError):
        r.quantize_fp4(x, out=q.codes)
    with pytest.raises(ValueError, match="CUDA"):
        r.quantize_fp4(x, out=q)


def test_rows_of_another_kind_are_a_type_error(abi):
    from combine_moe_gate_warp_gb300 import ExpertRows
    r = ExpertRows(rows=4, device="cpu")
    for bad in (torch.zeros(4, 32, dtype=torch.uint8), None, (1, 2)):
        with pytest.raises(TypeError, match="Fp4Rows"):
            r.dequantize_fp4(bad)


def test_a_rate_without_a_place_for_the_moved_bias(abi):
    from combine_moe_gate_warp_gb300 import Scoring
    with pytest.raises(ValueError, match="bias_next"):
        Scoring().c(bias_rate=1e-3)
    with pytest.raises(ValueError, match="bias_next"):
        Scoring().c(bias=OFF.value, bias_rate=1e-3)
    assert Scoring().c(bias_next=64, bias_rate=0.5).bias_rate == 0.5 and Scoring().c().bias_rate == 0.0
