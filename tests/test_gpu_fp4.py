"""Rows in 4 bits on the GPU, bit by bit against their definition: every
border between two codes, every scale, rows outside the experts', odd sizes
and alignments, the dispatch with dropped slots, and the way back to bf16."""
import pytest
import torch

from combine_moe_gate_warp_gb300 import (ExpertRows, Fp4Rows, RoutePlan, RouteShape, abi, fp4_pitch,
                                         quantize_weights_fp4)
from scored_util import VALUES, decode_fp4, encode_fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import combine_moe_gate_warp_gb300 as pkg
    pkg.build()


def randn(*shape, seed, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * torch.exp(spread * torch.randn(*shape[:-1], 1, generator=g))
    return x.bfloat16()


def borders(power):
    """A row that meets every code, every halfway point and its neighbours in
    bf16, blocks led by 6 (times a power of two)."""
    mid = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    v = torch.tensor(VALUES + mid, dtype=torch.float32).bfloat16()
    bits = v.view(torch.int16)
    v = torch.cat((v, (bits + 1).view(torch.bfloat16)[1:], (bits - 1).view(torch.bfloat16)[1:])).float()
    v = v[v <= 6]
    v = torch.cat((v, -v))
    v = torch.cat((v, v.new_zeros((-len(v)) % 31))).reshape(-1, 31)
    return (torch.cat((v, v.new_full((v.shape[0], 1), 6.0)), 1).flatten() * 2.0 ** power).bfloat16()


@pytest.mark.parametrize("power", [-126, -60, -1, 0, 7, 100])
def test_every_border(power):
    row = borders(power)
    x = torch.stack((row, -row, row.flip(0)))
    check(x)


def check(x):
    rows, K = x.shape
    r = ExpertRows(rows=rows)
    q = r.quantize_fp4(x.cuda())
    codes, scales = encode_fp4(x)
    assert torch.equal(q.scales.cpu(), scales)
    assert torch.equal(q.codes.cpu(), codes)
    back = r.dequantize_fp4(q)
    want = decode_fp4(codes, scales)
    assert torch.equal(back.cpu().double().nan_to_num(9e9), want.nan_to_num(9e9)), "decoded"
    assert r.status() == 0
    return q


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (37, 544), (1, 8192), (130, 1056), (64, 5120), (5, 512),
                                    (4099, 96), (2, 16416)])
def test_rows(rows, K):
    check(randn(rows, K, seed=rows + K, spread=3.0))


def test_every_scale():
    """Blocks led by every exponent that bf16 has, and by both sides of 1.5."""
    lead = (torch.arange(1, 0x7F80, 61, dtype=torch.int32)).to(torch.int16).view(torch.bfloat16)
    lead = torch.cat((lead, (torch.arange(255) << 7 | 0x40).to(torch.int16).view(torch.bfloat16)[:255],
                      (torch.arange(255) << 7 | 0x41).to(torch.int16).view(torch.bfloat16)[:255]))
    lead = lead[lead.float() < 1.75 * 2.0 ** 127]
    body = randn(len(lead), 32, seed=1).float().clamp(-3, 3) / 3
    x = (body * lead.float()[:, None]).bfloat16()
    x[:, 5] = lead
    check(x)


def test_zeros_and_bad_values():
    x = randn(6, 128, seed=1)
    x[0] = 0
    x[1, :32] = -0.0
    x[2, 40] = float("nan")
    x[3, 70] = float("inf")
    x[4, 127] = float("-inf")
    q = check(x)
    assert q.scales[0, :4].tolist() == [0] * 4
    assert q.scales[2, :4].tolist()[1] == 255 and q.scales[3, 2] == 255 and q.scales[4, 3] == 255
    assert int((q.scales == 255).sum()) == 3


def test_alignment_and_larger_buffers():
    """Rows that start 16 bytes past a 32-byte boundary, and buffers that hold more rows."""
    rows, K = 21, 288
    flat = randn(1, rows * K + 8, seed=2)[0].cuda()
    x = flat[8:].view(rows, K)
    assert x.data_ptr() % 32 == 16
    r = ExpertRows(rows=rows - 4)
    out = Fp4Rows(torch.full((rows, K // 2), 0x5A, dtype=torch.uint8, device="cuda"),
                  torch.full((rows, fp4_pitch(K)), 0x5A, dtype=torch.uint8, device="cuda"))
    assert r.quantize_fp4(x, out=out) is out
    codes, scales = encode_fp4(x[:rows - 4])
    assert torch.equal(out.codes[:rows - 4].cpu(), codes) and torch.equal(out.scales[:rows - 4].cpu(), scales)
    assert bool((out.codes[rows - 4:] == 0x5A).all()) and bool((out.scales[rows - 4:] == 0x5A).all())
    back = torch.full((rows * K + 8,), 7.0, dtype=torch.bfloat16, device="cuda")[8:].view(rows, K)
    r.dequantize_fp4(out, out=back)
    assert torch.equal(back[:rows - 4].cpu().double(), decode_fp4(codes, scales)) and bool((back[rows - 4:] == 7).all())


def test_rows_of_experts_only():
    counts = [3, 0, 5, 1]
    off = torch.tensor([0, 3, 3, 8, 9], dtype=torch.int32, device="cuda")
    x = randn(14, 64, seed=3)
    x[9:] = float("nan")
    r = ExpertRows(off, rows=14)
    out = Fp4Rows(torch.full((14, 32), 0x5A, dtype=torch.uint8, device="cuda"),
                  torch.full((14, 16), 0x5A, dtype=torch.uint8, device="cuda"))
    r.quantize_fp4(x.cuda(), out=out)
    codes, scales = encode_fp4(x[:9])
    assert r.status() == 0 and sum(counts) == 9
    assert torch.equal(out.codes[:9].cpu(), codes) and torch.equal(out.scales[:9].cpu(), scales)
    assert bool((out.codes[9:] == 0x5A).all()) and bool((out.scales[9:] == 0x5A).all())
    # offsets that fall, pass the rows or are negative leave their expert empty
    for bad, mine in (([0, 3, 2, 8, 9], [0, 1, 2, 8]), ([0, 3, 3, 8, 15], [0, 1, 2, 3, 4, 5, 6, 7]),
                      ([-1, 3, 3, 8, 9], [3, 4, 5, 6, 7, 8])):
        r = ExpertRows(torch.tensor(bad, dtype=torch.int32, device="cuda"), rows=14)
        out.codes.fill_(0x5A)
        out.scales.fill_(0x5A)
        r.quantize_fp4(x.cuda(), out=out)
        assert r.status() == abi.MOE_ERR_DEVICE_DATA
        rest = [i for i in range(14) if i not in mine]
        assert torch.equal(out.codes[mine].cpu(), codes[mine]) and bool((out.codes[rest] == 0x5A).all())
        back = torch.full((14, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        r.dequantize_fp4(out, out=back)
        assert r.status() == abi.MOE_ERR_DEVICE_DATA
        assert bool((back[rest] == 7).all()) and torch.equal(back[mine].cpu().double(), decode_fp4(codes, scales)[mine])


def test_no_rows():
    r = ExpertRows(rows=0)
    q = r.quantize_fp4(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert q.codes.shape == (0, 32) and r.dequantize_fp4(q).shape == (0, 64) and r.status() == 0


def test_weights():
    w = randn(3, 24, 160, seed=4, spread=1.0)
    q = quantize_weights_fp4(w.cuda())
    assert q.codes.shape == (3, 24, 80) and q.scales.shape == (3, 24, 16)
    codes, scales = encode_fp4(w.reshape(72, 160))
    assert torch.equal(q.codes.cpu().reshape(72, 80), codes) and torch.equal(q.scales.cpu().reshape(72, 16), scales)


@pytest.mark.parametrize("T,H,E,k,cap", [(1, 32, 4, 1, 0), (300, 512, 8, 2, 0), (777, 544, 16, 8, 120), (64, 5120, 32, 4, 3),
                                         (5000, 96, 64, 2, 100)])
def test_dispatch(T, H, E, k, cap):
    plan = RoutePlan(RouteShape(T=T, H=H, E=E, k=k, P=1, capacity=cap, fp4=True))
    x = randn(T, H, seed=T, spread=2.0)
    plan.packed.fill_(0x5A)
    plan.scales.fill_(0x5A)
    plan.route(torch.randn(T, E, generator=torch.Generator().manual_seed(5)).cuda())
    plan.dispatch(x.cuda())
    assert plan.status() == 0
    R = int(plan.layout.offsets[E])
    codes, scales = encode_fp4(x)
    src = (plan.layout.src_pos[:R] // k).cpu().long()
    assert torch.equal(plan.packed[:R].cpu(), codes[src]) and torch.equal(plan.scales[:R].cpu(), scales[src])
    assert bool((plan.packed[R:] == 0x5A).all()) and bool((plan.scales[R:] == 0x5A).all())
    back = ExpertRows.of(plan).dequantize_fp4(Fp4Rows(plan.packed, plan.scales))
    assert torch.equal(back[:R].cpu().double(), decode_fp4(codes, scales)[src])


def test_the_dispatch_call():
    T, H = 20, 96
    plan = RoutePlan(RouteShape(T=T, H=H, E=4, k=2, P=1))
    plan.route(torch.randn(T, 4, generator=torch.Generator().manual_seed(5)).cuda())
    x = randn(T, H, seed=1).cuda()
    codes = torch.zeros(2 * T, H // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2 * T, fp4_pitch(H), dtype=torch.uint8, device="cuda")
    abi.moe_dispatch_fp4(x, T, H, plan.layout, codes, scales)
    want = encode_fp4(x)
    src = (plan.layout.src_pos // 2).cpu().long()
    assert plan.status() == 0 and torch.equal(codes.cpu(), want[0][src]) and torch.equal(scales.cpu(), want[1][src])
    for args in ((x[:5], T, H, plan.layout, codes, scales), (x, T, H, plan.layout, codes[:9], scales),
                 (x, T, H, plan.layout, codes, scales[:, :8]), (x.float(), T, H, plan.layout, codes, scales)):
        with pytest.raises(ValueError):
            abi.moe_dispatch_fp4(*args)
    with pytest.raises(ValueError, match="two transports"):
        RoutePlan(RouteShape(T=T, H=H, E=4, k=2, P=1, fp4=True, fp8=1))
    with pytest.raises(ValueError, match="multiple of 32"):
        RoutePlan(RouteShape(T=T, H=48, E=4, k=2, P=1, fp4=True))


def test_dispatch_of_a_bad_layout():
    plan = RoutePlan(RouteShape(T=40, H=64, E=4, k=2, P=1, fp4=True))
    plan.route(torch.randn(40, 4, generator=torch.Generator().manual_seed(5)).cuda())
    x = randn(40, 64, seed=1)
    plan.layout.dst_row[7] = 80  # past the last row
    plan.layout.dst_row[9] = -1
    plan.packed.fill_(0x5A)
    plan.dispatch(x.cuda())
    assert plan.status() == abi.MOE_ERR_DEVICE_DATA
    src = plan.layout.src_pos[:80].cpu().long()
    good = (src != 7) & (src != 9)
    assert torch.equal(plan.packed[:80].cpu()[good], encode_fp4(x)[0][src // 2][good])
    assert bool((plan.packed[:80].cpu()[~good] == 0x5A).all())


def test_streams_and_graphs():
    st = torch.cuda.Stream()
    plan = RoutePlan(RouteShape(T=500, H=256, E=8, k=2, P=1, fp4=True), stream=st)
    rows = ExpertRows.of(plan)
    logits, x = torch.randn(500, 8, device="cuda"), randn(500, 256, seed=1).cuda()
    back = torch.empty(1000, 256, dtype=torch.bfloat16, device="cuda")

    def calls():
        plan.route(logits)
        plan.dispatch(x)
        rows.dequantize_fp4(Fp4Rows(plan.packed, plan.scales), out=back)

    torch.cuda.synchronize()
    calls()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        calls()
    for seed in (2, 3):
        x.copy_(randn(500, 256, seed=seed))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graph.replay()
        assert plan.status() == 0
        src = (plan.layout.src_pos // 2).cpu().long()
        assert torch.equal(back.cpu().double(), decode_fp4(*encode_fp4(x))[src])
