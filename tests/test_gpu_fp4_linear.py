"""The expert products from rows and weights in 4 bits against the same
products in 64 bits: single rows and long groups, tails of every axis, every
activation, scales of every size, blocks that hold a NaN, rows outside the
groups, and the path from the dispatch through two layers to the combine."""
import pytest
import torch

from combine_moe_gate_warp_gb300 import (ExpertRows, Fp4Rows, RoutePlan, RouteShape, Scoring, abi, fp4_pitch,
                                         quantize_weights_fp4)
from expert_util import BF16, act64, act_error, assert_near, normal, offsets_of, spans, sum_error
from scored_util import backward_error, decode_fp4, encode_fp4, gates64

pytestmark = pytest.mark.gpu

COUNTS = [0, 1, 15, 33, 0, 130, 257, 16, 0]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import combine_moe_gate_warp_gb300 as pkg
    pkg.build()


def fp4(*shape, seed, std=1.0, spread=1.0):
    """Random rows in 4 bits [.., K], the scales of their blocks apart by `spread` octaves."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * std
    x = x * torch.exp2(torch.round(spread * torch.randn(*shape[:-1], shape[-1] // 32, generator=g))).repeat_interleave(32, -1)
    codes, scales = encode_fp4(x.bfloat16().reshape(-1, shape[-1]))
    return Fp4Rows(codes.view(*shape[:-1], -1).cuda(), scales.view(*shape[:-1], -1).cuda())


def values(q):
    flat = decode_fp4(q.codes.reshape(-1, q.codes.shape[-1]), q.scales.reshape(-1, q.scales.shape[-1]))
    return flat.view(*q.codes.shape[:-1], -1).cuda()


def linear64(x, w, counts, bias=None):
    us, es = [], []
    for e, lo, hi in spans(counts):
        u, m = x[lo:hi] @ w[e].T, x[lo:hi].abs() @ w[e].abs().T
        if bias is not None:
            u, m = u + bias[e].double(), m + bias[e].double().abs()
        us.append(u)
        es.append(sum_error(x.shape[1], m))
    return torch.cat(us), torch.cat(es)


def padded(q, rows):
    """The rows in buffers that hold more, of any bits."""
    R = q.codes.shape[0]
    codes = torch.full((rows, q.codes.shape[1]), 0x77, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, q.scales.shape[1]), 0xFF, dtype=torch.uint8, device="cuda")
    codes[:R], scales[:R] = q.codes, q.scales
    return Fp4Rows(codes, scales)


def run(counts, rows, K, N, act="none", bias=False, residual=False, seed=1, spread=1.0):
    R, E = sum(counts), len(counts)
    x, w = fp4(R, K, seed=seed, spread=spread), fp4(E, N, K, seed=seed + 1, std=K ** -0.5, spread=spread)
    b = normal(E, N, seed=5) if bias else None
    cols = N // 2 if act == "swiglu" else N
    res = normal(R, cols, seed=6) if residual else None
    r = ExpertRows(offsets_of(counts), rows=rows)
    out = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    more = None
    if res is not None:
        more = torch.full((rows, cols), float("nan"), dtype=torch.bfloat16, device="cuda")
        more[:R] = res
    assert r.linear_fp4(padded(x, rows), w, bias=b, act=act, residual=more, out=out) is out
    assert r.status() == 0
    u, e = linear64(values(x), values(w), counts, b)
    want, err = act64(u, act), act_error(u, e, act)
    if residual:
        want = want + res.double()
    err = err + 2.0 ** -23 * want.abs()
    assert_near(out[:R], want, err + BF16 * (want.abs() + err), "y")
    assert bool((out[R:] == 7.0).all()), "rows past the last expert's were written"


@pytest.mark.parametrize("K,N", [(256, 128), (32, 8), (64, 264), (544, 96), (1056, 520), (2048, 136)])
@pytest.mark.parametrize("mean", [8, 300, 9000])
def test_linear(mean, K, N):
    counts = COUNTS if mean != 8 else [0, 1, 7, 0, 20, 33, 3]
    run(counts, max(sum(counts), mean * len(counts)), K, N)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("mean", [8, 300, 9000])
@pytest.mark.parametrize("bias,residual", [(True, False), (True, True), (False, True)])
def test_epilogues(act, mean, bias, residual):
    counts = COUNTS if mean != 8 else [3, 0, 1, 40]
    run(counts, max(sum(counts), mean * len(counts)), 288, 448, act, bias, residual)


CUTS = [((1, 32, 1), 7, 3, 96, 288), ((1, 32, 2), 7, 3, 1184, 4128), ((1, 32, 4), 7, 3, 96, 4128),
        ((1, 32, 8), 7, 3, 96, 8224), ((1, 64, 1), 2001, 9, 160, 288), ((1, 96, 1), 4001, 5, 288, 544),
        ((1, 128, 1), 611, 7, 4128, 288), ((1, 128, 2), 2001, 9, 160, 8224), ((1, 128, 4), 450, 3, 160, 4128),
        ((1, 128, 8), 130, 7, 160, 8224), ((2, 128, 1), 5001, 3, 160, 544), ((2, 160, 1), 1501, 7, 1184, 544),
        ((2, 192, 1), 6001, 3, 288, 544), ((2, 224, 1), 6001, 5, 288, 2080)]


def ragged(rows, E):
    """Uneven groups, an empty one among them, that leave some rows over."""
    share = [(i * 7 + 3) % 5 for i in range(E)]
    counts = [(rows - 2) * v // max(sum(share), 1) for v in share]
    assert 0 in counts and 0 < sum(counts) < rows
    return counts


@pytest.mark.parametrize("cut,rows,E,m,k", CUTS)
def test_every_cut(cut, rows, E, m, k):
    counts = ragged(rows, E)
    assert ExpertRows(offsets_of(counts), rows=rows).cut("linear_fp4", m, k) == cut
    run(counts, rows, k, m, "silu", True, True, seed=11, spread=2.0)


@pytest.mark.parametrize("cut,rows,E,m,k", [CUTS[0], CUTS[3], CUTS[6], CUTS[9], CUTS[13]])
def test_a_wait_that_runs_out(cut, rows, E, m, k):
    """The hook leaves a product's first load out, as the host sees it only:
    the status tells, and the next call is right again."""
    counts = ragged(rows, E)
    r = ExpertRows(offsets_of(counts), rows=rows)
    x, w = padded(fp4(sum(counts), k, seed=1), rows), fp4(E, m, k, seed=2)
    out = torch.zeros(rows, m, dtype=torch.bfloat16, device="cuda")
    want = r.linear_fp4(x, w, out=out).clone()
    assert r.status() == 0
    r.ws.view(torch.int32)[7] = 1  # inject_skip_load (byte offset 28)
    r.linear_fp4(x, w, out=out)
    assert r.status() == abi.MOE_ERR_TIMEOUT
    assert torch.equal(r.linear_fp4(x, w, out=out)[:sum(counts)], want[:sum(counts)]) and r.status() == 0


@pytest.mark.parametrize("rows", [1, 2, 17, 600, 3000])
def test_one_group(rows):
    """The shared experts' product: no expert axis; the same bits again."""
    K, N = 1056, 1032
    x, w = fp4(rows, K, seed=3), fp4(N, K, seed=4, std=K ** -0.5)
    b = normal(N, seed=5)
    r = ExpertRows(rows=rows)
    y = r.linear_fp4(x, w, bias=b, act="gelu")
    u, e = linear64(values(x), values(w)[None], [rows], b[None])
    want, err = act64(u, "gelu"), act_error(u, e, "gelu")
    assert_near(y, want, err + BF16 * (want.abs() + err), "y")
    for _ in range(3):
        assert torch.equal(r.linear_fp4(x, w, bias=b, act="gelu"), y)


def test_scales_far_apart():
    """Whole numbers times powers of two from 2^-60 to 2^60: the sum of one
    block is exact, and so is each product that stands alone."""
    rows, N = 40, 24
    for K in (32, 256, 800):
        g = torch.Generator().manual_seed(K)
        x, w = torch.zeros(rows, K), torch.zeros(N, K)
        at = torch.randint(0, K, (N,), generator=g)  # one column of w each
        w[torch.arange(N), at] = torch.exp2(torch.randint(-30, 30, (N,), generator=g).float()) * 3
        x = torch.randint(-2, 3, (rows, K), generator=g) * torch.exp2(
            torch.randint(-30, 30, (rows, K // 32), generator=g).float()).repeat_interleave(32, -1)
        xq, wq = (Fp4Rows(*(t.cuda() for t in encode_fp4(v.bfloat16()))) for v in (x, w))
        assert torch.equal(values(xq).cpu(), x.double()) and torch.equal(values(wq).cpu(), w.double())
        y = ExpertRows(rows=rows).linear_fp4(xq, wq)
        assert torch.equal(y.cpu().double(), (x.double() @ w.double().T).bfloat16().double())


def test_marked_blocks_make_their_sums_nan():
    counts, K, N = [3, 0, 40], 544, 64
    x, w = fp4(43, K, seed=1), fp4(3, N, K, seed=2)
    x.scales[5, 16] = 255      # the last block of a row
    x.scales[5, 17:] = 255     # past the last block: not used
    x.scales[9, 17:] = 255
    w.scales[2, 7, 3] = 255
    w.scales[0, :, 17:] = 255
    y = ExpertRows(offsets_of(counts), rows=43).linear_fp4(x, w)
    bad = torch.isnan(y)
    want = torch.zeros_like(bad)
    want[5] = True
    want[3:, 7] = True
    assert torch.equal(bad, want)


def test_bad_offsets_leave_their_expert_empty():
    K, N = 96, 40
    x, w = fp4(20, K, seed=1), fp4(3, N, K, seed=2)
    good = ExpertRows(offsets_of([5, 5, 10]), rows=20).linear_fp4(x, w)
    for off, rows in (([0, 5, 3, 20], range(0, 5)), ([-3, 5, 10, 20], range(5, 20)), ([0, 5, 10, 21], range(0, 10))):
        r = ExpertRows(torch.tensor(off, dtype=torch.int32, device="cuda"), rows=20)
        out = torch.full((20, N), 7.0, dtype=torch.bfloat16, device="cuda")
        r.linear_fp4(x, w, out=out)
        assert r.status() == abi.MOE_ERR_DEVICE_DATA
        mine = torch.zeros(20, dtype=torch.bool)
        mine[list(rows)] = True
        if off[2] != 3:
            assert torch.equal(out[mine], good[mine])
        else:
            assert torch.equal(out[:3], good[:3])
        assert bool((out[~mine] == 7.0).all()) or off[2] == 3


def test_rows_past_two_gigabytes():
    """Codes and values whose offsets pass 32 bits."""
    rows, K, N = 560_000, 8192, 8
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    tail = normal(64, K, seed=1)
    x[-64:] = tail
    r = ExpertRows(rows=rows)
    q = r.quantize_fp4(x)
    del x
    codes, scales = encode_fp4(tail)
    assert torch.equal(q.codes[-64:].cpu(), codes) and torch.equal(q.scales[-64:].cpu(), scales)
    assert int(q.codes[:-64].max()) == 0 and int(q.scales[:-64].max()) == 0
    w = fp4(N, K, seed=2, std=K ** -0.5)
    y = r.linear_fp4(q, w)
    t = decode_fp4(codes, scales).cuda()
    u, e = linear64(t, values(w)[None], [64])
    assert_near(y[-64:], u, e + BF16 * (u.abs() + e), "y")
    assert bool((y[:-64] == 0).all())
    back = r.dequantize_fp4(q)
    assert torch.equal(back[-64:].double(), t) and r.status() == 0


# --------------------------------------------------------------------------

def test_from_the_dispatch_to_the_combine():
    """Scores, dispatch in 4 bits, two layers with rows in 4 bits, combine:
    on the plan's own stream, and again from a captured graph."""
    T, H, F, E, k = 500, 544, 288, 16, 4
    st = torch.cuda.Stream()
    scoring = Scoring("sigmoid", 4, 2, 2, scale=1.5)
    plan = RoutePlan(RouteShape(T=T, H=H, E=E, k=k, P=1, scoring=scoring, fp4=True), stream=st)
    rows = ExpertRows.of(plan)
    g = torch.Generator().manual_seed(1)
    w1 = quantize_weights_fp4((torch.randn(E, 2 * F, H, generator=g) * H ** -0.5).bfloat16().cuda())
    w2 = quantize_weights_fp4((torch.randn(E, H, F, generator=g) * F ** -0.5).bfloat16().cuda())
    b1 = normal(E, 2 * F, seed=3)
    logits, bias = torch.randn(T, E, generator=g).cuda(), (torch.randn(E, generator=g) * 0.05).cuda()
    x = normal(T, H, seed=4)
    torch.cuda.synchronize()
    kept = {}

    def calls():
        plan.route(logits, bias)
        plan.dispatch(x)
        h = rows.linear_fp4(Fp4Rows(plan.packed, plan.scales), w1, bias=b1, act="swiglu")
        q = rows.quantize_fp4(h)
        kept["h"], kept["q"], kept["y"] = h, q, rows.linear_fp4(q, w2)
        plan.combine(kept["y"])

    def verify():
        st.synchronize()
        assert plan.status() == 0
        counts = plan.layout.counts.tolist()
        src = (plan.layout.src_pos // k).long()
        codes, scales = encode_fp4(x)
        a = decode_fp4(codes, scales).cuda()[src]
        u, e = linear64(a, values(w1), counts, b1)
        want, err = act64(u, "swiglu"), act_error(u, e, "swiglu")
        assert_near(kept["h"], want, err + BF16 * (want.abs() + err), "hidden")
        codes, scales = encode_fp4(kept["h"])
        assert torch.equal(kept["q"].codes.cpu(), codes) and torch.equal(kept["q"].scales.cpu(), scales)
        u, e = linear64(decode_fp4(codes, scales).cuda(), values(w2), counts)
        assert_near(kept["y"], u, e + BF16 * (u.abs() + e), "rows out")
        rows_of = plan.layout.dst_row.view(T, k).long()
        out = (kept["y"].double()[rows_of] * plan.gates.double()[..., None]).sum(1)
        mags = (kept["y"].double()[rows_of] * plan.gates.double()[..., None]).abs().sum(1)
        assert_near(plan.y, out, k * 2.0 ** -24 * mags + BF16 * out.abs(), "y")

    calls()
    verify()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        calls()
    for seed in (7, 8):
        x.copy_(normal(T, H, seed=seed))
        logits.copy_(torch.randn(T, E, generator=g))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            graph.replay()
        verify()


def test_refusals():
    x, w = fp4(8, 64, seed=1), fp4(2, 16, 64, seed=2)
    r = ExpertRows(offsets_of([3, 5]), rows=8)
    with pytest.raises(TypeError):
        r.linear_fp4(x.codes, w)
    with pytest.raises(TypeError):
        r.linear_fp4(x, w.codes)
    with pytest.raises(ValueError, match="w.scales"):
        r.linear_fp4(x, Fp4Rows(w.codes, w.scales[:, :, :8]))
    with pytest.raises(ValueError, match="x.codes"):
        r.linear_fp4(Fp4Rows(x.codes[:, :16].contiguous(), x.scales), w)
    with pytest.raises(ValueError, match="experts"):
        ExpertRows(offsets_of([3, 5, 0]), rows=8).linear_fp4(x, w)
    with pytest.raises(ValueError, match="bias"):
        r.linear_fp4(x, w, bias=torch.zeros(2, 8, dtype=torch.bfloat16, device="cuda"))
    assert fp4_pitch(64) == 16


def test_a_training_step():
    """Scores, dispatch in 4 bits, the experts' product in 4 bits and the
    combine, then the gradients of all of them: the quantisers are passed
    straight through, the products' gradients take the values that the codes
    stand for.  Against 64 bits; each bf16 on the way is off by half a step,
    2^-8 of its value, and fp32 sums add less than another tenth of that."""
    T, H, N, E, k = 300, 288, 160, 8, 3
    scoring = Scoring("sigmoid", 4, 3, 2, scale=1.25)
    plan = RoutePlan(RouteShape(T=T, H=H, E=E, k=k, P=1, scoring=scoring, fp4=True))
    out = RoutePlan(RouteShape(T=T, H=N, E=E, k=k, P=1, scoring=scoring))  # the combine's columns are the product's
    rows = ExpertRows.of(plan)
    g = torch.Generator().manual_seed(1)
    logits = torch.randn(T, E, generator=g).cuda()
    x, dy = normal(T, H, seed=2), normal(T, N, seed=3)
    w = quantize_weights_fp4((torch.randn(E, N, H, generator=g) * H ** -0.5).bfloat16().cuda())
    plan.route(logits)
    plan.dispatch(x)
    out.route(logits)
    eo = rows.linear_fp4(Fp4Rows(plan.packed, plan.scales), w)
    out.combine(eo)
    # backward
    out.combine_backward(dy, eo)
    out.gate_backward(logits)
    d_rows = out.d_expert_out
    w_values = ExpertRows(rows=E * N).dequantize_fp4(Fp4Rows(w.codes.view(E * N, -1), w.scales.view(E * N, -1))).view(E, N, H)
    x_rows = rows.dequantize_fp4(Fp4Rows(plan.packed, plan.scales))
    dw, _ = rows.wgrad(d_rows, x_rows)
    plan.dispatch_backward(rows.dgrad(d_rows, w_values))
    assert plan.status() == 0 and out.status() == 0
    # the same in 64 bits
    xq = decode_fp4(*encode_fp4(x)).cuda()
    wq = values(w)
    assert torch.equal(w_values.double(), wq)
    ids, gates = plan.topk_idx.long(), plan.gates.double()
    e_out = torch.einsum("th,tknh->tkn", xq, wq[ids])
    y = (e_out * gates[..., None]).sum(1)
    mags = (torch.einsum("th,tknh->tkn", xq.abs(), wq[ids].abs()) * gates[..., None]).sum(1)
    assert_near(out.y, y, 2.1 * BF16 * mags, "y")
    d = dy.double()
    gd = gates[..., None] * d[:, None]                       # [T, k, N]
    dx, mx = (torch.einsum("tkn,tknh->th", a, b) for a, b in ((gd, wq[ids]), (gd.abs(), wq[ids].abs())))
    assert_near(plan.dx, dx, 3.1 * BF16 * mx, "dx")
    for e in range(E):
        on = (ids == e).double()[..., None] * gd             # its slots' gradients
        want, mag = on.sum(1).T @ xq, on.abs().sum(1).T @ xq.abs()
        assert_near(dw[e], want, 2.1 * BF16 * mag, f"dw of expert {e}")
    # a product's own fp32 sum is off by the share that its magnitudes leave
    terms = torch.einsum("th,tknh->tkn", xq.abs(), wq[ids].abs())
    off = BF16 * e_out.abs() + 1.01 * sum_error(H, terms)
    assert_near(out.d_gates, (e_out * d[:, None]).sum(2), 1.1 * (off * d[:, None].abs()).sum(2), "d_gates")
    ref = logits.cpu().double().requires_grad_()
    (gates64(ref, ids.cpu(), "sigmoid", True, 1.25) * out.d_gates.cpu().double()).sum().backward()
    bound = backward_error(logits.cpu(), ids.cpu(), out.d_gates.cpu(), E, "sigmoid", True, 1.25)
    assert_near(out.d_logits.cpu(), ref.grad, bound, "d_logits")


@pytest.mark.parametrize("K", [544, 1024, 2048])
@pytest.mark.parametrize("rows", [3, 700])
def test_operands_at_any_16_bytes(K, rows):
    """Codes and scales that start 16 bytes past a multiple of 32."""
    N = 160
    x, w = fp4(rows, K, seed=1, spread=2.0), fp4(N, K, seed=2, std=K ** -0.5, spread=2.0)
    want = ExpertRows(rows=rows).linear_fp4(x, w)

    def moved(t):
        flat = torch.full((t.numel() + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        at = 16 + (-flat.data_ptr()) % 32
        out = flat[at:at + t.numel()].view(t.shape)
        out.copy_(t)
        assert out.data_ptr() % 32 == 16
        return out

    a, b = (Fp4Rows(moved(q.codes), moved(q.scales)) for q in (x, w))
    for xs in (x, a):
        for ws in (w, b):
            assert torch.equal(ExpertRows(rows=rows).linear_fp4(xs, ws), want)
    u, e = linear64(values(x), values(w)[None], [rows])
    assert_near(want, u, e + BF16 * (u.abs() + e), "y")


@pytest.mark.parametrize("cut,rows,m", [((2, 128, 1), 3001, 520), ((2, 160, 1), 12001, 520), ((2, 192, 1), 1501, 2056),
                                        ((2, 224, 1), 8001, 264), ((1, 32, 1), 2090, 136), ((1, 32, 4), 32, 2160),
                                        ((1, 32, 8), 58, 40), ((1, 64, 1), 641, 1544), ((1, 128, 2), 2477, 136),
                                        ((1, 128, 4), 34, 2136), ((1, 128, 8), 536, 40)])
def test_a_product_reads_the_scales_of_its_stage(cut, rows, m):
    """Scales that differ from block to block and row to row, over many rounds
    of the ring, in products of whole numbers whose sums fp32 holds: a scale of
    another stage, in shared or in tensor memory, in either block of a pair,
    gives other bits.  The values are 1, 0 or -1 times 2^0 to 2^3, so a sum
    stays below K * 2^6 < 2^24."""
    K = 8224
    assert ExpertRows(rows=rows).cut("linear_fp4", m, K) == cut
    for seed in range(6):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def whole(*shape):
            v = torch.randint(0, 3, (*shape, K), generator=g, device="cuda")
            s = torch.randint(127, 131, (*shape, K // 32), generator=g, device="cuda")
            c = torch.tensor([2, 0, 10], device="cuda")[v]  # the codes of 1, 0 and -1
            scales = torch.zeros(*shape, fp4_pitch(K), dtype=torch.uint8, device="cuda")
            scales[..., :K // 32] = s.to(torch.uint8)
            q = Fp4Rows((c[..., 0::2] | c[..., 1::2] << 4).to(torch.uint8), scales)
            return q, ((1 - v) << (s - 127).repeat_interleave(32, -1)).double()

        (x, xv), (w, wv) = whole(rows), whole(m)
        want = (xv @ wv.T).bfloat16()
        r = ExpertRows(rows=rows)
        for _ in range(3):
            assert torch.equal(r.linear_fp4(x, w), want)
        assert r.status() == 0


def test_falling_offsets_write_no_row_twice():
    """The third expert starts below the largest offset so far: it is left
    empty, with every row that only it would have."""
    K, N = 96, 40
    x, w = fp4(20, K, seed=1), fp4(3, N, K, seed=2)
    good = ExpertRows(offsets_of([5, 5, 10]), rows=20).linear_fp4(x, w)
    r = ExpertRows(torch.tensor([0, 5, 3, 20], dtype=torch.int32, device="cuda"), rows=20)
    out = torch.full((20, N), 7.0, dtype=torch.bfloat16, device="cuda")
    r.linear_fp4(x, w, out=out)
    assert r.status() == abi.MOE_ERR_DEVICE_DATA
    assert torch.equal(out[:5], good[:5]) and bool((out[5:] == 7.0).all())
