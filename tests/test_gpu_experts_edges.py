"""The expert products where they are most easily wrong: cuts and tails that
wide layers take, activations' far tails, offsets that do not rise, streams
and graphs, and the FFN's gradients element by element."""
import math

import pytest
import torch

from combine_moe_gate_warp_gb300 import ExpertFFN, ExpertRows, RoutePlan, RouteShape, SavedLayer, abi
from expert_util import (BF16, act64, act_error, assert_near, decode64, encode_saved, grad64, grad_error, linear64,
                         normal, offsets_of, spans, sum_error)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import combine_moe_gate_warp_gb300 as pkg
    pkg.build()


def ragged(rows, E):
    """Counts that leave experts empty, fill no tile and not all rows."""
    share = [(7 * e * e + 3 * e) % 11 for e in range(E)]
    counts = [(rows - 2) * v // max(sum(share), 1) for v in share]
    assert 0 in counts and 0 < sum(counts) < rows
    return counts


def fill(t, rows, value=float("nan")):
    out = torch.full((rows, *t.shape[1:]), value, dtype=t.dtype, device=t.device)
    out[:t.shape[0]] = t
    return out


# SMs of a tile, rows per tile, blocks that share its sums; rows, experts, output columns, k
CUTS = [((1, 32, 1), 7, 3, 96, 64), ((1, 32, 2), 7, 3, 1184, 1040), ((1, 32, 4), 7, 3, 96, 1040),
        ((1, 32, 8), 7, 3, 96, 2064), ((1, 64, 1), 2001, 9, 160, 64), ((1, 96, 1), 4001, 5, 288, 144),
        ((1, 128, 1), 4001, 7, 288, 272), ((1, 128, 2), 2001, 9, 160, 1168), ((1, 128, 4), 450, 3, 160, 1040),
        ((1, 128, 8), 130, 7, 160, 2064), ((2, 128, 1), 5001, 3, 160, 144), ((2, 160, 1), 1501, 7, 1184, 144),
        ((2, 192, 1), 6001, 3, 288, 144), ((2, 224, 1), 6001, 5, 288, 528), ((2, 256, 1), 450, 3, 4128, 528)]


@pytest.mark.parametrize("cut,rows,E,m,k", CUTS)
def test_every_cut_of_linear_and_dgrad(cut, rows, E, m, k):
    """Each way in which the rows' products are cut, forward with everything
    in the epilogue, and the rows' gradient, plain and through a saved layer."""
    counts = ragged(rows, E)
    R = sum(counts)
    r = ExpertRows(offsets_of(counts), rows=rows)
    assert r.cut("linear", m, k) == cut and r.cut("dgrad", k, m) == cut
    x, w = normal(R, k, seed=131), normal(E, m, k, seed=132, std=k ** -0.5)
    b, res = normal(E, m, seed=133), normal(R, m, seed=134)
    xp, saved = fill(x, rows), r.new_saved(m)
    y = r.linear(xp, w, bias=b, act="silu", residual=fill(res, rows), saved=saved)
    assert r.status() == 0
    u, e = linear64(x, w, counts, b)
    want, err = act64(u, "silu") + res.double(), act_error(u, e, "silu")
    err = err + 2.0 ** -23 * want.abs()
    assert_near(y[:R], want, err + BF16 * (want.abs() + err), "y")
    # half a step of a code is 2^-4 of the value or 2^-10 of the scale
    kept, scale = decode64(saved.codes[:R], saved.scales[:R]), torch.pow(2.0, saved.scales[:R].double() - 127)
    assert_near(kept, u, 2.0 ** -4 * (u.abs() + e) + 2.0 ** -10 * scale.repeat_interleave(32, -1) + e, "saved")
    wt = w.mT.contiguous()  # its product's k is the forward's
    dx = r.dgrad(xp, wt)
    d, e = linear64(x, w, counts)
    assert r.status() == 0
    assert_near(dx[:R], d, e + BF16 * (d.abs() + e), "dx")
    codes, scales = encode_saved(normal(R, m, seed=135, std=1.5))
    a = torch.full((rows, m), 7.0, dtype=torch.bfloat16, device="cuda")
    du = r.dgrad(xp, wt, act="gelu", saved=SavedLayer(fill(codes, rows, 0x7F), fill(scales, rows, 0xFF)), a=a)
    assert r.status() == 0
    u = decode64(codes, scales)
    want, err = grad64(u, d, "gelu"), grad_error(u, d, e, "gelu")
    assert_near(du[:R], want, err + BF16 * (want.abs() + err), "du")
    want, err = act64(u, "gelu"), act_error(u, torch.zeros_like(u), "gelu")
    assert_near(a[:R], want, err + BF16 * (want.abs() + err), "a")
    assert bool((a[R:] == 7.0).all())


CUTS_E4M3 = [((1, 32, 1), 7, 3, 96, 64), ((1, 32, 2), 7, 3, 1184, 2064), ((1, 32, 4), 7, 3, 96, 2064),
             ((1, 32, 8), 7, 3, 96, 4112), ((1, 64, 1), 2001, 9, 160, 64), ((1, 96, 1), 4001, 5, 288, 272),
             ((1, 128, 1), 611, 7, 4128, 144), ((1, 128, 2), 2001, 9, 160, 4112), ((1, 128, 4), 450, 3, 160, 2064),
             ((1, 128, 8), 130, 7, 160, 4112), ((2, 128, 1), 5001, 3, 160, 272), ((2, 160, 1), 1501, 7, 1184, 272),
             ((2, 192, 1), 6001, 3, 288, 272), ((2, 224, 1), 6001, 5, 288, 1040), ((2, 256, 1), 450, 3, 4128, 1040)]


@pytest.mark.parametrize("cut,rows,E,m,k", CUTS_E4M3)
def test_every_cut_of_e4m3_rows(cut, rows, E, m, k):
    """x = zero + scale * code, w = scale * code, from the codes in 64 bits.
    The sums are fp32 (products of codes, then three fp32 steps)."""
    counts = ragged(rows, E)
    R = sum(counts)
    r = ExpertRows(offsets_of(counts), rows=rows)
    assert r.cut("linear", m, k, e4m3=True) == cut
    g = torch.Generator().manual_seed(141)
    xq, wq = ((torch.randn(*s, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
              for s in ((R, k), (E, m, k)))
    xs = (torch.rand(R, 2, generator=g) * 0.02 + 0.001).cuda()
    ws = torch.empty(E, m, 2, device="cuda")
    ws[..., 0] = (torch.rand(E, m, generator=g) * 1e-3 + 1e-4).cuda()
    ws[..., 1] = (wq.double().sum(2) * ws[..., 0].double()).float()
    y = r.linear(fill(xq.view(torch.uint8), rows, 0x7F), wq.view(torch.uint8), x_scales=fill(xs, rows), w_scales=ws)
    assert r.status() == 0
    for e, lo, hi in spans(counts):
        a, b = xq[lo:hi].double(), wq[e].double()
        s, z = xs[lo:hi, :1].double() * ws[e, :, 0].double(), xs[lo:hi, 1:].double() * ws[e, :, 1].double()
        acc = a @ b.T
        want = s * acc + z
        err = s * sum_error(k, a.abs() @ b.abs().T) + 2.0 ** -22 * ((s * acc).abs() + z.abs())
        assert_near(y[lo:hi], want, err + BF16 * (want.abs() + err), f"y of expert {e}")


@pytest.mark.parametrize("cut,rows,E,m,k", [
    ((1, 128, 1), 20, 9, 96, 1040), ((1, 128, 2), 2500, 3, 96, 64), ((1, 128, 4), 3001, 3, 96, 64),
    ((1, 128, 8), 6001, 3, 96, 64), ((2, 128, 1), 2001, 9, 520, 392), ((2, 128, 1), 4001, 7, 288, 528),
    ((2, 256, 1), 7, 7, 1056, 4112), ((2, 256, 1), 6001, 5, 1032, 520)])
def test_every_cut_of_wgrad(cut, rows, E, m, k):
    counts = ragged(rows, E)
    R = sum(counts)
    r = ExpertRows(offsets_of(counts), rows=rows)
    assert r.cut("wgrad", m, k) == cut
    dy, x = normal(R, m, seed=151), normal(R, k, seed=152)
    dw, db = r.wgrad(fill(dy, rows), fill(x, rows), bias=True)
    assert r.status() == 0
    for e, lo, hi in spans(counts):
        d, v = dy[lo:hi].double(), x[lo:hi].double()
        want, err = d.T @ v, sum_error(hi - lo, d.abs().T @ v.abs())
        assert_near(dw[e], want, err + BF16 * (want.abs() + err), f"dw[{e}]")
        want, err = d.sum(0), sum_error(hi - lo, d.abs().sum(0))
        assert_near(db[e], want, err + BF16 * (want.abs() + err), f"db[{e}]")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(2560, 1024), (2560, 1152), (1416, 1160), (2056, 1352), (1032, 1416)])
def test_wgrad_of_wide_layers(N, K, dtype):
    """Pairs of SMs with 256 columns between them: tails of every length
    beside rows that are not finite (another expert's, or nobody's), last
    tiles of at most 128 and of more columns, columns that are whole blocks
    of 64 or not."""
    counts = [0, 1, 15, 33, 0, 130, 257, 16, 79]
    wild = (3, 7)  # experts whose rows are not finite
    R, rows, E = sum(counts), 900, len(counts)
    dy, x = normal(R, N, seed=101), normal(R, K, seed=102)
    for e, lo, hi in spans(counts):
        if e in wild:
            x[lo:hi], dy[lo:hi] = float("nan"), float("inf")
    dp = torch.full((rows, N), float("inf"), dtype=torch.bfloat16, device="cuda")
    xp = torch.full((rows, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    dp[:R], xp[:R] = dy, x
    r = ExpertRows(offsets_of(counts), rows=rows)
    assert r.cut("wgrad", N, K) == (2, 256, 1)
    half = BF16 if dtype == torch.bfloat16 else 2.0 ** -24
    first = None
    for _ in range(4):
        dw, db = r.wgrad(dp, xp, bias=True, dtype=dtype)
        assert r.status() == 0
        for e, lo, hi in spans(counts):
            if e in wild:
                assert bool(torch.isnan(dw[e]).all()) and bool((db[e] == float("inf")).all())
        dw, db = dw.nan_to_num(0.0), db.nan_to_num(0.0, posinf=0.0)
        if first is None:
            first = (dw, db)
        assert torch.equal(dw, first[0]) and torch.equal(db, first[1]), "another result the second time"
    dw, db = first
    for e, lo, hi in spans(counts):
        if e in wild:
            continue
        d, v = dy[lo:hi].double(), x[lo:hi].double()
        want, err = d.T @ v, sum_error(hi - lo, d.abs().T @ v.abs())
        assert_near(dw[e], want, err + half * (want.abs() + err), f"dw[{e}]")
        want, err = d.sum(0), sum_error(hi - lo, d.abs().sum(0))
        assert_near(db[e], want, err + half * (want.abs() + err), f"db[{e}]")


@pytest.mark.parametrize("own_stream", [True, False])
def test_a_plan_on_a_stream_of_its_own(own_stream):
    """route, dispatch, experts and combine follow each other on the plan's
    stream, forward and backward, called while another stream is current and
    the plan's is held up by work before them."""
    T, H, E, k, F = 200, 128, 8, 2, 64
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(111)).cuda()
    x, dy = normal(T, H, seed=112), normal(T, H, seed=113)
    w1, w2 = normal(E, 2 * F, H, seed=114, std=H ** -0.5), normal(E, H, F, seed=115, std=F ** -0.5)

    def layer(plan, ffn):
        plan.route(logits)
        plan.dispatch(x)
        plan.combine(ffn.forward(plan.packed))
        plan.combine_backward(dy, ffn.y)
        plan.dispatch_backward(ffn.backward(plan.d_expert_out, plan.packed).dx)

    def parts(plan, ffn):
        return [t.clone() for t in (plan.y, plan.dx, ffn.grads.dw1, ffn.grads.dw2)]

    def build(stream=None):
        plan = RoutePlan(RouteShape(T=T, H=H, E=E, k=k, P=4), "cuda", stream=stream)
        return plan, ExpertFFN(ExpertRows.of(plan), w1, w2)

    plan, ffn = build()
    layer(plan, ffn)
    assert plan.status() == 0
    want = parts(plan, ffn)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if own_stream:   # the plan on a side stream, the caller on the default one
        plan, ffn = build(side)
        run, current = side, torch.cuda.current_stream()
    else:            # the other way round
        plan, ffn = build()
        run, current = torch.cuda.current_stream(), side
    torch.cuda.synchronize()
    with torch.cuda.stream(current):
        for _ in range(2):
            for t in (plan.packed, plan.y, ffn.y, ffn.hidden):
                t.fill_(float("nan"))
            torch.cuda.synchronize()
            with torch.cuda.stream(run):
                torch.cuda._sleep(20_000_000)  # about 10 ms
            layer(plan, ffn)
            assert plan.status() == 0
            torch.cuda.synchronize()
            for got, w in zip(parts(plan, ffn), want):
                assert torch.equal(got, w)
            # outputs that the handle allocates are the stream's as well
            r = ffn.rows
            assert torch.equal(r.linear(plan.packed, w1, act="swiglu"), r.linear(plan.packed, w1, act="swiglu"))
            assert r.status() == 0


# Evaluated in fp32, relative to the value: exp's argument is rounded (2^-24 of
# up to 85) and exp is off by 2 + 1.18 |argument| steps of 2^-23, which makes
# 2^-15.6 at the far end; the rest (a fit, a division, a few products) stays
# below 2^-18.
FAR = 2.0 ** -15


def phi64(u):
    """The normal distribution function; 1 + erf has no digits left below -6."""
    return torch.special.erfc(-u / math.sqrt(2)) / 2


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_keep_their_tails(act):
    """Where u is far below zero the activation is small, but it is a number
    with the digits of its type: half a step of bf16 relative to the value."""
    lo = -12.5 if act == "gelu" else -70.0   # further out fp32's exponential ends
    u = torch.linspace(lo, 8.0, 8 * 4096).bfloat16().reshape(-1, 8).cuda()
    eye = torch.eye(8).bfloat16().cuda()
    r = ExpertRows(rows=u.shape[0])
    y = r.linear(u, eye, act=act)
    assert r.status() == 0
    u = u.double()
    want = u * phi64(u) if act == "gelu" else act64(u, act)
    assert_near(y, want, (BF16 * (1 + FAR) + FAR) * want.abs(), "y")


def test_gelus_slope_keeps_its_tail():
    """The slope Phi(u) + u phi(u), through a saved layer: its error is
    relative to the two terms (they cancel near u = -0.75)."""
    u = torch.linspace(-12.5, 8.0, 64 * 512).bfloat16().reshape(-1, 64)
    u[:, 32:] = u[:, 32:].flip(0)  # the blocks of a row have other scales
    codes, scales = encode_saved(u)
    saved = SavedLayer(codes.cuda(), scales.cuda())
    u = decode64(saved.codes, saved.scales)
    rows = u.shape[0]
    dy = torch.ones(rows, 64, dtype=torch.bfloat16, device="cuda")
    r = ExpertRows(rows=rows)
    du = r.act_backward(dy, act="gelu", saved=saved)
    assert r.status() == 0
    density = torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
    want, size = phi64(u) + u * density, phi64(u) + u.abs() * density
    assert_near(du, want, BF16 * want.abs() + 2 * FAR * size, "du")


@pytest.mark.parametrize("with_a", [False, True])
@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
@pytest.mark.parametrize("out", [32, 160, 2080])
def test_act_backward_of_ragged_rows(act, out, with_a):
    """The activation's gradient alone: rows of several experts, the first of
    them past the buffer's start, the last before its end."""
    counts, first = [0, 3, 41, 0, 128, 1], 7
    R, rows = sum(counts), first + sum(counts) + 20
    N = 2 * out if act == "swiglu" else out
    codes, scales = encode_saved(normal(rows, N, seed=121, std=1.5))
    codes[:first], scales[:first], codes[first + R:], scales[first + R:] = 0x7F, 0xFF, 0x7F, 0xFF
    saved, dy = SavedLayer(codes, scales), normal(rows, out, seed=122)
    r = ExpertRows(offsets_of(counts) + first, rows=rows)
    du = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    a = torch.full((rows, out), 7.0, dtype=torch.bfloat16, device="cuda") if with_a else None
    assert r.act_backward(dy, act=act, saved=saved, out=du, a=a) is du
    assert r.status() == 0
    mine = slice(first, first + R)
    u, d = decode64(codes[mine], scales[mine]), dy[mine].double()
    want, err = grad64(u, d, act), grad_error(u, d, torch.zeros_like(d), act)
    assert_near(du[mine], want, err + BF16 * (want.abs() + err), "du")
    if with_a:
        want, err = act64(u, act), act_error(u, torch.zeros_like(u), act)
        assert_near(a[mine], want, err + BF16 * (want.abs() + err), "a")
    for t in (du, a):
        if t is not None:
            assert bool((t[:first] == 7.0).all()) and bool((t[first + R:] == 7.0).all())


@pytest.mark.parametrize("off", [[0, 40, 30, 100], [0, 40, 101, 100], [-1, 40, 70, 100], [0, 40, 70, 101],
                                 [0, 40, 70, -5], [0, 90, 20, 80]])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_act_backward_takes_bad_offsets_for_empty(off, act):
    """As the products do: an expert whose offsets are negative, pass the
    rows, decrease or start below an earlier one is empty, and recorded."""
    rows, out = 100, 64
    N = 2 * out if act == "swiglu" else out
    codes, scales = encode_saved(normal(rows, N, seed=123))
    r = ExpertRows(torch.tensor(off, dtype=torch.int32, device="cuda"), rows=rows)
    du = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    whole = torch.empty_like(du)
    dy = normal(rows, out, seed=124)
    r.act_backward(dy, act=act, saved=SavedLayer(codes, scales), out=du)
    assert r.status() == abi.MOE_ERR_DEVICE_DATA and r.status() == 0
    ExpertRows(rows=rows).act_backward(dy, act=act, saved=SavedLayer(codes, scales), out=whole)
    good = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for e in range(3):
        lo, hi = off[e], off[e + 1]
        if lo >= max([0] + off[:e]) and lo <= hi <= rows:
            good[lo:hi] = True
    assert torch.equal(du[good], whole[good]) and bool((du[~good] == 7.0).all())


def test_an_expert_with_very_many_rows():
    """One expert of 152 has 2^28 rows: its weight gradient is one block's
    tile, which takes longer than a wait's second.  Small whole numbers that
    cancel, so that the sums are exact."""
    rows, E, hot = (1 << 28) + 37, 152, 40
    sign = 1 - 2 * (torch.arange(rows, device="cuda", dtype=torch.int32) & 1).to(torch.int8)
    cols = torch.arange(1, 9, device="cuda", dtype=torch.bfloat16)
    dy, x = torch.empty(rows, 8, dtype=torch.bfloat16, device="cuda"), cols.repeat(rows, 1)
    torch.mul(sign[:, None], cols, out=dy)
    del sign
    out = rows // 3 * 2 + 1  # an odd row: what it would have taken off stays
    x[out] = 0
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[hot + 1:] = rows
    r = ExpertRows(off, rows=rows)
    dw, db = r.wgrad(dy, x, bias=True, dtype=torch.float32)
    assert r.status() == 0
    c = cols.float()
    # rows is odd: the last row's product is left over, and the missing odd row's
    assert torch.equal(dw[hot], 2 * c[:, None] * c) and torch.equal(db[hot], c)
    dw[hot], db[hot] = 0, 0
    assert bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act,H,F", [("swiglu", 264, 96), ("gelu", 128, 160), ("silu", 1032, 544)])
def test_ffn_element_by_element(act, H, F, dtype):
    """The network's output and every gradient against the formulas in 64
    bits, from the layer that the forward pass saved: the roundings to bf16 of
    the hidden layer and of its gradient, and the sums."""
    counts = [70, 0, 33, 150, 1]
    R, rows, E, N = sum(counts), 300, 5, 2 * F if act == "swiglu" else F
    x, dy = normal(R, H, seed=161), normal(R, H, seed=162)
    w1, w2 = normal(E, N, H, seed=163, std=H ** -0.5), normal(E, H, F, seed=164, std=F ** -0.5)
    b1, b2 = normal(E, N, seed=165, std=0.3), normal(E, H, seed=166, std=0.3)
    ffn = ExpertFFN(ExpertRows(offsets_of(counts), rows=rows), w1, w2, b1=b1, b2=b2, act=act, dtype=dtype)
    y = ffn.forward(fill(x, rows))[:R].clone()
    g = ffn.backward(fill(dy, rows), fill(x, rows))
    assert ffn.rows.status() == 0
    half = BF16 if dtype == torch.bfloat16 else 2.0 ** -24

    def near(got, want, err, what, step=BF16):
        assert_near(got, want, err + step * (want.abs() + err), what)

    u, eu = linear64(x, w1, counts, b1)
    scale = torch.pow(2.0, ffn.saved.scales[:R].double() - 127).repeat_interleave(32, -1)
    kept = decode64(ffn.saved.codes[:R], ffn.saved.scales[:R])
    assert_near(kept, u, 2.0 ** -4 * (u.abs() + eu) + 2.0 ** -10 * scale + eu, "saved")
    for e, lo, hi in spans(counts):
        xe, de, w1e, w2e = x[lo:hi].double(), dy[lo:hi].double(), w1[e].double(), w2[e].double()
        # forward: the hidden layer is rounded to bf16
        a, ea = act64(u[lo:hi], act), act_error(u[lo:hi], eu[lo:hi], act)
        ea = ea + BF16 * (a.abs() + ea)
        want = a @ w2e.T + b2[e].double()
        near(y[lo:hi], want, ea @ w2e.abs().T + sum_error(F, (a.abs() + ea) @ w2e.abs().T + b2[e].double().abs()),
             f"y of expert {e}")
        # backward: the gradient of the hidden layer, and the activation of what was kept
        k = kept[lo:hi]
        d, ed = de @ w2e, sum_error(H, de.abs() @ w2e.abs())
        du, edu = grad64(k, d, act), grad_error(k, d, ed, act)
        edu = edu + BF16 * (du.abs() + edu)
        size = du.abs() + edu
        near(g.dx[lo:hi], du @ w1e, edu @ w1e.abs() + sum_error(N, size @ w1e.abs()), f"dx of expert {e}")
        near(g.dw1[e], du.T @ xe, edu.T @ xe.abs() + sum_error(hi - lo, size.T @ xe.abs()), f"dw1[{e}]", half)
        near(g.db1[e], du.sum(0), edu.sum(0) + sum_error(hi - lo, size.sum(0)), f"db1[{e}]", half)
        a, ea = act64(k, act), act_error(k, torch.zeros_like(k), act)
        ea = ea + BF16 * (a.abs() + ea)
        near(g.dw2[e], de.T @ a, de.abs().T @ ea + sum_error(hi - lo, de.abs().T @ (a.abs() + ea)), f"dw2[{e}]", half)
        near(g.db2[e], de.sum(0), sum_error(hi - lo, de.abs().sum(0)), f"db2[{e}]", half)


def test_the_experts_in_a_graph():
    """A layer's calls captured once, on the plan's stream, and replayed on
    other tokens: the same bits as the calls themselves."""
    T, H, E, k, F = 64, 128, 8, 2, 96
    side = torch.cuda.Stream()
    plan = RoutePlan(RouteShape(T=T, H=H, E=E, k=k, P=4), "cuda", stream=side)
    w1, w2 = normal(E, 2 * F, H, seed=171, std=H ** -0.5), normal(E, H, F, seed=172, std=F ** -0.5)
    b1, b2 = normal(E, 2 * F, seed=173), normal(E, H, seed=174)
    ffn = ExpertFFN(ExpertRows.of(plan), w1, w2, b1=b1, b2=b2)
    logits = torch.zeros(T, E, device="cuda")
    x, dy = (torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def layer():
        plan.route(logits)
        plan.dispatch(x)
        plan.combine(ffn.forward(plan.packed))
        plan.combine_backward(dy, ffn.y)
        plan.dispatch_backward(ffn.backward(plan.d_expert_out, plan.packed).dx)

    def parts():
        g = ffn.grads
        return [t.clone() for t in (plan.y, plan.dx, g.dw1, g.dw2, g.db1, g.db2)]

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        layer()  # the kernels' attributes are set on first use
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer()
    for seed in (175, 178, 181):
        logits.copy_(torch.randn(T, E, generator=torch.Generator().manual_seed(seed)))
        x.copy_(normal(T, H, seed=seed + 1))
        dy.copy_(normal(T, H, seed=seed + 2))
        torch.cuda.synchronize()
        layer()
        torch.cuda.synchronize()
        want = parts()
        for t in (plan.y, plan.dx, ffn.y, ffn.grads.dw1, ffn.grads.dw2, ffn.grads.db1, ffn.grads.db2):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        assert plan.status() == 0
        for got, w in zip(parts(), want):
            assert torch.equal(got, w)


def test_the_example_layers_gradients():
    """examples/moe_layer.py: forward and backward of the whole layer, the
    gradients to tokens and router against differentiation in 64 bits.

    The hidden layer's 8 bits are off by up to 2^-4 of each value; the slopes
    and the other factor of swiglu follow with at most 1.13 and 1 times that,
    so that dx is off by 2.2 * 2^-4 of its size.  The gates' gradients do not
    pass through it: a handful of roundings to bf16 in a row, 4 * 2^-8."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    torch.manual_seed(7)
    T, H, F, E, k = 200, 128, 64, 8, 3
    layer = module.MoELayer(T, H=H, F=F, E=E, k=k, P=4)
    x, dy = normal(T, H, seed=191), normal(T, H, seed=192)
    y = layer.forward(x).clone()
    dx, d_router = layer.backward(dy)
    assert layer.plan.status() == 0 and layer.shared.rows.status() == 0

    x64 = x.double().requires_grad_()
    router = layer.router.double().requires_grad_()

    def ffn(rows, w1, w2):
        return act64(rows @ w1.double().T, "swiglu") @ w2.double().T

    p = torch.softmax(x64 @ router.T, 1)
    want = ffn(x64, layer.shared.w1, layer.shared.w2)
    idx = layer.plan.topk_idx.long()
    for j in range(k):
        for e in range(E):
            at = (idx[:, j] == e).nonzero()[:, 0]
            if len(at):
                part = ffn(x64[at], layer.experts.w1[e], layer.experts.w2[e])
                want = want.index_add(0, at, p[at, e: e + 1] * part)
    (want * dy.double()).sum().backward()

    def off(got, exact):
        return float((got.double() - exact).norm() / exact.norm())

    assert off(y, want.detach()) <= 4 * BF16
    assert off(d_router, router.grad) <= 4 * BF16
    assert off(dx, x64.grad) <= 2.2 * 2.0 ** -4
