"""The expert products where they are most easily wrong: cuts and tails that
wide layers take, activations' far tails, offsets that do not rise, streams
and graphs, and the FFN's gradients element by element."""
import math

import pytest
import torch

from combine_moe_gate_warp_gb300 import ExpertFFN, ExpertRows, RoutePlan, RouteShape, SavedLayer, abi
from expert_util import (BF16, act64, act_error, assert_near, decode64, encode_saved, grad64, grad_error, normal,
                         offsets_of, spans, sum_error)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import combine_moe_gate_warp_gb300 as pkg
    pkg.build()


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
