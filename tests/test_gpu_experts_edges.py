"""The expert products where they are most easily wrong: cuts and tails that
wide layers take, activations' far tails, offsets that do not rise, streams
and graphs, and the FFN's gradients element by element."""
import pytest
import torch

from combine_moe_gate_warp_gb300 import ExpertFFN, ExpertRows, RoutePlan, RouteShape, abi
from expert_util import BF16, assert_near, normal, offsets_of, spans, sum_error

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
