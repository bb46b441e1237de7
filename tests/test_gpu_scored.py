"""Routing by scores on the GPU against the same selection in 64 bits: every
score, groups, biases, ties and near ties, the statistics and the next bias,
the gradient, and the plan, graph and pipeline that use it."""
import pytest
import torch

from combine_moe_gate_warp_gb300 import (MoeError, RouteGraph, RoutePipeline, RoutePlan, RouteShape, Scoring, abi,
                                         alloc_workspace, moe_gate_scored, moe_gate_scored_backward, moe_get_status)
from scored_util import backward_error, gates64, gates_error, scores64, select64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import combine_moe_gate_warp_gb300 as pkg
    pkg.build()


def randn(*shape, seed, std=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std


def gate(logits, k, scoring, bias=None, bias_next=None, rate=0.0, stats=True):
    T, E = logits.shape
    dev = "cuda"
    idx = torch.full((T, k), -7, dtype=torch.int32, device=dev)
    gates = torch.full((T, k), 9.0, device=dev)
    counts = torch.full((E,), -7, dtype=torch.int32, device=dev)
    aux, ent = (torch.full((1,), -7.0, dtype=torch.float64, device=dev) for _ in range(2))
    ws = alloc_workspace(T, E, k, 1)
    moe_gate_scored(logits.to(dev), k, scoring, None if bias is None else bias.to(dev), idx, gates, counts,
                    aux if stats else None, ent if stats else None, ws, bias_next=bias_next, bias_rate=rate)
    return idx, gates, counts, aux, ent, ws


def undecided(logits, k, scoring, bias):
    """Tokens whose selection hangs on values that fp64 itself cannot order:
    exp() is off by a step of 2^-52 in this library and in that one, a score
    below 1 by 3 half steps more, the sum of two by another, 2^-50 in all, so
    of two values nearer than 2^-49 either may come out the larger.  Sums of
    two scores that lie a few steps of fp32 apart, 2^-24, differ by the
    square of that."""
    T, E = logits.shape
    v = scores64(logits, scoring.score) + (0 if bias is None else bias.double())
    g = v.reshape(T, scoring.groups, -1).sort(2, descending=True)[0][:, :, :scoring.group_top].sum(2)
    g = g.sort(1, descending=True)[0]
    out = (-v.sort(1, descending=True)[0].diff(dim=1) <= 2.0 ** -49).any(1)
    if scoring.top_groups < scoring.groups:
        out |= g[:, scoring.top_groups - 1] - g[:, scoring.top_groups] <= 2.0 ** -49
    return out


def check(logits, k, scoring, bias=None, near=False):
    T, E = logits.shape
    idx, gates, counts, aux, ent, ws = gate(logits, k, scoring, bias)
    assert moe_get_status(ws) == 0
    want = select64(logits, k, scoring.score, scoring.groups, scoring.top_groups, scoring.group_top, bias)
    got = idx.cpu().long()
    wrong = (got != want).any(1)
    if near and bool(wrong.any()):
        assert bool(undecided(logits[wrong], k, scoring, bias).all())
        want = torch.where(wrong[:, None], got, want)
    assert torch.equal(got, want), f"{int(wrong.sum())} of {T} tokens"
    g = gates64(logits, want, scoring.score, scoring.renorm, scoring.scale)
    off = (gates.cpu().double() - g).abs()
    bound = gates_error(g, logits, want, scoring.score, scoring.renorm, scoring.scale)
    assert bool((off <= bound).all()), f"gates off by {off.max()}"
    n = torch.bincount(want.flatten(), minlength=E)
    assert torch.equal(counts.cpu().long(), n)
    p = n.double() / (T * k)
    assert abs(aux.item() - E * ((n.double() / T) ** 2).sum().item()) <= 1e-12 * E * k * k
    assert abs(ent.item() + (p * torch.log2(p + 1e-8)).sum().item()) <= 1e-6
    return idx, gates


SHAPES = [  # T, E, k, groups, top_groups, group_top
    (1, 64, 8, 8, 4, 2), (3, 1, 1, 1, 1, 1), (5, 2, 2, 2, 2, 1), (33, 8, 2, 1, 1, 1), (257, 60, 6, 5, 3, 1),
    (1000, 64, 8, 8, 4, 2), (513, 256, 8, 16, 6, 2), (300, 256, 16, 32, 9, 2), (129, 255, 5, 85, 40, 2),
    (70, 256, 4, 256, 7, 1), (65, 64, 16, 4, 1, 2), (2048, 16, 1, 4, 2, 2), (31, 33, 3, 11, 11, 2),
    (40000, 64, 8, 8, 3, 2), (20000, 24, 4, 1, 1, 1),
    # as many tokens as one lane each takes
    (39001, 33, 3, 11, 4, 2), (39040, 60, 6, 5, 3, 1), (39007, 17, 16, 1, 1, 1), (40001, 8, 2, 1, 1, 1),
    (39500, 64, 16, 4, 2, 2), (117001, 128, 8, 16, 5, 2), (117000, 96, 4, 1, 1, 1), (39009, 1, 1, 1, 1, 1),
    (39002, 62, 5, 31, 30, 1), (39003, 48, 7, 2, 1, 2), (38999, 3, 2, 3, 2, 1),
    # many groups, and groups by their best that hold fewer than k of them
    (39100, 64, 8, 32, 9, 2), (39101, 60, 5, 20, 13, 2), (6000, 256, 8, 128, 40, 2), (300, 256, 16, 128, 9, 2),
    (39102, 64, 6, 32, 3, 1), (5000, 128, 4, 64, 2, 1), (5001, 160, 9, 80, 5, 1), (39103, 40, 1, 20, 19, 2),
    (9000, 160, 6, 8, 3, 2), (17, 96, 12, 12, 5, 1),
]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,top,two", SHAPES)
def test_selection(T, E, k, groups, top, two, score):
    logits = randn(T, E, seed=T + E) + 0.5 * randn(E, seed=E)
    spread = 0.05 if score == "sigmoid" else 0.5 / E
    bias = randn(E, seed=k, std=spread)
    check(logits, k, Scoring(score, groups, top, two, renorm=True, scale=2.5), bias)
    check(logits * 3, k, Scoring(score, groups, top, two, renorm=False, scale=1.0))
    # the bias decides, not the score
    check(logits, k, Scoring(score, groups, top, two), bias * 100)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,top,two", [(700, 64, 8, 8, 4, 2), (700, 256, 8, 16, 6, 2), (6000, 64, 6, 8, 4, 1),
                                                  (50000, 64, 8, 8, 4, 2), (500, 60, 4, 1, 1, 1),
                                                  (40000, 64, 8, 32, 9, 2), (5000, 256, 8, 128, 40, 2),
                                                  (40000, 64, 4, 32, 3, 1)])
def test_ties_and_near_ties(T, E, k, groups, top, two, score):
    s = Scoring(score, groups, top, two)
    # every score the same: the lowest ids
    zero = torch.zeros(T, E)
    idx, _ = check(zero, k, s, torch.zeros(E))
    assert torch.equal(idx.cpu().long(), torch.arange(k).expand(T, k))
    check(zero + 1.25, k, s)
    # logits as bf16 leaves them: many are equal
    coarse = randn(T, E, seed=1).bfloat16().float()
    check(coarse, k, s)
    check(coarse, k, s, randn(E, seed=2, std=0.01).bfloat16().float())
    # neighbours a few steps of fp32 apart, in and out of order
    steps = torch.randint(-3, 4, (T, E), generator=torch.Generator().manual_seed(3))
    base = coarse[:, :1].expand(T, E).contiguous().abs() + 0.5
    close = (base.view(torch.int32) + steps.int()).view(torch.float32)
    check(close, k, s, near=True)
    check(close, k, s, randn(E, seed=4, std=1e-7), near=True)
    # scores that differ, sums with the bias that do not (to fp32)
    bias = randn(E, seed=5, std=0.1)
    level = torch.log((0.5 - bias) / (0.5 + bias)) if score == "sigmoid" else randn(E, seed=6, std=1e-6)
    check(level.expand(T, E) + randn(T, 1, seed=7, std=1e-3), k, s, bias if score == "sigmoid" else None,
          near=True)


def test_far_logits():
    """Scores that 64 bits round to 0 or 1, and large biases."""
    pick = torch.tensor([-800.0, -120.0, -50.0, -3.0, 0.0, 3.0, 45.0, 50.0, 120.0, 800.0])
    logits = pick[torch.randint(0, 10, (400, 64), generator=torch.Generator().manual_seed(1))]
    for score in ("sigmoid", "softmax"):
        for bias in (None, randn(64, seed=2), randn(64, seed=3, std=1e4)):
            check(logits, 8, Scoring(score, 8, 4, 2, renorm=False), bias)
            check(logits, 3, Scoring(score, 1, 1, 1, renorm=True), bias)


def test_no_tokens_and_optional_outputs():
    s = Scoring()
    idx, gates, counts, aux, ent, ws = gate(torch.zeros(0, 8), 2, s)
    assert counts.tolist() == [0] * 8 and aux.item() == 0 and ent.item() == 0 and moe_get_status(ws) == 0
    logits = randn(50, 8, seed=1)
    full, none = gate(logits, 2, s), gate(logits, 2, s, stats=False)
    assert all(torch.equal(a, b) for a, b in zip(full[:3], none[:3]))
    assert none[3].item() == -7 and none[4].item() == -7


def test_bad_data_is_recorded_and_ids_stay_valid():
    for value in (float("nan"), float("inf"), float("-inf")):
        for score in ("sigmoid", "softmax"):
            for T in (200, 60000):
                logits = randn(T, 64, seed=1)
                logits[7, 3] = value
                logits[9] = value
                idx, _, counts, _, _, ws = gate(logits, 8, Scoring(score, 8, 4, 2))
                assert moe_get_status(ws) == abi.MOE_ERR_DEVICE_DATA
                got = idx.cpu().long()
                assert int(got.min()) >= 0 and int(got.max()) < 64 and int(counts.sum()) == T * 8
                assert bool((got.sort(1)[0].diff(dim=1) > 0).all()), "an expert twice"
                good = torch.ones(T, dtype=torch.bool)
                good[7] = good[9] = False
                assert torch.equal(got[good], select64(logits[good], 8, score, 8, 4, 2))
    bias = torch.zeros(64)
    bias[5] = float("nan")
    assert moe_get_status(gate(randn(9, 64, seed=1), 8, Scoring(), bias)[-1]) == abi.MOE_ERR_DEVICE_DATA


@pytest.mark.parametrize("T", [37, 4096, 70000])
def test_next_bias(T):
    E, k = 48, 4
    logits, bias = randn(T, E, seed=1) + randn(E, seed=2), randn(E, seed=3, std=0.02).cuda()
    out = torch.empty(E, device="cuda")
    s = Scoring("sigmoid", 6, 3, 2)
    counts = gate(logits, k, s, bias.cpu(), out, 1e-3)[2].long()
    want = bias + 1e-3 * torch.sign(T * k - counts * E).float()
    assert torch.equal(out, want)
    # in place, and from no bias at all
    ws = alloc_workspace(T, E, k, 1)
    ids, g = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    n = torch.empty(E, dtype=torch.int32, device="cuda")
    moe_gate_scored(logits.cuda(), k, s, bias, ids, g, n, None, None, ws, bias_next=bias, bias_rate=1e-3)
    assert torch.equal(bias, want) and torch.equal(n.long(), counts)
    moe_gate_scored(logits.cuda(), k, s, None, ids, g, n, None, None, ws, bias_next=out, bias_rate=0.5)
    assert torch.equal(out, 0.5 * torch.sign(T * k - n.long() * E).float())


def test_bias_brings_balance():
    """Batch after batch, the counts come nearer to the mean."""
    T, E, k = 4096, 32, 4
    logits = (randn(T, E, seed=1) + randn(E, seed=2)).cuda()
    bias = torch.zeros(E, device="cuda")
    ws = alloc_workspace(T, E, k, 1)
    ids, g = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    n = torch.empty(E, dtype=torch.int32, device="cuda")
    first = None
    for _ in range(200):
        moe_gate_scored(logits, k, Scoring(), bias, ids, g, n, None, None, ws, bias_next=bias, bias_rate=0.005)
        first = int(n.max()) if first is None else first
    assert int(n.max()) < 1.2 * T * k / E < first


# --------------------------------------------------------------------------

@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (7, 2, 2), (65, 4, 3), (100, 7, 2), (50, 16, 16), (33, 33, 5),
                                   (1021, 60, 6), (500, 128, 4), (300, 256, 16), (20000, 64, 8), (3, 200, 1)])
def test_backward(T, E, k, renorm, score):
    logits, d = randn(T, E, seed=E) * 2, randn(T, k, seed=k)
    idx = select64(logits, k, score)
    ref = logits.double().requires_grad_()
    (gates64(ref, idx, score, renorm, 1.7) * d.double()).sum().backward()
    out = torch.full((T, E), 5.0, device="cuda")
    ws = alloc_workspace(T, E, k, 1)
    moe_gate_scored_backward(logits.cuda(), idx.int().cuda(), d.cuda(), Scoring(score, renorm=renorm, scale=1.7), out,
                             ws)
    assert moe_get_status(ws) == 0
    off = (out.cpu().double() - ref.grad).abs()
    bound = backward_error(logits, idx, d, E, score, renorm, 1.7)
    assert bool((off <= bound).all()), f"off by {off.max()}, {(off / bound).max()} of the bound"
    # along a direction, against differences of the gates
    v = randn(T, E, seed=3).double()
    h = 1e-5
    diff = sum(s * (gates64(logits.double() + s * h * v, idx, score, renorm, 1.7) * d.double()).sum() for s in (1, -1))
    got = (out.cpu().double() * v).sum()
    assert abs(got - diff / (2 * h)) <= 1e-6 * (v.abs() * bound).sum() / 2.0 ** -23 + 1e-7


def test_backward_bad_and_repeated_ids():
    T, E, k = 40, 24, 3
    logits, d = randn(T, E, seed=1), randn(T, k, seed=2)
    idx = select64(logits, k)
    ws = alloc_workspace(T, E, k, 1)
    out = torch.empty(T, E, device="cuda")
    bad = idx.clone()
    bad[3, 1], bad[4, 0] = -1, E
    s = Scoring(renorm=False)
    moe_gate_scored_backward(logits.cuda(), bad.int().cuda(), d.cuda(), s, out, ws)
    assert moe_get_status(ws) == abi.MOE_ERR_DEVICE_DATA
    q = scores64(logits, "sigmoid")
    each = d.double() * torch.gather(q * (1 - q), 1, bad.clamp(0, E - 1)) * (bad == idx)
    want = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, bad.clamp(0, E - 1), each)
    assert float((out.cpu().double() - want).abs().max()) <= 2.0 ** -20
    twice = idx.clone()
    twice[:, 1] = twice[:, 0]
    moe_gate_scored_backward(logits.cuda(), twice.int().cuda(), d.cuda(), s, out, ws)
    assert moe_get_status(ws) == 0
    want = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, twice, d.double() * torch.gather(q * (1 - q), 1, twice))
    assert float((out.cpu().double() - want).abs().max()) <= 2.0 ** -20


# --------------------------------------------------------------------------

def shape(**kw):
    a = dict(T=777, H=512, E=32, k=4, P=4, scoring=Scoring("sigmoid", 8, 4, 2, scale=1.5))
    return RouteShape(**{**a, **kw})


def test_plan_with_scores():
    s = shape(capacity=120)
    logits, bias = randn(s.T, s.E, seed=1), randn(s.E, seed=2, std=0.1)
    x = randn(s.T, s.H, seed=3).bfloat16().cuda()
    plan = RoutePlan(s)
    plan.route(logits.cuda(), bias.cuda())
    plan.dispatch(x)
    plan.combine(plan.packed)
    assert plan.status() == 0 and plan.launches_per_step() == 4
    idx = select64(logits, s.k, "sigmoid", 8, 4, 2, bias)
    assert torch.equal(plan.topk_idx.cpu().long(), idx)
    g = gates64(logits, idx, scale=1.5)
    kept = plan.layout.dst_row[:s.T * s.k].reshape(s.T, s.k).cpu() >= 0
    assert int((~kept).sum()) > 0
    want = x.cpu().double() * (g * kept).sum(1, keepdim=True)
    assert bool(((plan.y.cpu().double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-30).all())
    # backward through the same gate
    dy = randn(s.T, s.H, seed=4).bfloat16().cuda()
    plan.combine_backward(dy, plan.packed)
    plan.gate_backward(logits.cuda())
    ref = logits.double().requires_grad_()
    (gates64(ref, idx, scale=1.5) * plan.d_gates.cpu().double()).sum().backward()
    bound = backward_error(logits, idx, plan.d_gates.cpu(), s.E, "sigmoid", True, 1.5)
    assert bool(((plan.d_logits.cpu().double() - ref.grad).abs() <= bound).all())


def test_plan_reassigns_with_scores():
    s = shape(capacity=110, reassign=True)
    logits = randn(s.T, s.E, seed=1) + randn(s.E, seed=5)
    plan = RoutePlan(s)
    plan.route(logits.cuda())
    assert plan.status() == 0 and torch.equal(plan.topk_idx.cpu().long(), select64(logits, s.k, "sigmoid", 8, 4, 2))
    assert int(plan.layout.counts.max()) <= 110


def test_graph_with_scores():
    s = shape()
    g = RouteGraph(s)
    eo = randn(s.T * s.k, s.H, seed=9).bfloat16().cuda()
    for seed in (1, 2):
        logits, bias = randn(s.T, s.E, seed=seed), randn(s.E, seed=10 + seed, std=0.1)
        x = randn(s.T, s.H, seed=20 + seed).bfloat16().cuda()
        plan = g.step(logits.cuda(), x, eo, bias=bias.cuda())
        assert g.status() == 0
        assert torch.equal(plan.topk_idx.cpu().long(), select64(logits, s.k, "sigmoid", 8, 4, 2, bias))
        rows = plan.layout.src_pos[:s.T * s.k].long() // s.k
        assert torch.equal(plan.packed[:s.T * s.k], x[rows])


def test_pipeline_with_scores():
    s = shape()
    pipe = RoutePipeline(s)
    eo = randn(s.T * s.k, s.H, seed=9).bfloat16().cuda()
    batches = [(randn(s.T, s.E, seed=i).cuda(), randn(s.E, seed=50 + i, std=0.1).cuda(),
                randn(s.T, s.H, seed=90 + i).bfloat16().cuda()) for i in range(5)]
    torch.cuda.synchronize()
    for i, (logits, bias, x) in enumerate(batches):
        plan = pipe.step(logits, x, eo, bias=bias)
        pipe.synchronize()
        assert torch.equal(plan.topk_idx.cpu().long(), select64(logits.cpu(), s.k, "sigmoid", 8, 4, 2, bias.cpu()))
    assert pipe.status() == 0


def test_own_stream_and_two_at_once():
    """Two gates on two streams, each with its workspace, and one captured."""
    T, E, k = 3000, 64, 8
    s = Scoring("sigmoid", 8, 4, 2)
    made = []
    for i in range(2):
        st = torch.cuda.Stream()
        logits = randn(T, E, seed=i)
        with torch.cuda.stream(st):
            made.append((st, logits, gate(logits, k, s)))
    for st, logits, out in made:
        st.synchronize()
        assert torch.equal(out[0].cpu().long(), select64(logits, k, "sigmoid", 8, 4, 2))
    logits = randn(T, E, seed=3).cuda()
    ids, g = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    n, ws = torch.empty(E, dtype=torch.int32, device="cuda"), alloc_workspace(T, E, k, 1)
    call = lambda: moe_gate_scored(logits, k, s, None, ids, g, n, None, None, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (4, 5):
        logits.copy_(randn(T, E, seed=seed))
        ids.fill_(-1)
        graph.replay()
        assert torch.equal(ids.cpu().long(), select64(logits.cpu(), k, "sigmoid", 8, 4, 2))


def test_refusals_of_the_call():
    T, E, k = 6, 16, 4
    z = lambda *s, **kw: torch.zeros(*s, device="cuda", **kw)  # noqa: E731
    i32 = dict(dtype=torch.int32)
    good = dict(logits=z(T, E), k=k, scoring=Scoring(groups=4, top_groups=2, group_top=2), bias=z(E), topk_idx=z(T, k, **i32),
                gates=z(T, k), expert_counts=z(E, **i32), aux_loss=z(1, dtype=torch.float64), entropy=None,
                ws=alloc_workspace(T, E, k, 1))
    moe_gate_scored(**good)
    for name, bad in (("logits", z(T * E)), ("logits", z(E, T).T), ("logits", z(T, E).double()), ("bias", z(E - 1)),
                      ("bias", z(E).cpu()), ("topk_idx", z(T, k)), ("topk_idx", z(T, k - 1, **i32)),
                      ("gates", z(T, 2 * k)[:, ::2]), ("expert_counts", z(E - 1, **i32)), ("aux_loss", z(1)),
                      ("ws", z(8192, dtype=torch.uint8).int())):
        with pytest.raises(ValueError):
            moe_gate_scored(**{**good, name: bad})
    with pytest.raises(TypeError):
        moe_gate_scored(**{**good, "gates": [0.0] * 24})
    with pytest.raises(MoeError):
        moe_gate_scored(**{**good, "ws": z(64, dtype=torch.uint8)})
    with pytest.raises(MoeError):
        moe_gate_scored(**{**good, "scoring": Scoring(groups=5)})
    with pytest.raises(ValueError):
        moe_gate_scored(**good, bias_next=z(E + 1))
    back = dict(logits=z(T, E), topk_idx=z(T, k, **i32), d_gates=z(T, k), scoring=Scoring(), d_logits=z(T, E),
                ws=good["ws"])
    moe_gate_scored_backward(**back)
    for name, bad in (("topk_idx", z(T * k, **i32)), ("d_gates", z(T, k - 1)), ("d_logits", z(T, E - 1)),
                      ("d_logits", z(T, E).half())):
        with pytest.raises(ValueError):
            moe_gate_scored_backward(**{**back, name: bad})


def test_refusals_of_the_plan():
    plan = RoutePlan(RouteShape(T=4, H=64, E=8, k=2, P=1))
    logits, bias = torch.zeros(4, 8, device="cuda"), torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="only with scoring"):
        plan.route(logits, bias)
    plan = RoutePlan(RouteShape(T=4, H=64, E=8, k=2, P=1, scoring=Scoring()))
    with pytest.raises(ValueError, match="bias"):
        plan.route(logits, bias[:4])
    plan = RoutePlan(RouteShape(T=4, H=64, E=8, k=2, P=1, scoring=Scoring(groups=8, top_groups=1)))
    with pytest.raises(MoeError):
        plan.route(logits)  # one group of one expert does not hold two


@pytest.mark.parametrize("T", [70, 6000, 40000])
def test_scores_that_64_bits_make_equal(T):
    """A softmax score is exp(l - max) / sum in 64 bits, on every way to the
    answer: few near candidates or more than a warp's lanes, with a bias of
    zeros or without one, and in a group's value.  exp(-1.2e-16) is 1 - 2^-53;
    divided by the sums below it and 1 give the same score, a tie that goes to
    the lower id, while the product with 1 / sum, or no division, tells them
    apart.  The sums are whole: every order of adding gives them."""
    below = -1.2e-16
    for n in (3, 6, 48, 60):  # equal scores
        assert (1 - 2.0 ** -53) / n == 1 / n
        logits = torch.full((T, 64), -1000.0)
        logits[:, 1:n] = 0.0
        logits[:, 0] = below
        logits[1::2] = logits[1::2].roll(4, 1)
        k = min(n, 8)
        for bias in (None, torch.zeros(64)):
            idx, _ = check(logits, k, Scoring("softmax"), bias)
            assert torch.equal(idx.cpu().long(), torch.arange(k) + 4 * (torch.arange(T) % 2)[:, None])
    # groups by their best, and by the sum of two
    for two in (1, 2):
        logits = torch.full((T, 64), -1000.0)
        logits[:, 9], logits[:, 17], logits[:, 40] = below, 0.0, 0.0
        for bias in (None, torch.zeros(64)):
            idx, _ = check(logits, 2, Scoring("softmax", 8, 1, two), bias)
            assert torch.equal(idx.cpu().long(), torch.tensor([9, 8]).expand(T, 2))


def test_a_rate_that_nothing_takes_is_refused():
    logits, bias = torch.zeros(4, 8, device="cuda"), torch.zeros(8, device="cuda")
    plan = RoutePlan(RouteShape(T=4, H=64, E=8, k=2, P=1, scoring=Scoring()))
    for call in (plan.gate, plan.route):
        with pytest.raises(ValueError, match="bias_next"):
            call(logits, bias, bias_rate=1e-3)
        call(logits, bias, bias_next=bias, bias_rate=0.0)
    plan = RoutePlan(RouteShape(T=4, H=64, E=8, k=2, P=1))
    for call in (plan.gate, plan.route):
        with pytest.raises(ValueError, match="only with scoring"):
            call(logits, bias_rate=1e-3)
    with pytest.raises(ValueError, match="bias_next"):
        gate(logits, 2, Scoring(), bias, None, 1e-3)


def test_the_graph_s_bias_is_one_of_each_expert():
    """As RoutePlan.gate takes it: no single value for all experts, no other type."""
    graph = RouteGraph(RouteShape(T=4, H=64, E=8, k=2, P=1, scoring=Scoring()))
    bias = torch.linspace(0, 1, 8, device="cuda")
    graph.step(bias=bias)
    for bad in (bias[:1], bias[3], bias[:4], bias.double(), bias.expand(2, 8)):
        with pytest.raises(ValueError, match="bias"):
            graph.step(bias=bad)
    assert torch.equal(graph.bias, bias)
    with pytest.raises(ValueError, match="only with scoring"):
        RouteGraph(RouteShape(T=4, H=64, E=8, k=2, P=1)).step(bias=bias)
