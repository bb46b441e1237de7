"""Routing by scores where the scores are close: exact ties beside near ones,
in the experts and in the groups' values.  A token is excused from the exact
answer only where its own choice hangs on values that 64 bits cannot order,
and how many those are follows from the inputs alone."""
import pytest
import torch

from combine_moe_gate_warp_gb300 import Scoring, alloc_workspace, moe_gate_scored, moe_get_status
from scored_util import scores64, select64

pytestmark = pytest.mark.gpu

def nearest(logits, s, bias):
    """[T, 1]: exp() is off by a step of 2^-52 of itself in this library and in
    that one, a score by 3 half steps more, a value and the sum of two by
    another each: 2^-50 in all, of the largest score and bias, so two values
    nearer than 2^-49 of that may come out in either order."""
    top = scores64(logits, s.score).amax(1, keepdim=True)
    return 2.0 ** -49 * (top + (0 if bias is None else bias.abs().max().double()))


@pytest.fixture(scope="module", autouse=True)
def _built():
    import combine_moe_gate_warp_gb300 as pkg
    pkg.build()


def randn(*shape, seed, std=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std


def values64(logits, s, bias):
    return scores64(logits, s.score) + (0 if bias is None else bias.double())


def group_sums(v, s):
    return v.reshape(v.shape[0], s.groups, -1).sort(2, descending=True)[0][:, :, :s.group_top].sum(2)


def open_choices(logits, k, s, bias):
    """(groups, experts) [T] each: whether the choice of the groups, or of the
    experts of these groups, hangs on values nearer than that which do not
    come from equal logits with equal biases."""
    T, E = logits.shape
    v, eps, b = values64(logits, s, bias), nearest(logits, s, bias), torch.zeros(E) if bias is None else bias
    groups = torch.zeros(T, dtype=torch.bool)
    kept = torch.ones(T, E, dtype=torch.bool)
    if s.top_groups < s.groups:
        per = E // s.groups
        g = group_sums(v, s)
        last, first = (g.sort(1, descending=True)[0][:, i:i + 1] for i in (s.top_groups - 1, s.top_groups))
        near = (g >= first - eps) & (g <= last + eps)  # the border's groups, if its two sides are near
        at = v.reshape(T, s.groups, per).argsort(dim=2, descending=True, stable=True)[:, :, :s.group_top]
        parts = (logits.reshape(T, s.groups, per).gather(2, at), b.reshape(1, s.groups, per).expand(T, -1, -1).gather(2, at))
        alike = torch.ones(T, dtype=torch.bool)
        for p in parts:
            low = torch.where(near[..., None], p, float("inf")).amin(1)
            alike &= (low == torch.where(near[..., None], p, float("-inf")).amax(1)).all(1)
        groups = (last - first <= eps)[:, 0] & ~alike
        order = g.argsort(dim=1, descending=True, stable=True)[:, :s.top_groups]
        kept = torch.zeros(T, s.groups, dtype=torch.bool).scatter_(1, order, True).repeat_interleave(per, 1)
    v = torch.where(kept, v, float("-inf"))
    order = v.argsort(dim=1, descending=True, stable=True)[:, :k + 1]
    top, l, c = v.gather(1, order), logits.gather(1, order), b.expand(T, E).gather(1, order)
    alike = (l.diff(dim=1) == 0) & (c.diff(dim=1) == 0)
    return groups, ((-top.diff(dim=1) <= eps) & ~alike).any(1)


def check(logits, k, s, bias=None, most=0.0):
    T, E = logits.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    gates, n = torch.empty(T, k, device="cuda"), torch.empty(E, dtype=torch.int32, device="cuda")
    ws = alloc_workspace(T, E, k, 1)
    moe_gate_scored(logits.cuda(), k, s, None if bias is None else bias.cuda(), idx, gates, n, None, None, ws)
    assert moe_get_status(ws) == 0
    got = idx.cpu().long()
    assert int(got.min()) >= 0 and int(got.max()) < E
    assert bool((got.sort(1)[0].diff(dim=1) > 0).all()), "an expert twice"
    want = select64(logits, k, s.score, s.groups, s.top_groups, s.group_top, bias)
    groups, experts = open_choices(logits, k, s, bias)
    free = groups | experts
    assert float(free.float().mean()) <= most, f"{float(free.float().mean())} of the tokens cannot be decided"
    wrong = (got != want).any(1)
    assert not bool((wrong & ~free).any()), f"{int((wrong & ~free).sum())} of {T} tokens"
    # what an open choice leaves fixed: the values of the selected, in order,
    # and that their groups are among the best
    v, eps = values64(logits, s, bias), nearest(logits, s, bias)
    x = v.gather(1, got)
    assert bool((x.diff(dim=1) <= eps).all())
    assert bool(((x - v.gather(1, want)).abs() <= eps)[~groups].all())
    if s.top_groups < s.groups:
        g, of = group_sums(v, s), got // (E // s.groups)
        cut = g.sort(1, descending=True)[0][:, s.top_groups - 1:s.top_groups]
        assert bool((g.gather(1, of) >= cut - eps).all())
        assert int((torch.nn.functional.one_hot(of, s.groups).sum(1) > 0).sum(1).max()) <= s.top_groups


SHAPES = [(700, 64, 8, 8, 4, 2), (700, 256, 8, 16, 6, 2), (6000, 64, 6, 8, 4, 1), (40000, 64, 8, 8, 4, 2),
          (500, 60, 4, 1, 1, 1), (40000, 64, 8, 32, 9, 2), (5000, 256, 8, 128, 40, 2), (40000, 64, 4, 32, 3, 1),
          (6000, 128, 16, 1, 1, 1), (39003, 48, 16, 1, 1, 1), (5003, 192, 5, 12, 4, 1), (300, 96, 12, 12, 5, 2)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,top,two", SHAPES)
def test_neighbours_a_few_steps_apart(T, E, k, groups, top, two, score):
    """Logits a few steps of fp32 apart, or some tens of them (the kernel's
    margin), many of them equal.  Between experts nothing is open: a step of a
    logit of 1/2 or more is 2^-24, and moves its score by more than 2^-37.
    Sums of two of (i, j) and (p, q) steps, i + j = p + q, differ by the
    square of a step, 2^-48 and less: those alone are open, less often the
    further the steps go (counted from the inputs)."""
    s = Scoring(score, groups, top, two)
    base = randn(T, 1, seed=1).bfloat16().float().expand(T, E).contiguous().abs() + 0.5
    for reach, share in ((3, 0.5), (60, 0.02), (2000, 1e-3)):
        steps = torch.randint(-reach, reach + 1, (T, E), generator=torch.Generator().manual_seed(reach))
        close = (base.view(torch.int32) + steps.int()).view(torch.float32)
        check(close, k, s, None, share if two == 2 else 0.0)
        check(close, k, s, torch.zeros(E), share if two == 2 else 0.0)
        # biases in steps of 2^-10: still ties, and fp64 holds the sums apart
        bias = torch.randint(-2, 3, (E,), generator=torch.Generator().manual_seed(4)).float() * 2.0 ** -10
        check(close, k, s, bias, share if two == 2 else 0.0)
        # biases beside the steps: at most a few in a thousand are open
        check(close, k, s, randn(E, seed=4, std=1e-7), share if two == 2 else 1e-3)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,top,two", SHAPES)
def test_values_on_a_level(T, E, k, groups, top, two, score):
    """Scores that differ, whose sums with the bias do not, to fp32; and
    softmax logits so near that many are equal."""
    s = Scoring(score, groups, top, two)
    if score == "sigmoid":
        bias = randn(E, seed=5, std=0.1)
        check(torch.log((0.5 - bias) / (0.5 + bias)).expand(T, E) + randn(T, 1, seed=7, std=1e-3), k, s, bias, 1e-3)
    else:
        check(randn(E, seed=6, std=1e-6).expand(T, E) + randn(T, 1, seed=7, std=1e-3), k, s, None, 1e-3 if two == 2 else 0.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_drawn_shapes(score):
    """Drawn sizes, groups and biases on logits as bf16 leaves them: every id
    as in 64 bits.  Without a bias two sums of two may be open; with one a
    handful of values in a million."""
    g = torch.Generator().manual_seed(11)
    pick = lambda *c: c[int(torch.randint(0, len(c), (1,), generator=g))]
    for n in range(60):
        groups, per = pick(1, 2, 3, 4, 5, 8, 12, 16, 32), pick(1, 2, 3, 4, 7, 8, 16)
        E = groups * per
        if E > 256:
            continue
        top = int(torch.randint(1, groups + 1, (1,), generator=g))
        k = min(int(torch.randint(1, 17, (1,), generator=g)), top * per)
        T = pick(50, 3000, 9000, 40000)
        s = Scoring(score, groups, top, 2 if per > 1 and n % 2 else 1)
        logits = (randn(T, E, seed=n) * pick(0.3, 1.0, 3.0)).bfloat16().float()
        bias = pick(None, 1e-4, 0.02, 1.0)
        check(logits, k, s, None if bias is None else randn(E, seed=n, std=bias), 1e-3)


@pytest.mark.parametrize("T", [40, 6000, 40000])
def test_three_near_values_in_a_group_of_two(T):
    """A group's two best are the two equal ones above a near third, which
    comes first by its id and takes the place of the first in fp32."""
    for score, high, low in (("sigmoid", 30.0, 20.0), ("sigmoid", 1.5, 1.5 - 2.0 ** -23), ("softmax", 1.5, 1.5 - 2.0 ** -23)):
        logits = torch.full((T, 24), -9.0)
        logits[:, 1], logits[:, 4] = high, low                    # high + low
        logits[:, 9], logits[:, 10], logits[:, 12] = low, high, high  # high + high
        logits[1::2] = logits[1::2].roll(8, 1)
        s = Scoring(score, 3, 1, 2)
        check(logits, 4, s)
        check(logits, 4, s, torch.zeros(24))
        assert torch.equal(select64(logits, 1, score, 3, 1, 2)[:, 0], 10 + 8 * (torch.arange(T) % 2))
