"""The expert products on the GPU against the same products in 64 bits:
ragged groups (empty ones, one row, odd counts), tails of every axis, every
activation, bias, residual, the e4m3 operands, the saved layer, the
gradients, rows outside the groups, and the FFN they make."""
import pytest
import torch

from combine_moe_gate_warp_gb300 import (ExpertFFN, ExpertRows, RoutePlan, RouteShape, SavedLayer, abi,
                                         quantize_weights)
from expert_util import (BF16, act64, act_error, assert_near, decode64, encode_saved, grad64, grad_error, linear64,
                         normal, offsets_of, spans, sum_error)

pytestmark = pytest.mark.gpu

COUNTS = [0, 1, 15, 33, 0, 130, 257, 16, 0]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import combine_moe_gate_warp_gb300 as pkg
    pkg.build()


def rows_for(counts, mean):
    """Rows of buffers that hold these groups and make `mean` rows per expert:
    the library cuts its tiles by the rows that buffers hold, 32 wide for few
    of them and 256 wide for pairs of SMs for the most."""
    return max(sum(counts), mean * len(counts))


def padded(t, rows, fill=float("nan")):
    out = torch.full((rows, *t.shape[1:]), fill, dtype=t.dtype, device=t.device)
    out[:t.shape[0]] = t
    return out


@pytest.mark.parametrize("mean", [8, 300, 9000])
@pytest.mark.parametrize("K,N", [(64, 128), (8, 8), (72, 264), (520, 96), (1032, 520)])
def test_linear_plain(mean, K, N):
    counts = COUNTS if mean != 8 else [0, 1, 7, 0, 20, 33, 3]
    R, rows = sum(counts), rows_for(counts, mean)
    x, w = normal(R, K, seed=1), normal(len(counts), N, K, seed=2, std=K ** -0.5)
    r = ExpertRows(offsets_of(counts), rows=rows)
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    assert r.linear(padded(x, rows), w, out=out) is out
    assert r.status() == 0
    u, e = linear64(x, w, counts)
    assert_near(out[:R], u, e + BF16 * (u.abs() + e), "y")
    assert bool((out[R:] == 7.0).all()), "rows past the last expert's were written"


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("mean", [8, 300, 9000])
@pytest.mark.parametrize("bias,residual,save", [(True, False, False), (True, True, True), (False, True, False)])
def test_linear_epilogues(act, mean, bias, residual, save):
    counts, K, N = COUNTS, 200, 448
    if mean == 8:
        counts = [3, 0, 1, 40]
    R, rows, E = sum(counts), rows_for(counts, mean), len(counts)
    x, w = normal(R, K, seed=3), normal(E, N, K, seed=4, std=K ** -0.5)
    b = normal(E, N, seed=5) if bias else None
    cols = N // 2 if act == "swiglu" else N
    res = normal(R, cols, seed=6) if residual else None
    r = ExpertRows(offsets_of(counts), rows=rows)
    saved = r.new_saved(N) if save else None
    y = r.linear(padded(x, rows), w, bias=b, act=act, residual=None if res is None else padded(res, rows),
                 saved=saved)
    assert r.status() == 0
    u, e = linear64(x, w, counts, b)
    want, err = act64(u, act), act_error(u, e, act)
    if residual:
        want = want + res.double()
    err = err + 2.0 ** -23 * want.abs()
    assert_near(y[:R], want, err + BF16 * (want.abs() + err), "y")
    if save:
        check_saved(saved, u, e, R)


def check_saved(saved, u, e, R):
    """The scale is the smallest power of two that holds the block (up to the
    error e of u), and a code is the nearest: half a step is 2^-4 of the
    value, or 2^-10 of the scale among the subnormal codes."""
    scale = torch.pow(2.0, saved.scales[:R].double() - 127)
    top = u.abs().reshape(R, -1, 32).amax(2)
    slack = e.reshape(R, -1, 32).amax(2)
    assert bool((top - slack <= 448 * scale).all()), "a block's values pass its scale"
    assert bool((top + slack > 224 * scale)[scale > 2.0 ** -127].all()), "a block's scale is too large"
    got = decode64(saved.codes[:R], saved.scales[:R])
    half = 2.0 ** -4 * (u.abs() + e) + 2.0 ** -10 * scale.repeat_interleave(32, -1)
    assert_near(got, u, half + e, "saved")


@pytest.mark.parametrize("mean", [8, 300, 9000])
@pytest.mark.parametrize("act,K,N", [("none", 16, 24), ("swiglu", 400, 288), ("silu", 1040, 136)])
def test_linear_e4m3(mean, act, K, N):
    """x = zero + scale * code, w = scale * code: from the codes in 64 bits.
    The sums are fp32 (products of codes, then three fp32 steps)."""
    counts = COUNTS if mean != 8 else [5, 0, 1, 17, 40]
    R, rows, E = sum(counts), rows_for(counts, mean), len(counts)
    g = torch.Generator().manual_seed(9)
    # codes of magnitude up to 448, no NaN patterns
    def codes(*shape):
        return (torch.randn(*shape, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
    xq, wq = codes(R, K), codes(E, N, K)
    xs = (torch.rand(R, 2, generator=g) * 0.02 + 0.001).cuda()
    ws = torch.empty(E, N, 2, device="cuda")
    ws[..., 0] = (torch.rand(E, N, generator=g) * 1e-3 + 1e-4).cuda()
    ws[..., 1] = (wq.double().sum(2) * ws[..., 0].double()).float()
    r = ExpertRows(offsets_of(counts), rows=rows)
    y = r.linear(padded(xq.view(torch.uint8), rows, 0x7F), wq.view(torch.uint8), act=act,
                 x_scales=padded(xs, rows), w_scales=ws)
    assert r.status() == 0
    us, es = [], []
    for e, lo, hi in spans(counts):
        a, b = xq[lo:hi].double(), wq[e].double()
        s = xs[lo:hi, :1].double() * ws[e, :, 0].double()
        z = xs[lo:hi, 1:].double() * ws[e, :, 1].double()
        acc = a @ b.T
        us.append(s * acc + z)
        es.append(s * sum_error(K, a.abs() @ b.abs().T) + 2.0 ** -22 * ((s * acc).abs() + z.abs()))
    u, e = torch.cat(us), torch.cat(es)
    want, err = act64(u, act), act_error(u, e, act)
    assert_near(y[:R], want, err + BF16 * (want.abs() + err), "y")


@pytest.mark.parametrize("mean", [8, 300, 9000])
@pytest.mark.parametrize("K,N", [(128, 64), (8, 8), (264, 72), (96, 1000)])
def test_dgrad(mean, K, N):
    counts = COUNTS if mean != 8 else [0, 1, 7, 0, 20, 33, 3]
    R, rows, E = sum(counts), rows_for(counts, mean), len(counts)
    dy, w = normal(R, N, seed=11), normal(E, N, K, seed=12, std=N ** -0.5)
    r = ExpertRows(offsets_of(counts), rows=rows)
    out = torch.full((rows, K), 7.0, dtype=torch.bfloat16, device="cuda")
    r.dgrad(padded(dy, rows), w, out=out)
    assert r.status() == 0
    d, e = linear64(dy, w.mT, counts)
    assert_near(out[:R], d, e + BF16 * (d.abs() + e), "dx")
    assert bool((out[R:] == 7.0).all())


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
@pytest.mark.parametrize("mean", [8, 300, 9000])
@pytest.mark.parametrize("recompute", [True, False])
def test_dgrad_through_saved(act, mean, recompute):
    counts, K, N = ([3, 0, 1, 40] if mean == 8 else COUNTS), 160, 200
    R, rows, E = sum(counts), rows_for(counts, mean), len(counts)
    C = 2 * K if act == "swiglu" else K
    dy, w = normal(R, N, seed=13), normal(E, N, K, seed=14, std=N ** -0.5)
    codes, scales = encode_saved(normal(R, C, seed=15, std=1.5))
    saved = SavedLayer(padded(codes, rows, 0x7F), padded(scales, rows, 0xFF))
    r = ExpertRows(offsets_of(counts), rows=rows)
    a = torch.full((rows, K), 7.0, dtype=torch.bfloat16, device="cuda") if recompute else None
    du = r.dgrad(padded(dy, rows), w, act=act, saved=saved, a=a)
    assert r.status() == 0
    d, e = linear64(dy, w.mT, counts)
    u = decode64(codes, scales)
    want, err = grad64(u, d, act), grad_error(u, d, e, act)
    assert_near(du[:R], want, err + BF16 * (want.abs() + err), "du")
    if recompute:
        want = act64(u, act)
        err = act_error(u, torch.zeros_like(u), act)
        assert_near(a[:R], want, err + BF16 * (want.abs() + err), "a")
        assert bool((a[R:] == 7.0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts", [COUNTS, [64, 0, 63, 65, 128, 1], [700], [0, 0]])
@pytest.mark.parametrize("N,K", [(128, 128), (8, 8), (264, 72), (520, 392)])
def test_wgrad(counts, N, K, dtype):
    R, E = sum(counts), len(counts)
    dy, x = normal(R, N, seed=16), normal(R, K, seed=17)
    rows = R + 5
    r = ExpertRows(offsets_of(counts), rows=rows)
    dw, db = r.wgrad(padded(dy, rows), padded(x, rows), bias=True, dtype=dtype)
    assert r.status() == 0
    check_wgrad(dw, db, dy, x, counts, dtype)


def check_wgrad(dw, db, dy, x, counts, dtype):
    half = BF16 if dtype == torch.bfloat16 else 2.0 ** -24
    for e, lo, hi in spans(counts):
        d, v = dy[lo:hi].double(), x[lo:hi].double()
        want, err = d.T @ v, sum_error(hi - lo, d.abs().T @ v.abs())
        assert_near(dw[e], want, err + half * (want.abs() + err), f"dw[{e}]")
        want, err = d.sum(0), sum_error(hi - lo, d.abs().sum(0))
        assert_near(db[e], want, err + half * (want.abs() + err), f"db[{e}]")


@pytest.mark.parametrize("E,N,K", [(12, 512, 512), (40, 256, 264)])
def test_wgrad_many_tiles(E, N, K):
    """More tiles than blocks (several per block, both accumulators)."""
    counts = [(37 * e) % 190 for e in range(E)]
    R = sum(counts)
    dy, x = normal(R, N, seed=18), normal(R, K, seed=19)
    r = ExpertRows(offsets_of(counts), rows=R)
    dw, db = r.wgrad(dy, x, bias=True)
    assert r.status() == 0
    check_wgrad(dw, db, dy, x, counts, torch.bfloat16)


@pytest.mark.parametrize("mean", [40, 3000])
def test_linear_many_tiles(mean):
    counts = [(53 * e) % 400 + (700 if e == 5 else 0) for e in range(24)]
    rows = max(sum(counts), 24 * mean)
    R, K, N = sum(counts), 136, 1536
    x, w = normal(R, K, seed=20), normal(24, N, K, seed=21, std=K ** -0.5)
    r = ExpertRows(offsets_of(counts), rows=rows)
    y = r.linear(padded(x, rows), w)
    assert r.status() == 0
    u, e = linear64(x, w, counts)
    assert_near(y[:R], u, e + BF16 * (u.abs() + e), "y")
    dx = r.dgrad(y, w)
    d, e = linear64(y[:R], w.mT, counts)
    assert_near(dx[:R], d, e + BF16 * (d.abs() + e), "dx")


@pytest.mark.parametrize("counts,K,N", [
    ([4], 2048, 256), ([33], 2048, 4096), ([20], 1040, 8192), ([1000], 4096, 1024), ([512], 4096, 512),
    ([3, 0, 40, 1], 2048, 512), ([130, 5, 0, 200], 2056, 272)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_split_sums(counts, K, N, act):
    """Few tiles and a long k: blocks of a cluster share it and join their
    sums.  Forward with everything in the epilogue, the rows' gradient plain
    and through the saved layer, the weights' gradient."""
    R, E = sum(counts), len(counts)
    rows = R + 3
    x, w, b = normal(R, K, seed=60), normal(E, N, K, seed=61, std=K ** -0.5), normal(E, N, seed=62)
    cols = N // 2 if act == "swiglu" else N
    res = normal(R, cols, seed=63)
    r = ExpertRows(offsets_of(counts), rows=rows)
    can_save = N % 64 == 0
    saved = r.new_saved(N) if can_save else None
    out = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    r.linear(padded(x, rows), w, bias=b, act=act, residual=padded(res, rows), saved=saved, out=out)
    assert r.status() == 0
    u, e = linear64(x, w, counts, b)
    want, err = act64(u, act) + res.double(), act_error(u, e, act)
    err = err + 2.0 ** -23 * want.abs()
    assert_near(out[:R], want, err + BF16 * (want.abs() + err), "y")
    assert bool((out[R:] == 7.0).all())
    if can_save:
        check_saved(saved, u, e, R)
    # dgrad with the long axis as its k
    wt = normal(E, K, N, seed=64, std=K ** -0.5)
    dy = normal(R, K, seed=65)
    d, e = linear64(dy, wt.mT, counts)
    dx = r.dgrad(padded(dy, rows), wt)
    assert_near(dx[:R], d, e + BF16 * (d.abs() + e), "dx")
    if can_save:
        C = 2 * N if act == "swiglu" else N
        codes, scales = encode_saved(normal(R, C, seed=66, std=1.5))
        name = "gelu" if act == "none" else act
        du = r.dgrad(padded(dy, rows), wt, act=name, saved=SavedLayer(padded(codes, rows, 0x7F),
                                                                      padded(scales, rows, 0xFF)))
        u = decode64(codes, scales)
        want, err = grad64(u, d, name), grad_error(u, d, e, name)
        assert_near(du[:R], want, err + BF16 * (want.abs() + err), "du")
    assert r.status() == 0


@pytest.mark.parametrize("counts", [[4000], [2111], [1500, 0, 700], [64, 3000]])
@pytest.mark.parametrize("N,K", [(256, 256), (136, 72), (1024, 512)])
def test_wgrad_split(counts, N, K):
    """Many rows and few tiles: blocks share the rows of a tile."""
    R = sum(counts)
    dy, x = normal(R, N, seed=67), normal(R, K, seed=68)
    r = ExpertRows(offsets_of(counts), rows=R + 9)
    for dtype in (torch.bfloat16, torch.float32):
        dw, db = r.wgrad(padded(dy, R + 9), padded(x, R + 9), bias=True, dtype=dtype)
        assert r.status() == 0
        check_wgrad(dw, db, dy, x, counts, dtype)


@pytest.mark.parametrize("mean", [4, 900])
def test_256_experts(mean):
    """The largest number of experts, most with a few rows, some with none."""
    counts = [(e * 37) % 11 if e % 3 else 0 for e in range(256)]
    counts[200] = 400
    R, K, N = sum(counts), 136, 64
    rows = rows_for(counts, mean)
    x, w, dy = normal(R, K, seed=71), normal(256, N, K, seed=72, std=K ** -0.5), normal(R, N, seed=73)
    r = ExpertRows(offsets_of(counts), rows=rows)
    y, dx = r.linear(padded(x, rows), w), r.dgrad(padded(dy, rows), w)
    dw, db = r.wgrad(padded(dy, rows), padded(x, rows), bias=True)
    assert r.status() == 0
    u, e = linear64(x, w, counts)
    assert_near(y[:R], u, e + BF16 * (u.abs() + e), "y")
    d, e = linear64(dy, w.mT, counts)
    assert_near(dx[:R], d, e + BF16 * (d.abs() + e), "dx")
    check_wgrad(dw, db, dy, x, counts, torch.bfloat16)


@pytest.mark.parametrize("mean", [8, 9000])
def test_same_bits_twice(mean):
    """No result depends on timing."""
    counts = [50, 0, 31, 129]
    rows = rows_for(counts, mean)
    x, w = normal(210, 2048, seed=69), normal(4, 512, 2048, seed=70, std=0.02)
    r = ExpertRows(offsets_of(counts), rows=rows)
    xp = padded(x, rows, 0.0)
    y, dw = r.linear(xp, w)[:210].clone(), None
    for _ in range(5):
        assert torch.equal(r.linear(xp, w)[:210], y)
        again = r.wgrad(xp, xp, bias=True, dtype=torch.float32)
        assert dw is None or (torch.equal(again[0], dw[0]) and torch.equal(again[1], dw[1]))
        dw = again


@pytest.mark.parametrize("T", [1, 4, 33, 129, 1000])
@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
def test_plain_linear_and_backward(T, act):
    """One group (the shared experts): forward with bias and residual, and
    the gradients through the saved layer."""
    K, N = 328, 576
    cols = N // 2 if act == "swiglu" else N
    x, w, b, res = normal(T, K, seed=22), normal(N, K, seed=23, std=K ** -0.5), normal(N, seed=24), normal(T, cols, seed=25)
    r = ExpertRows(rows=T)
    saved = None if act == "none" else r.new_saved(N)
    y = r.linear(x, w, bias=b, act=act, residual=res, saved=saved)
    u, e = linear64(x, w[None], [T], b[None])
    want, err = act64(u, act) + res.double(), act_error(u, e, act)
    err = err + 2.0 ** -23 * want.abs()
    assert_near(y, want, err + BF16 * (want.abs() + err), "y")
    dy = normal(T, cols, seed=26)
    dx, dw, db = r.linear_backward(dy, x, w, act=act, saved=saved, bias=True)
    assert r.status() == 0
    du, slack = dy.double(), 0.0
    if saved is not None:
        du = grad64(decode64(saved.codes, saved.scales), dy.double(), act)
        # du is rounded to bf16 on its way into the products
        slack = BF16 * du.abs() + grad_error(decode64(saved.codes, saved.scales), dy.double(),
                                             torch.zeros_like(dy.double()), act)
    wd, xd = w.double(), x.double()
    for got, want, err in ((dx, du @ wd, slack @ wd.abs() if saved else 0, ),
                           (dw, du.T @ xd, slack.T @ xd.abs() if saved else 0),
                           (db, du.sum(0), slack.sum(0) if saved else 0)):
        n = N if got is dx else T
        mags = (du.abs() @ wd.abs() if got is dx else du.abs().T @ xd.abs() if got is dw else du.abs().sum(0))
        err = err + sum_error(n, mags * (1 + BF16))
        assert_near(got, want, err + BF16 * (want.abs() + err), "gradient")


def test_no_row_reads_another():
    """NaN and infinity in one expert's rows and weights, and in rows past R,
    stay there: forward, rows' gradient and weights' gradient."""
    counts, K, N = [20, 30, 65, 0, 9], 96, 160
    R, rows = sum(counts), sum(counts) + 40
    x, w, dy = normal(R, K, seed=27), normal(5, N, K, seed=28, std=0.1), normal(R, N, seed=29)
    x[20:50] = float("nan")
    dy[25] = float("inf")
    w[1] = float("nan")
    for mean in (8, 300, 9000):
        buf = max(rows, 5 * mean)
        r = ExpertRows(offsets_of(counts), rows=buf)
        xp, dp = padded(x, buf), padded(dy, buf, float("inf"))
        y, dx = r.linear(xp, w), r.dgrad(dp, w)
        dw, db = r.wgrad(dp, xp, bias=True)
        assert r.status() == 0
        clean = torch.ones(R, dtype=torch.bool, device="cuda")
        clean[20:50] = False
        for t in (y, dx):
            assert bool(torch.isfinite(t[:R][clean]).all()) and bool(torch.isnan(t[:R][~clean]).all())
        for e in (0, 2, 3, 4):
            assert bool(torch.isfinite(dw[e]).all()) and bool(torch.isfinite(db[e]).all())
        assert bool(torch.isnan(dw[1]).all()) and bool((db[1] == float("inf")).all())
        assert bool((dw[3] == 0).all()) and bool((db[3] == 0).all())


def test_saved_non_finite_and_zero_blocks():
    """A block with a NaN or an infinity decodes as NaN, a block of zeros as
    zeros, tiny values without overflow of the scale."""
    x = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(96, 8, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(96, dtype=torch.bfloat16, device="cuda")
    b[3], b[40] = float("nan"), float("inf")
    b[64:] = 2.0 ** -130
    r = ExpertRows(rows=4)
    s = r.new_saved(96)
    r.linear(x, w, bias=b, act="silu", saved=s)
    v = decode64(s.codes, s.scales)
    assert bool((s.scales[:, :2] == 255).all())
    # 2^-130 at the smallest scale 2^-127 is the code of 2^-3
    assert bool((s.scales[:, 2] == 0).all()) and bool((v[:, 64:] == 2.0 ** -130).all())
    b.zero_()
    r.linear(x, w, bias=b, act="silu", saved=s)
    assert bool((decode64(s.codes, s.scales) == 0).all()) and bool((s.codes & 0x7F == 0).all())
    # the largest finite values: amax 1.75 * 2^127 gives 448 * 2^119
    b.fill_(1.75 * 2.0 ** 127)
    r.linear(x, w, bias=b, act="silu", saved=s)
    assert bool((s.scales == 119 + 127).all()) and bool((decode64(s.codes, s.scales) == 1.75 * 2.0 ** 127).all())
    b.fill_(1.875 * 2.0 ** 127)
    r.linear(x, w, bias=b, act="silu", saved=s)
    assert bool((s.scales == 120 + 127).all()) and bool((decode64(s.codes, s.scales) == 1.875 * 2.0 ** 127).all())


def test_bad_offsets_are_recorded():
    """An expert whose offsets are negative, pass the rows, decrease or start
    below an earlier one is empty, the others are computed, and the status
    tells."""
    K = N = 64
    x, w = normal(100, K, seed=30), normal(3, N, K, seed=31, std=0.1)
    for off in ([0, 40, 30, 100], [0, 40, 101, 100], [-1, 40, 70, 100]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        r = ExpertRows(o, rows=100)
        y = torch.full((100, N), 7.0, dtype=torch.bfloat16, device="cuda")
        r.linear(x, w, out=y)
        assert r.status() == abi.MOE_ERR_DEVICE_DATA and r.status() == 0
        dw, db = r.wgrad(y, x, bias=True)
        assert r.status() == abi.MOE_ERR_DEVICE_DATA
        for e in range(3):
            lo, hi = off[e], off[e + 1]
            if lo < max([0] + off[:e]) or hi < lo or hi > 100:
                assert bool((dw[e] == 0).all()) and bool((db[e] == 0).all())
            else:
                u, err = linear64(x[lo:hi], w[e: e + 1], [hi - lo])
                assert_near(y[lo:hi], u, err + BF16 * (u.abs() + err), "y")


def test_nothing_to_do():
    r = ExpertRows(offsets_of([0, 0]), rows=0)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = normal(2, 32, 64, seed=1)
    assert r.linear(e, w).shape == (0, 32)
    assert r.dgrad(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), w).shape == (0, 64)
    dw, db = r.wgrad(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), e, bias=True)
    assert bool((dw == 0).all()) and bool((db == 0).all()) and r.status() == 0


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_ffn_gradients_against_differences(act):
    """The FFN's gradients against the formulas in 64 bits on the layer it
    saved, and the loss's change along a direction of each argument."""
    counts, H, F = [70, 0, 33, 150], 128, 96
    R, E, N = sum(counts), 4, 192 if act == "swiglu" else 96
    x, dy = normal(R, H, seed=32), normal(R, H, seed=33)
    w1, w2 = normal(E, N, H, seed=34, std=H ** -0.5), normal(E, H, F, seed=35, std=F ** -0.5)
    b1, b2 = normal(E, N, seed=36, std=0.3), normal(E, H, seed=37, std=0.3)
    r = ExpertRows(offsets_of(counts), rows=R)
    ffn = ExpertFFN(r, w1, w2, b1=b1, b2=b2, act=act, dtype=torch.float32)
    ffn.forward(x)
    g = ffn.backward(dy, x)
    assert r.status() == 0

    def loss(x, w1, w2, b1, b2):
        total = 0.0
        for e, lo, hi in spans(counts):
            a = act64(x[lo:hi] @ w1[e].T + b1[e], act)
            total = total + (dy[lo:hi].double() * (a @ w2[e].T + b2[e])).sum()
        return total

    args = [t.double() for t in (x, w1, w2, b1, b2)]
    for i, got in enumerate((g.dx, g.dw1, g.dw2, g.db1, g.db2)):
        d = torch.randn(args[i].shape, generator=torch.Generator().manual_seed(40 + i), dtype=torch.float64).cuda()
        h = 1e-5
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + h * d, args[i] - h * d
        diff = (loss(*up) - loss(*dn)) / (2 * h)
        mine = (got.double() * d).sum()
        # the saved layer's values are off by up to 2^-4 each, at random:
        # the inner product over many of them is off by a few percent of its
        # own scale, |g| |d| / sqrt(n) per independent term
        scale = (got.double() * d).square().sum().sqrt()
        assert abs(float(mine - diff)) <= 0.3 * float(scale), (i, float(mine), float(diff), float(scale))


def test_ffn_between_dispatch_and_combine():
    """The path in one piece: route, dispatch, experts, combine, against the
    same in 64 bits from the plan's own routing."""
    T, H, E, k, F = 300, 256, 8, 2, 128
    plan = RoutePlan(RouteShape(T=T, H=H, E=E, k=k, P=4), "cuda")
    x = normal(T, H, seed=50)
    plan.route(torch.randn(T, E, generator=torch.Generator().manual_seed(51)).cuda())
    plan.dispatch(x)
    w1, w2 = normal(E, 2 * F, H, seed=52, std=H ** -0.5), normal(E, H, F, seed=53, std=F ** -0.5)
    rows = ExpertRows.of(plan)
    ffn = ExpertFFN(rows, w1, w2)
    plan.combine(ffn.forward(plan.packed))
    assert plan.status() == 0
    idx, gates = plan.topk_idx.long(), plan.gates.double()
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for j in range(k):
        for e in range(E):
            at = idx[:, j] == e
            a = act64(x[at].double() @ w1[e].double().T, "swiglu")
            y = a @ w2[e].double().T
            want[at] += gates[at, j: j + 1] * y
            # roundings to bf16: a, y
            size[at] += gates[at, j: j + 1] * (1.1 * a.abs() @ w2[e].double().abs().T + y.abs())
    assert_near(plan.y, want, BF16 * (1.05 * size + want.abs()), "y")


@pytest.mark.parametrize("T", [0, 1, 77])
def test_fp8_dispatch_into_the_experts(T):
    """The FP8 dispatch's rows and scales go straight into a product: against
    the same codes and scales in 64 bits; a batch without tokens is fine."""
    H, E, k, N = 160, 8, 2, 96
    plan = RoutePlan(RouteShape(T=T, H=H, E=E, k=k, P=4, fp8=abi.MOE_FP8_PER_TOKEN), "cuda")
    plan.route(torch.randn(T, E, generator=torch.Generator().manual_seed(81)).cuda())
    plan.dispatch(normal(T, H, seed=82))
    codes, scales = quantize_weights(normal(E, N, H, seed=83, std=H ** -0.5))
    y = ExpertRows.of(plan).linear(plan.packed, codes, x_scales=plan.scales, w_scales=scales)
    assert plan.status() == 0 and y.shape == (T * k, N)
    off = plan.layout.offsets.tolist() if T else [0] * (E + 1)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        q, c = plan.packed[lo:hi].view(torch.float8_e4m3fn).double(), codes[e].view(torch.float8_e4m3fn).double()
        s, z = plan.scales[lo:hi, :1].double(), plan.scales[lo:hi, 1:].double()
        acc, mags = q @ c.T, q.abs() @ c.abs().T
        ws, total = scales[e, :, 0].double(), scales[e, :, 1].double()
        want = s * ws * acc + z * total
        err = s * ws * sum_error(H, mags) + 2.0 ** -22 * ((s * ws * acc).abs() + (z * total).abs())
        assert_near(y[lo:hi], want, err + BF16 * (want.abs() + err), "y")
        # the sums the weights carry are their own
        assert_near(total, ws * c.sum(1), 2.0 ** -23 * (ws * c.sum(1)).abs() + 1e-30, "sum")


@pytest.mark.parametrize("T,K,N,call", [(40, 256, 256, "linear"), (40, 256, 256, "dgrad"), (300, 256, 128, "wgrad"),
                                        (4, 2048, 256, "linear"), (6000, 256, 2048, "linear"),
                                        (6000, 2048, 2048, "wgrad")])
def test_waits_expire_with_timeout_status(T, K, N, call):
    """The first load of a product is left out (a workspace hook, from the
    host): its waits run out after their limit of 1 s, the call ends with
    MOE_ERR_TIMEOUT, and the next one is right.  One SM, blocks that share k,
    and pairs."""
    x, w, dy = normal(T, K, seed=91), normal(N, K, seed=92, std=K ** -0.5), normal(T, N, seed=93)
    r = ExpertRows(rows=T)
    run = {"linear": lambda: r.linear(x, w), "dgrad": lambda: r.dgrad(dy, w), "wgrad": lambda: r.wgrad(dy, x)[0]}[call]
    want = run()
    assert r.status() == 0
    r.ws.view(torch.int32)[7] = 1  # inject_skip_load (byte offset 28)
    run()
    assert r.status() == abi.MOE_ERR_TIMEOUT
    assert int(r.ws.view(torch.int32)[7].item()) == 0  # the hook was consumed
    assert torch.equal(run(), want) and r.status() == 0
