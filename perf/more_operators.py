"""Scored routing and the 4-bit path behind it, as they are measured.

Beside the softmax gates, the 8-bit transport and the experts' bf16 and e4m3
products of the routing path stand

  gate           routing by scores: sigmoid or softmax scores of every expert,
                 a bias that only the selection sees, groups of experts of
                 which the best are kept, the k best experts of these, their
                 scores renormalised and scaled as gates; the rows of each
                 expert and the bias for the next batch
  gate_backward  the gradient of these gates with respect to the logits
  dispatch       a batch routed by scores and its token rows packed by expert
                 as 4-bit values that share a power of two for 32 of them
  linear         y[r] = act(W[e] x[r] + b[e]) for the packed rows r of each
                 expert e from 4-bit rows and weights; from bf16 rows the call
                 first brings them to 4 bits

Shapes are those of the routing workloads and their tests (hidden sizes 512 ..
5120, 8 .. 64 experts, up to the 256 that the path allows, top-2 and top-8,
one token to a long prompt) with generic inner sizes.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32  # values that share a power of two
TINY = 1e-20  # beside the sum of the selected scores


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _case(name, op, **kw):
    return dict(name=name, op=op, **kw)


def listed():
    return [
        # 16 sequences decoding: one call of a few microseconds
        _case("gate decode", "gate", T=16, E=64, k=8, score="sigmoid", groups=8, top_groups=4, group_top=2, renorm=True,
              scale=2.0, bias=True, rate=0.0),
        # a training batch over the most experts the path takes, the bias moved towards balance
        _case("gate train", "gate", T=16384, E=256, k=8, score="sigmoid", groups=16, top_groups=6, group_top=2,
              renorm=True, scale=1.5, bias=True, rate=0.001),
        # one long prompt batch through fine-grained experts
        _case("gate prompt", "gate", T=262144, E=64, k=8, score="sigmoid", groups=8, top_groups=4, group_top=2,
              renorm=True, scale=2.0, bias=True, rate=0.0),
        # softmax scores, groups by their best expert, gates as they are; an odd number of everything
        _case("gate softmax", "gate", T=50021, E=60, k=6, score="softmax", groups=5, top_groups=3, group_top=1,
              renorm=False, scale=4.0, bias=False, rate=0.0),
        # the backward pass of a small odd batch, and of a large one through all experts' softmax
        _case("gate backward odd", "gate_backward", T=1021, E=60, k=6, score="sigmoid", renorm=True, scale=2.0),
        _case("gate backward large", "gate_backward", T=131072, E=128, k=4, score="softmax", renorm=True, scale=1.0),
        # a decode batch on its way to the experts
        _case("dispatch decode", "dispatch", T=48, E=64, k=2, H=4096, score="sigmoid", groups=8, top_groups=4,
              group_top=2, renorm=True, scale=1.0, bias=True),
        # a prompt batch on its way to the experts
        _case("dispatch prompt", "dispatch", T=65536, E=64, k=2, H=4096, score="sigmoid", groups=8, top_groups=4,
              group_top=2, renorm=True, scale=1.0, bias=True),
        # one token through a shared expert: the weights' bytes
        _case("linear one token", "linear", T=1, K=4096, N=8192, act="gelu", bias=True, residual=False, rows="bf16"),
        # 16 sequences decoding through fine-grained experts
        _case("linear decode", "linear", T=16, k=8, E=32, skew=0.5, K=2048, N=4096, act="swiglu", bias=False,
              residual=False, rows="fp4"),
        # nothing fills a tile or a group of scales
        _case("linear odd", "linear", T=1021, k=3, E=7, skew=1.0, K=1056, N=1416, act="silu", bias=True,
              residual=True, rows="bf16"),
        # a prompt batch through wide experts
        _case("linear prompt", "linear", T=16384, k=4, E=16, skew=0.25, K=5120, N=4096, act="swiglu", bias=True,
              residual=False, rows="fp4"),
    ]


def _log(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / mult)) * mult))


def _scoring(rng, c):
    """Score, groups and gates of a drawn case."""
    per = rng.choice((1, 2, 4, 6, 8, 16))
    groups = rng.randint(-(-4 // per), 256 // per if per > 1 else 64)
    c["E"] = groups * per
    c["k"] = min(rng.choice((1, 2, 2, 3, 4, 6, 8, 8, 16)), c["E"])
    least = -(-c["k"] // per)  # groups that hold k experts
    c.update(groups=groups, top_groups=rng.randint(least, groups), group_top=min(rng.choice((1, 2)), per),
             score=rng.choice(("sigmoid", "softmax")), scale=rng.choice((1.0, 1.5, 2.0)), bias=rng.random() < 0.7)
    c["renorm"] = c["k"] > 1 and rng.random() < 0.7  # one gate renormalised is a constant


def draw(rng):
    while True:
        op = rng.choice(("gate", "gate", "gate_backward", "dispatch", "linear", "linear"))
        c = dict(op=op)
        if op in ("gate", "gate_backward", "dispatch"):
            _scoring(rng, c)
        if op == "gate":
            c.update(T=_log(rng, 1, 262144), rate=rng.choice((0.0, 0.001)) if c["bias"] else 0.0)
        elif op == "gate_backward":
            c["T"] = _log(rng, 1, 131072)
        elif op == "dispatch":
            c.update(T=_log(rng, 1, 65536), H=_log(rng, 256, 5120, 32))
        else:
            c["T"] = _log(rng, 1, 16384)
            if rng.random() < 0.75:
                c.update(E=rng.choice((4, 7, 8, 16, 32, 64)), k=rng.choice((1, 2, 2, 3, 4, 6, 8)),
                         skew=rng.choice((0.0, 0.25, 0.5, 1.0)))
                if c["k"] > c["E"]:
                    continue
            act = rng.choice(("none", "silu", "gelu", "swiglu"))
            c.update(K=_log(rng, 256, 5120, 32), N=_log(rng, 256, 8192, 16), act=act, bias=rng.random() < 0.5,
                     residual=rng.random() < 0.3, rows=rng.choice(("bf16", "fp4")))
        w, most = work(c), {w["op"]: work(w) for w in listed()}[op]
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def _counts(case):
    """Rows of the experts, hottest first: T*k assignments shared out in
    proportion to rank^-skew."""
    E, A = case["E"], case["T"] * case["k"]
    share = np.arange(1, E + 1, dtype=np.float64) ** -case["skew"]
    share = share / share.sum() * A
    n = np.floor(share).astype(np.int64)
    n[np.argsort(-(share - n), kind="stable")[: A - int(n.sum())]] += 1
    return n


def _rows(c):
    """Packed rows, experts that have any, experts."""
    if "E" not in c:
        return c["T"], 1, 1
    n = _counts(c)
    return int(n.sum()), int((n > 0).sum()), c["E"]


def work(case):
    c, op = case, case["op"]
    T = c["T"]
    if op == "gate":
        E, k = c["E"], c["k"]
        return {"bytes": 4 * T * E + 8 * T * k + 4 * E * (1 + c["bias"] + (c["rate"] != 0)) + 8,
                "flops": T * (4 * E + 2 * k)}
    if op == "gate_backward":
        E, k = c["E"], c["k"]
        read = E if c["score"] == "softmax" else k  # logits of a token that its gradient depends on
        return {"bytes": 4 * T * (read + E) + 8 * T * k, "flops": T * (4 * read + 6 * k)}
    if op == "dispatch":
        E, k, H = c["E"], c["k"], c["H"]
        return {"bytes": 4 * T * E + 2 * T * H + 2 * T * k * H + 8 * T * k, "flops": T * (4 * E + 4 * H)}
    K, N = c["K"], c["N"]
    out = N // 2 if c["act"] == "swiglu" else N
    R, live, _ = _rows(c)
    four = K // 2 + K // BLOCK
    b = R * (2 * K if c["rows"] == "bf16" else four) + live * N * four + 2 * R * out
    b += (2 * live * N if c["bias"] else 0) + (2 * R * out if c["residual"] else 0)
    return {"bytes": b, "flops": 2 * R * K * N}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _pitch(K):
    """Scale bytes of a row of K values: one for 32, rows a multiple of 16 bytes apart."""
    return (K + 511) // 512 * 16


def _power(n):
    """2^n in fp32 for whole n from -127 to 127, bit for bit (pow() is not)."""
    return torch.where(n > -127, (n + 127) << 23, 1 << 22).int().view(torch.float32)


def _fp4(v):
    """Rows [.., K] as 4-bit values: e2m1 codes, two to a byte, the even
    column in the low half [.., K / 2], and for 32 consecutive columns the
    exponent byte of the smallest power of two that brings them to 6 or less
    (the byte is the exponent + 127) [.., pitch]."""
    b = v.float().unflatten(-1, (-1, BLOCK))
    m, e = torch.frexp(b.abs().amax(-1))  # amax = m * 2^e, 0.5 <= m < 1; 6 = 0.75 * 2^3
    e = torch.where(m <= 0.75, e - 3, e - 2).clamp(min=-127)
    q = (b * _power(-e[..., None])).flatten(-2)
    a = q.abs()
    # the halfway points between the values 0, 0.5, 1, 1.5, 2, 3, 4, 6 go to the even code
    n = (a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    n = n | (torch.signbit(q).byte() << 3)
    scales = torch.zeros(*v.shape[:-1], _pitch(v.shape[-1]), dtype=torch.uint8, device=v.device)
    scales[..., : e.shape[-1]] = (e + 127).byte()
    return n[..., 0::2] | (n[..., 1::2] << 4), scales


def _from_fp4(codes, scales):
    """The values that _fp4's codes stand for, in fp32."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat((table, -table))
    v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()].unflatten(-1, (-1, BLOCK))
    return (v * _power(scales[..., : v.shape[-2], None].int() - 127)).flatten(-2)


def _logits(c, g):
    """Router logits: some experts are more popular than others."""
    popular = torch.randn(c["E"], generator=g, device="cuda") * 0.5
    return torch.randn(c["T"], c["E"], generator=g, device="cuda") + popular


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).bfloat16()

    s = dict(op=op, case=c)
    if op != "linear":
        s["logits"] = _logits(c, g)
        s["bias"] = None
        if c.get("bias"):
            spread = 0.05 if c["score"] == "sigmoid" else 0.5 / c["E"]
            s["bias"] = torch.randn(c["E"], generator=g, device="cuda") * spread
    if op == "gate_backward":
        # any k experts of a token, in any order: here those of its largest logits
        s["idx"] = torch.sort(s["logits"], dim=1, descending=True, stable=True)[1][:, : c["k"]].int().contiguous()
        s["d_gates"] = torch.randn(c["T"], c["k"], generator=g, device="cuda")
    if op == "dispatch":
        # token rows of different sizes
        size = torch.exp(torch.randn(c["T"], 1, generator=g, device="cuda") * 0.5)
        s["x"] = (normal(c["T"], c["H"]).float() * size).bfloat16()
    if op != "linear":
        return s
    K, N = c["K"], c["N"]
    E = c.get("E", 1)
    s["act"] = c["act"]
    if "E" in c:
        n = _counts(c)[np.random.default_rng(seed).permutation(E)]
        off = np.concatenate(([0], np.cumsum(n)))
        s["most"] = int(n.max())
        s["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
    R = s["R"] = _rows(c)[0]
    x = normal(R, K)
    s["x"], s["x_scales"] = _fp4(x) if c["rows"] == "fp4" else (x, None)
    s["w"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s["w_scales"] = torch.empty(E, N, _pitch(K), dtype=torch.uint8, device="cuda")
    for e in range(E):
        s["w"][e], s["w_scales"][e] = _fp4(normal(N, K, std=K ** -0.5))
    s["b"] = normal(E, N, std=0.5) if c["bias"] else None
    s["residual"] = normal(R, N // 2 if c["act"] == "swiglu" else N) if c["residual"] else None
    if "E" not in c:
        for name in ("w", "w_scales", "b"):
            s[name] = None if s[name] is None else s[name][0]
    return s


# --------------------------------------------------------------------------
# the plain form
# --------------------------------------------------------------------------

def _silu(u):
    return u / (1 + torch.exp(-u))


def _act(u, act):
    if act == "silu":
        return _silu(u)
    if act == "gelu":
        return 0.5 * u * (1 + torch.erf(u * 0.5 ** 0.5))
    if act == "swiglu":
        gate, up = u.chunk(2, -1)
        return _silu(gate) * up
    return u


def _scores(logits, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_gate(s):
    """(expert ids [T, k], gates [T, k]).  Which of two experts is the better
    one is told in 64 bits: scores that 32 bits cannot tell apart are common."""
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    score = _scores(s["logits"].double(), c["score"])
    v = score if s["bias"] is None else score + s["bias"].double()
    in_group = torch.sort(v.reshape(T, G, E // G), dim=2, descending=True)[0]
    of_group = in_group[:, :, : c["group_top"]].sum(2)
    best = torch.sort(of_group, dim=1, descending=True, stable=True)[1][:, : c["top_groups"]]
    kept = torch.zeros(T, G, dtype=torch.bool, device=v.device).scatter_(1, best, True)
    v = torch.where(kept.repeat_interleave(E // G, 1), v, -math.inf)
    idx = torch.sort(v, dim=1, descending=True, stable=True)[1][:, :k]
    g = torch.gather(score, 1, idx)
    if c["renorm"]:
        g = g / (g.sum(1, keepdim=True) + TINY)
    return idx.int(), (g * c["scale"]).float()


def _plain(s):
    op, c = s["op"], s["case"]
    if op == "gate":
        idx, gates = _plain_gate(s)
        counts = torch.bincount(idx.flatten(), minlength=c["E"])
        out = {"idx": idx, "gates": gates, "counts": counts.int(),
               "aux": c["E"] * ((counts.double() / c["T"]) ** 2).sum(0, keepdim=True)}
        if c["rate"]:  # experts below the mean get more, those above it less
            out["bias"] = s["bias"] + c["rate"] * torch.sign(c["T"] * c["k"] - c["E"] * counts).float()
        return out
    if op == "gate_backward":
        score, idx, d = _scores(s["logits"], c["score"]), s["idx"].long(), s["d_gates"] * c["scale"]
        sel = torch.gather(score, 1, idx)
        if c["renorm"]:
            total = sel.sum(1, keepdim=True) + TINY
            d = (d - (d * sel).sum(1, keepdim=True) / total) / total
        ds = torch.zeros_like(score).scatter_(1, idx, d)
        if c["score"] == "sigmoid":
            return ds * score * (1 - score)
        return score * (ds - (d * sel).sum(1, keepdim=True))
    if op == "dispatch":
        idx, gates = _plain_gate(s)
        of = torch.sort(idx.flatten(), stable=True)[1]  # packed row -> assignment
        offsets = torch.zeros(c["E"] + 1, dtype=torch.int32, device=of.device)
        offsets[1:] = torch.cumsum(torch.bincount(idx.flatten(), minlength=c["E"]), 0)
        rows = _from_fp4(*_fp4(s["x"])).bfloat16()
        return {"idx": idx, "gates": gates, "offsets": offsets, "rows": rows[of // c["k"]]}
    x, xs = (s["x"], s["x_scales"]) if s["x_scales"] is not None else _fp4(s["x"])
    x, w = _from_fp4(x, xs), _from_fp4(s["w"], s["w_scales"])
    if "offsets" in s:
        # [E, rows of the fullest expert, K], zeros after an expert's last
        off = s["offsets"].long()
        at = off[:-1, None] + torch.arange(s["most"], device=x.device)
        keep = at < off[1:, None]
        u = torch.bmm(torch.where(keep[..., None], x[at.clamp(max=s["R"] - 1)], 0.0), w.mT)
        r = torch.arange(s["R"], device=x.device)
        e = torch.searchsorted(off[1:], r, right=True)
        u = u.flatten(0, 1)[e * s["most"] + r - off[e]]
        u = u if s["b"] is None else u + s["b"].float()[e]
    else:
        u = x @ w.T
        u = u if s["b"] is None else u + s["b"].float()
    y = _act(u, s["act"])
    return (y if s["residual"] is None else y + s["residual"].float()).bfloat16()


# --------------------------------------------------------------------------
# the framework's operators
# --------------------------------------------------------------------------

def _own(s):
    import combine_moe_gate_warp_gb300 as moe
    op, c = s["op"], s["case"]
    if op == "linear":
        if "rows" not in s:
            s["rows"] = moe.ExpertRows(s.get("offsets"), rows=s["R"], device="cuda")
            s["weights"] = moe.Fp4Rows(s["w"], s["w_scales"])
        rows = s["rows"]
        x = rows.quantize_fp4(s["x"]) if s["x_scales"] is None else moe.Fp4Rows(s["x"], s["x_scales"])
        return rows.linear_fp4(x, s["weights"], bias=s["b"], act=s["act"], residual=s["residual"])
    T, E, k = c["T"], c["E"], c["k"]
    if "scoring" not in s:  # the description, workspace and buffers that a program keeps for its sizes
        groups = {n: c[n] for n in ("groups", "top_groups", "group_top") if n in c}
        s["scoring"] = moe.Scoring(score=c["score"], renorm=c["renorm"], scale=c["scale"], **groups)
        if op == "dispatch":
            s["plan"] = moe.RoutePlan(moe.RouteShape(T=T, H=c["H"], E=E, k=k, P=1, scoring=s["scoring"], fp4=True))
            s["rows"] = moe.ExpertRows.of(s["plan"])
        else:
            s["ws"] = moe.alloc_workspace(T, E, k, 1)
            f32 = dict(dtype=torch.float32, device="cuda")
            s["gates"], s["ids"] = torch.empty(T, k, **f32), torch.empty(T, k, dtype=torch.int32, device="cuda")
            s["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
            s["aux"] = torch.empty(1, dtype=torch.float64, device="cuda")
            s["next"] = torch.empty(E, **f32) if c.get("rate") else None
            s["d_logits"] = torch.empty(T, E, **f32)
    if op == "gate":
        moe.moe_gate_scored(s["logits"], k, s["scoring"], s["bias"], s["ids"], s["gates"], s["counts"], s["aux"], None,
                            s["ws"], bias_next=s["next"], bias_rate=c["rate"])
        out = {"idx": s["ids"], "gates": s["gates"], "counts": s["counts"], "aux": s["aux"]}
        if c["rate"]:
            out["bias"] = s["next"]
        return out
    if op == "gate_backward":
        moe.moe_gate_scored_backward(s["logits"], s["idx"], s["d_gates"], s["scoring"], s["d_logits"], s["ws"])
        return s["d_logits"]
    plan = s["plan"]
    plan.route(s["logits"], s["bias"])
    plan.dispatch(s["x"])
    rows = s["rows"].dequantize_fp4(moe.Fp4Rows(plan.packed, plan.scales))
    return {"idx": plan.topk_idx, "gates": plan.gates, "offsets": plan.layout.offsets, "rows": rows}


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def _first_max(v):
    """Each row's largest value and the lowest column that holds it."""
    m = v.amax(1, keepdim=True)
    col = torch.arange(v.shape[1], device=v.device)
    return m, torch.where(v == m, col, v.shape[1]).amin(1, keepdim=True)


def _exact_scores(s):
    l = s["logits"].double()
    return torch.sigmoid(l) if s["case"]["score"] == "sigmoid" else torch.softmax(l, 1)


def _exact_gate(s):
    c = s["case"]
    per = c["E"] // c["groups"]
    score = _exact_scores(s)
    v = score.clone()
    if s["bias"] is not None:
        v += s["bias"].double()
    of_group = []
    for i in range(c["groups"]):
        part, total = v[:, i * per: (i + 1) * per].clone(), 0.0
        for _ in range(c["group_top"]):
            m, at = _first_max(part)
            total = total + m
            part.scatter_(1, at, -math.inf)
        of_group.append(total)
    of_group = torch.cat(of_group, 1)
    # a group is kept if fewer than top_groups stand before it
    n = torch.arange(c["groups"], device=v.device)
    for i in range(c["groups"]):
        mine = of_group[:, i: i + 1]
        before = ((of_group > mine) | ((of_group == mine) & (n < i))).sum(1)
        v[:, i * per: (i + 1) * per][before >= c["top_groups"]] = -math.inf
    ids, gates = [], []
    for _ in range(c["k"]):
        at = _first_max(v)[1]
        ids.append(at)
        gates.append(torch.take_along_dim(score, at, 1))
        v.scatter_(1, at, -math.inf)
    gates = torch.cat(gates, 1)
    if c["renorm"]:
        gates = gates / (gates.sum(1, keepdim=True) + TINY)
    return torch.cat(ids, 1).int(), gates * c["scale"]


def _power64(n):
    """2^n in fp64 for whole n, bit for bit."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _nearest(x):
    """Rows as their 4-bit form stands for them."""
    b = x.double().reshape(x.shape[0], x.shape[1] // BLOCK, BLOCK)
    # 6 = 1.5 * 2^2
    top = b.abs().amax(2, keepdim=True).clamp(min=6 * 2.0 ** -127)
    up = ((top.view(torch.int64) & ((1 << 52) - 1)) > (1 << 51)).long()  # amax past 1.5 of its power of two
    scale = _power64((top.view(torch.int64) >> 52) - 1023 - 2 + up)
    q = b / scale
    step = _power64((q.abs().clamp(min=1.0).view(torch.int64) >> 52) - 1024)
    return (torch.round(q / step) * step * scale).reshape(x.shape)


def _values64(codes, scales):
    """fp64 values of 4-bit rows, from the format: sign, 2 bits of exponent
    (bias 1), 1 bit of fraction; exponent 0 is subnormal."""
    c = np.arange(16)
    e, f = (c >> 1) & 3, c & 1
    v = np.where(e == 0, f / 2, (1 + f / 2) * 2.0 ** (e - 1.0)) * np.where(c & 8, -1.0, 1.0)
    pairs = torch.tensor(np.stack((np.tile(v, 16), np.repeat(v, 16)), 1), device=codes.device)  # of a byte
    v = pairs[codes.int()].reshape(codes.shape[0], codes.shape[1] * 2 // BLOCK, BLOCK)
    v = v * _power64(scales[:, : v.shape[1], None].long() - 127)
    return v.reshape(codes.shape[0], codes.shape[1] * 2)


def exact(case, seed):
    s = prepare(case, seed)
    op, c = s["op"], case
    if op in ("gate", "dispatch"):
        idx, gates = _exact_gate(s)
        counts = torch.stack([(idx == e).sum() for e in range(c["E"])])
    if op == "gate":
        out = {"idx": idx, "gates": gates, "counts": counts.int(),
               "aux": (counts.double() ** 2).sum().reshape(1) * c["E"] / c["T"] ** 2}
        if c["rate"]:
            less, more = counts * c["E"] < c["T"] * c["k"], counts * c["E"] > c["T"] * c["k"]
            out["bias"] = s["bias"].double() + c["rate"] * (less.double() - more.double())
        return out
    if op == "gate_backward":
        p, idx, k = _exact_scores(s), s["idx"].long(), c["k"]
        q = torch.take_along_dim(p, idx, 1)
        d, scale = s["d_gates"].double(), c["scale"]
        out = torch.zeros_like(p)
        # gate j's slope with respect to the score of selected expert i
        total = q.sum(1) + TINY
        for i in range(k):
            slope = d[:, i] * scale
            if c["renorm"]:
                slope = slope / total - scale * (d * q).sum(1) / total ** 2
            if c["score"] == "sigmoid":
                out.scatter_(1, idx[:, i: i + 1], (slope * q[:, i] * (1 - q[:, i]))[:, None])
            else:
                out -= (slope * q[:, i])[:, None] * p
                out.scatter_add_(1, idx[:, i: i + 1], (slope * q[:, i])[:, None])
        return out
    if op == "dispatch":
        values = _nearest(s["x"])
        token = torch.arange(c["T"], device=idx.device)[:, None].expand(c["T"], c["k"])
        rows = torch.cat([values[token[idx == e]] for e in range(c["E"])])
        offsets = torch.zeros(c["E"] + 1, dtype=torch.int32, device=idx.device)
        for e in range(c["E"]):
            offsets[e + 1] = offsets[e] + counts[e]
        return {"idx": idx, "gates": gates, "offsets": offsets, "rows": rows}
    if work(c)["flops"] > 8e12:
        return None
    off = s["offsets"].tolist() if "offsets" in s else [0, s["R"]]
    ys = []
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        of = (lambda t: t[e]) if "offsets" in s else (lambda t: t)
        x = s["x"][lo:hi]
        x = _nearest(x) if s["x_scales"] is None else _values64(x, s["x_scales"][lo:hi])
        u = x @ _values64(of(s["w"]), of(s["w_scales"])).T
        u = u if s["b"] is None else u + of(s["b"]).double()
        if s["act"] == "swiglu":
            f = u.shape[1] // 2
            y = u[:, :f] * torch.sigmoid(u[:, :f]) * u[:, f:]
        else:
            y = u * torch.sigmoid(u) if s["act"] == "silu" else u * torch.special.ndtr(u) if s["act"] == "gelu" else u
        ys.append(y if s["residual"] is None else y + s["residual"][lo:hi].double())
    return torch.cat(ys)
