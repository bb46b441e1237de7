"""Routing by scores in 64 bits, on the CPU, and rows in 4 bits by their
definition."""
import torch

TINY = 1e-20


def scores64(logits, score):
    l = logits.double()
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def select64(logits, k, score="sigmoid", groups=1, top_groups=1, group_top=1, bias=None):
    """The selected experts [T, k], one round of arg-max after the other."""
    T, E = logits.shape
    v = scores64(logits, score)
    if bias is not None:
        v = v + bias.double()
    g = v.reshape(T, groups, E // groups).sort(2, descending=True)[0][:, :, :group_top].sum(2)
    for _ in range(groups - top_groups):  # drop the worst group, of equal ones the last
        m = g.amin(1, keepdim=True)
        at = torch.where(g == m, torch.arange(groups), -1).amax(1)
        g[torch.arange(T), at] = float("inf")
        v.reshape(T, groups, E // groups)[torch.arange(T), at] = float("-inf")
    out = []
    for _ in range(k):
        m = v.amax(1, keepdim=True)
        at = torch.where(v == m, torch.arange(E), E).amin(1)
        out.append(at)
        v[torch.arange(T), at] = float("-inf")
    return torch.stack(out, 1)


def gates64(logits, idx, score="sigmoid", renorm=True, scale=1.0):
    """The gates of given experts; differentiable in double logits."""
    s = torch.gather(scores64(logits, score), 1, idx)
    if renorm:
        s = s / (s.sum(1, keepdim=True) + TINY)
    return s * scale


def gates_error(want, logits, idx, score, renorm, scale):
    """expf is off by 2 steps of 2^-23 at most, sums of E (softmax) and k
    values by half a step an addition, the divisions and products by half a
    step each: below (E + k) / 2 + 12 steps of the value.  A score below
    2^-126 has lost digits to fp32's range, at most 2^-126 of them, which the
    renormalisation magnifies as it does the score."""
    n = (logits.shape[1] if score == "softmax" else 0) + idx.shape[1]
    lost = 2.0 ** -126 * abs(scale)
    if renorm:
        lost = lost / (torch.gather(scores64(logits, score), 1, idx).sum(1, keepdim=True) + TINY)
    return (n / 2 + 12) * 2.0 ** -23 * want.abs() + lost


def backward_error(logits, idx, d, E, score, renorm, scale):
    """The same count of steps on every product and sum of the gradient's
    terms, whose magnitudes are taken for their sum."""
    s = scores64(logits, score)
    sel = torch.gather(s, 1, idx)
    d = d.double().abs() * abs(scale)
    if renorm:
        n = sel.sum(1, keepdim=True) + TINY
        d = (d + (d * sel).sum(1, keepdim=True) / n) / n
    each = d * sel * (1 - sel if score == "sigmoid" else 1)
    out = torch.zeros_like(s).scatter_add_(1, idx, each)
    if score == "softmax" and not renorm:
        out = out + s * each.sum(1, keepdim=True)
    # with renorm the softmax's common term is tiny / sum of the gates', and
    # what 64 bits make of it is the rest of two equal sums, 2^-52 of them for
    # each of some 16 operations
    if score == "softmax":
        out = out + 2.0 ** -25 * s * each.sum(1, keepdim=True)
    return ((E + idx.shape[1]) / 2 + 40) * 2.0 ** -23 * out + 1e-30


VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def power(n):
    """2^n for a tensor of whole n, in fp64 bit for bit."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def encode_fp4(x):
    """(codes [rows, K / 2], scales [rows, pitch]) of bf16 rows, on the CPU."""
    x = x.detach().cpu()
    rows, K = x.shape
    b = x.double().reshape(rows, K // 32, 32)
    top = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    e = torch.full(top.shape, -127)
    for n in range(-127, 127):  # the smallest power of two that holds the block
        e = torch.where(top > 6 * 2.0 ** n, n + 1, e)
    q = (b.nan_to_num(0.0, 0.0, 0.0) / power(e)[..., None]).reshape(rows, K)
    values = torch.tensor(VALUES, dtype=torch.float64)
    off = (q.abs()[..., None] - values).abs()
    least = off.amin(-1, keepdim=True)
    even = torch.tensor([0.0, 0.25] * 4)  # of two as near the even code
    code = torch.where(off == least, even, 1.0).argmin(-1)
    code = torch.where(bad.repeat_interleave(32, 1), 7, code + 8 * torch.signbit(x).long())
    scales = torch.zeros(rows, (K + 511) // 512 * 16, dtype=torch.uint8)
    scales[:, :K // 32] = torch.where(bad, 255, e + 127).to(torch.uint8)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8), scales


def decode_fp4(codes, scales):
    """The values of rows in 4 bits, in fp64."""
    codes, scales = codes.cpu(), scales.cpu()
    K = 2 * codes.shape[-1]
    table = torch.tensor(VALUES + [-v for v in VALUES], dtype=torch.float64)
    v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()]
    s = scales[..., :K // 32].long()
    s = torch.where(s == 255, float("nan"), power(s - 127))
    return v * s.repeat_interleave(32, -1)
