"""Helpers of the expert-product tests: seeded inputs, the products in 64
bits, and how far a result may be off.

An accumulated sum of n products is held in fp32: the tensor cores add 16
products at a time, and each of the n/16 steps (and a few more on the way)
is off by at most 2^-22 of the sum of the magnitudes (a truncated fp32
step).  A bf16 result is off by half a step more, 2^-8 of its value."""
import math

import torch

BF16 = 2.0 ** -8


def sum_error(n, magnitudes):
    """Bound on the error of fp32 sums of n products, given the sums of the
    products' magnitudes."""
    return (n / 16 + 8) * 2.0 ** -22 * magnitudes


def offsets_of(counts, device="cuda"):
    off = [0]
    for n in counts:
        off.append(off[-1] + n)
    return torch.tensor(off, dtype=torch.int32, device=device)


def normal(*shape, seed, std=1.0, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).bfloat16().to(device)


def spans(counts):
    lo, out = 0, []
    for e, n in enumerate(counts):
        out.append((e, lo, lo + n))
        lo += n
    return out


def act64(u, act):
    if act == "swiglu":
        g, v = u.chunk(2, -1)
        return g * torch.sigmoid(g) * v
    if act == "silu":
        return u * torch.sigmoid(u)
    if act == "gelu":
        return u * torch.special.ndtr(u)
    return u


def act_error(u, eu, act):
    """Bound on act's error (before its rounding to bf16) from an error eu of
    u.  The slopes of silu and gelu are at most 1.13; the evaluation in fp32
    adds 2^-18 of the value and 2^-20 of u (gelu's 1 + erf cancels)."""
    if act == "none":
        return eu
    if act == "swiglu":
        g, v = u.chunk(2, -1)
        eg, ev = eu.chunk(2, -1)
        s = (g * torch.sigmoid(g)).abs()
        es = 1.13 * eg + 2.0 ** -18 * s
        return es * (v.abs() + ev) + s * ev + 2.0 ** -20 * (s * v).abs()
    return 1.13 * eu + 2.0 ** -18 * act64(u, act).abs() + 2.0 ** -20 * u.abs()


def slope64(u, act):
    if act == "silu":
        q = torch.sigmoid(u)
        return q * (1 + u * (1 - q))
    if act == "gelu":
        return torch.special.ndtr(u) + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(u)


def grad64(u, d, act):
    """d times act'(u), laid out as u."""
    if act == "swiglu":
        g, v = u.chunk(2, -1)
        return torch.cat((d * v * slope64(g, "silu"), d * g * torch.sigmoid(g)), -1)
    return d * slope64(u, act)


def grad_error(u, d, ed, act):
    """Bound on grad64's error from an error ed of d; u is exact."""
    if act == "swiglu":
        g, v = u.chunk(2, -1)
        s = (g * torch.sigmoid(g)).abs()
        one = (1.13 * ed + 2.0 ** -17 * (1 + g.abs()) * d.abs()) * v.abs()
        return torch.cat((one, ed * s + 2.0 ** -17 * d.abs() * s), -1)
    return 1.13 * ed + 2.0 ** -17 * (1 + u.abs()) * d.abs()


def linear64(x, w, counts, bias=None):
    """(u, error bound of u) in 64 bits; x, w, bias in any float type."""
    us, es = [], []
    for e, lo, hi in spans(counts):
        xe, we = x[lo:hi].double(), w[e].double()
        u, m = xe @ we.T, xe.abs() @ we.abs().T
        if bias is not None:
            u, m = u + bias[e].double(), m + bias[e].double().abs()
        us.append(u)
        es.append(sum_error(xe.shape[1], m))
    return torch.cat(us), torch.cat(es)


def decode64(codes, scales):
    """Values of a saved layer, in 64 bits."""
    v = codes.view(torch.float8_e4m3fn).double()
    s = torch.pow(2.0, scales.double() - 127)
    return v * s.repeat_interleave(32, -1)


def encode_saved(u):
    """A saved layer of given values, by its definition (32 bits are exact for bf16 values)."""
    b = u.float().reshape(u.shape[0], u.shape[1] // 32, 32)
    m, e = torch.frexp(b.abs().amax(2))
    x = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-127)
    codes = torch.ldexp(b, -x[..., None]).to(torch.float8_e4m3fn).reshape(u.shape)
    return codes.view(torch.uint8).contiguous(), (x + 127).to(torch.uint8)


def assert_near(got, want, bound, what):
    """got within bound of want, element by element; says where it is not."""
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    if bool(bad.any()):
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, the first at {i}: got "
                             f"{got[tuple(i)].item()!r}, expected {want[tuple(i)].item()!r} "
                             f"within {bound[tuple(i)].item():.3g}")
