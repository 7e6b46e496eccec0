"""64-bit references and error bounds of the BF16 expert layer's tests.

Bounds. Products of two bf16 values are exact in fp32. A sum of K of them in
fp32, in any order, is off by at most K * 2^-24 * S to first order, S = sum of
|a b|; the bounds below allow 2^-23 per term (an accumulator that truncates
instead of rounding). Rounding the result to bf16 adds at most 2^-8 of it
(half a step, torch.finfo(torch.bfloat16).eps / 2).
"""
import torch

U8, U23 = 2.0 ** -8, 2.0 ** -23


def d64(t):
    return t.detach().cpu().to(torch.float64)


def matmul_bound(a, b):
    """(a @ b, its fp32 summation bound) for 64-bit a [m, K], b [K, n]."""
    return a @ b, a.shape[1] * U23 * (a.abs() @ b.abs())


def out_bound(ref, err, f32):
    """Bound of an output whose fp32 value is within err of ref, after its rounding (subnormal results: 2^-126)."""
    return err + (0.0 if f32 else U8 * (ref.abs() + err)) + 2.0 ** -126


def check(got, ref, bound, what):
    got = d64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound; first at {i}: got "
                             f"{got[i].item()!r}, reference {ref[i].item()!r}, bound {bound[i].item()!r}")


NONE, RELU, GELU, GELU_TANH, SILU, SWIGLU = range(6)


def act_ref(z, act, n):
    """64-bit (value, factors of dout in dz, per half of z)."""
    if act == NONE:
        return z, (torch.ones_like(z),)
    if act == RELU:
        return torch.where(z > 0, z, 0.0 * z), ((z > 0).double(),)
    if act == GELU:
        c = torch.special.ndtr(z)
        return z * c, (c + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5,)
    if act == GELU_TANH:
        a = (2 / torch.pi) ** 0.5
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z),)
    if act == SILU:
        s = torch.sigmoid(z)
        return z * s, (s + z * s * (1 - s),)
    g, u = z[:, :n], z[:, n:]
    s = torch.sigmoid(g)
    return g * s * u, (u * (s + g * s * (1 - s)), g * s)


def act_bound(z, dz, act, n):
    """Bound of act's fp32 value when its fp32 argument is within dz of z. |act'| <= 1.2 for every activation
    here; the fp32 function itself: an exponential whose argument (up to |z| or, for the tanh form, v = 1.6 z +
    0.072 z^3) is rounded a few times, relative error (|arg| + 16) 2^-23 of a result no larger than |z|."""
    if act == SWIGLU:
        g, u, dg, du = z[:, :n], z[:, n:], dz[:, :n], dz[:, n:]
        return 1.2 * dg * (u.abs() + du) + g.abs() * (du + u.abs() * (g.abs() + 16) * U23)
    if act in (NONE, RELU):
        return dz + z.abs() * U23
    arg = z.abs() if act != GELU_TANH else 1.6 * z.abs() + 0.08 * z.abs() ** 3
    # past |arg| = 40 the sigmoid is 0 or 1 to more than 2^-50: its argument's error no longer shows
    return 1.2 * dz + z.abs() * (arg.clamp_max(40.0) + 16) * U23


def segments(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out
