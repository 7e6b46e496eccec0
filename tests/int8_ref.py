"""64-bit references and error bounds of the int8 products' tests.

The sum of a product is an exact integer below 2^31 in magnitude. Its fp32 value takes three roundings (to fp32, times the
row's scale, times the channel's), each of at most 2^-24 of the value: 3.1 * 2^-24 with the second-order terms.
"""
import torch

from bf16_ref import U23, d64

U_SUM = 3.1 * 2.0 ** -24


def quantize(x):
    """(codes, fp32 scales) of a bf16 tensor on the CPU. In 64 bits 127 x / amax is off by 2^-53 of itself, a quotient that
    is no tie is 2^-16 of itself away from one (15 bits over 8), and a tie is exact: torch.round decides as the definition."""
    x = x.detach().cpu()
    v = x.to(torch.float64)
    top = v.abs().amax(-1)
    bad = ~torch.isfinite(v).all(-1)
    live = (top > 0) & ~bad
    q = torch.round(torch.where(live[..., None], v, torch.zeros_like(v)) * 127.0 / torch.where(live, top, 1.0)[..., None])
    scale = torch.where(live, top.float() / 127.0, torch.ones_like(top, dtype=torch.float32))
    scale[bad] = float("nan")
    return q.to(torch.int8), scale


def product(xq, xs, wq, ws):
    """(x w^T with its scales in 64 bits, bound of its fp32 value). The sums are taken in int64 pieces, exactly."""
    s = (xq.cpu().to(torch.float64) @ wq.cpu().to(torch.float64).T)   # integers below 2^53: exact
    z = s * d64(xs)[:, None] * d64(ws)
    return z, z.abs() * U_SUM + 2.0 ** -126


def with_bias(z, dz, bias):
    if bias is None:
        return z, dz
    z = z + d64(bias)
    return z, dz + z.abs() * U23
