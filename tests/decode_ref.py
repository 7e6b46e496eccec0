"""64-bit reference and error bounds of the whole expert layer for a few tokens.

Bounds, U = 2^-23 per fp32 operation of a sum (2^-24 rounded, twice that where the matrix pipe truncates):
  logits   every 32 products are summed to fp32, then in fp64: U * sum |x w|
  weights  a softmax or a ratio of sigmoids of logits off by dl: 2.1 dl relative, and the rounding to fp32
  g, u     K U sum |x w|, and one product with a scale
  h        bf16_ref.act_bound, and its rounding: two bf16 parts, 2^-16 of it; NVFP4 fp16, 2^-11 of it and half the smallest
           subnormal, 2^-25, times 2^exp, where 2^(exp + 15) is the square of three factors' product rounded up to powers
           of two (each at most twice): the sum of |x|, 2688 and w1's tensor scale
  out      f U sum |w2 h|, a product with a scale, weights and the at most k + 16 partial sums that are added
"""
import torch

from bf16_ref import SWIGLU, U23, act_bound, act_ref, d64

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def values(w, fmt):
    """fp64 values of weights in a format (bf16 tensor; int8 (codes, scales); NVFP4 (codes, scales, tscale))."""
    if fmt == "bf16":
        return d64(w)
    if fmt == "int8":
        return d64(w[0]) * d64(w[1])[..., None]
    c = w[0].cpu()
    c = torch.stack([c & 15, c >> 4], -1).flatten(-2).long()
    v = torch.where(c >= 8, -E2M1[c & 7], E2M1[c & 7])
    s = w[1].cpu().view(torch.float8_e4m3fn).to(torch.float64) * d64(w[2])[:, None, None]
    return v * s.repeat_interleave(16, -1)


def route(x, wr, bias, k, sigmoid):
    """(keys, logits, bound of either) in 64 bits."""
    lg = d64(x) @ d64(wr).T
    dl = U23 * (d64(x).abs() @ d64(wr).abs().T)
    key = torch.sigmoid(lg) if sigmoid else lg
    if bias is not None:
        key = key + d64(bias)
    return key, lg, dl


def check_choice(ids, weights, key, lg, dl, k, sigmoid):
    """The ids choose and order the largest keys (to within the logits' bound) and the weights are theirs."""
    ids, weights = ids.cpu().long(), d64(weights)
    T, E = key.shape
    assert ids.shape == (T, k) and ((ids >= 0) & (ids < E)).all()
    for t in range(T):
        assert len(set(ids[t].tolist())) == k
    slack = 2 * dl.amax(1, keepdim=True) + 1e-15
    chosen = key.gather(1, ids)
    assert (chosen[:, :-1] >= chosen[:, 1:] - slack).all()
    if k < E:
        rest = key.scatter(1, ids, float("-inf")).amax(1, keepdim=True)
        assert (chosen[:, -1:] >= rest - slack).all()
    v = lg.gather(1, ids)
    w = torch.sigmoid(v) if sigmoid else torch.exp(v - v.amax(1, keepdim=True))
    w = w / w.sum(1, keepdim=True)
    dw = w * (2.1 * dl.amax(1, keepdim=True) + U23) + 2.0 ** -149
    assert ((weights - w).abs() <= dw).all()
    return ids, w, dw


def layer(x, ids, w, dw, w1, w2, residual, t1=None):
    """(out, bound of its fp32 value) for 64-bit weights w1 [E, 2f, d], w2 [E, d, f]. t1: NVFP4's tensor scales of w1."""
    T, k = ids.shape
    f, d = w2.shape[2], w2.shape[1]
    out = torch.zeros((T, d), dtype=torch.float64)
    err, mag = torch.zeros_like(out), torch.zeros_like(out)
    for t in range(T):
        xt = d64(x[t:t + 1])
        for s in range(k):
            e = int(ids[t, s])
            z = xt @ w1[e].T
            dz = (d + 2) * U23 * (xt.abs() @ w1[e].abs().T)
            h = act_ref(z, SWIGLU, f)[0]
            dh = act_bound(z, dz, SWIGLU, f)
            if t1 is None:
                dh = dh + 2.0 ** -16 * (h.abs() + dh) + 2.0 ** -133
            else:
                top = float(xt.abs().sum()) * 2688.0 * float(t1[e])
                dh = dh + 2.0 ** -11 * (h.abs() + dh) + 2.0 ** -40 * (4.0 * top) ** 2
            y, a = (h @ w2[e].T)[0], ((h.abs() + dh) @ w2[e].abs().T)[0]
            dy = (dh @ w2[e].abs().T)[0] + (f + 2) * U23 * a
            out[t] += w[t, s] * y
            err[t] += w[t, s] * dy + dw[t, s] * (y.abs() + dy)
            mag[t] += w[t, s] * a
    err = err + (k + 17) * U23 * mag
    if residual is not None:
        out = out + d64(residual)
        err = err + out.abs() * U23
    return out, err
