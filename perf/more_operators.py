"""The INT8 products' and the few-token expert layer's operators with their plain forms, case by case.

Four operators for serving the expert layer: int8 quantization per row (per token, per weight channel)
and back, the dense int8 product with its epilogue, the whole expert forward in int8, and the whole
mixture-of-experts layer for a few tokens (router, experts and combine in one call) on bf16, int8 or
NVFP4 weights. With `own` true `run` makes the library's calls; with `own` false it computes the same
in elementary torch operations: 32-bit products and sums (64 where a choice hangs on them), one
rounding at the end.

A case is a dict; `op` names the path:
  quant    codes and scales of bf16 rows, and the values they stand for
  linear   out = act((xq wq^T) xs ws + bias) + residual
  experts  y[t][s] = the s-th chosen expert of token t, int8 weights, activations quantized per row
  decode   out = residual + the weighted sum of the chosen experts, from the hidden state
"""
import math

import torch

own = False

NONE, RELU, GELU, GELU_TANH, SILU, SWIGLU = "none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"
ACTS = (NONE, RELU, GELU, GELU_TANH, SILU, SWIGLU)
BF16, INT8, NVFP4 = "bf16", "int8", "nvfp4"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    moe = dict(d=4096, E=384, k=8, d_ff=1024)   # the moe_layer workload's layer
    dec = dict(op="decode", router="softmax", bias=True, residual=True)
    return [
        # serving: the hidden states of four sequences, quantized for an int8 product
        dict(name="quant_decode", op="quant", R=4, C=4096, f32=True),
        # a prompt batch of the moe_layer workload, quantized and read back
        dict(name="quant_prompt", op="quant", R=16384, C=4096, f32=False),
        # serving: a shared SwiGLU expert on eight tokens, bound by its weights
        dict(name="linear_decode", op="linear", M=8, N=1024, K=4096, act=SWIGLU, bias=False, residual=False, f32=False),
        # a chunk of a prompt of odd length through a product whose sizes fill no tile
        dict(name="linear_ragged", op="linear", M=1003, N=2056, K=4112, act=SILU, bias=True, residual=False, f32=True),
        # a dense feed-forward product of a large prompt batch with everything in its epilogue
        dict(name="linear_prompt", op="linear", M=8192, N=8192, K=4096, act=GELU, bias=True, residual=True, f32=False),
        # the tiny_moe workload's layer: latency of a chain of small launches
        dict(name="experts_tiny", op="experts", T=256, d=256, E=8, k=2, d_ff=512, skew=0.0),
        # prompts: the whole moe_layer batch, experts of very different load
        dict(name="experts_prompt", op="experts", T=16384, skew=1.0, **moe),
        # decoding one sequence with bf16 weights
        dict(name="decode_bf16_1", T=1, weights=BF16, **moe, **dec),
        # decoding four sequences with int8 weights
        dict(name="decode_int8_4", T=4, weights=INT8, **moe, **dec),
        # decoding one sequence with NVFP4 weights: a quarter of bf16's bytes, launches count
        dict(name="decode_nvfp4_1", T=1, weights=NVFP4, **moe, **dec),
        # decoding a batch: most experts are hit, by one or two tokens each
        dict(name="decode_nvfp4_64", T=64, weights=NVFP4, **moe, **dec),
        # a small layer with the sigmoid router, three tokens: the smallest call
        dict(name="decode_small", op="decode", T=3, d=256, E=8, k=2, d_ff=512, weights=BF16, router="sigmoid", bias=True,
             residual=False),
    ]


def _log_int(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / mult)) * mult))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "experts", "decode", "decode", "decode"])
    if op == "quant":
        return dict(op=op, R=_log_int(rng, 1, 16384), C=_log_int(rng, 16, 8192, 16), f32=rng.random() < 0.5)
    if op == "linear":
        return dict(op=op, M=_log_int(rng, 1, 16384), N=_log_int(rng, 8, 4096, 8), K=_log_int(rng, 64, 4096, 16),
                    act=rng.choice(ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.5, f32=rng.random() < 0.3)
    E = _log_int(rng, 4, 384)
    c = dict(op=op, d=_log_int(rng, 64, 4096, 32), E=E, k=rng.randint(1, min(8, E)), d_ff=_log_int(rng, 64, 1024, 32))
    if op == "experts":
        c.update(T=_log_int(rng, 1, 16384), skew=rng.choice([0.0, 1.0]))
        return c
    c.update(T=_log_int(rng, 1, 64), weights=rng.choice([BF16, INT8, NVFP4]), router=rng.choice(["softmax", "sigmoid"]),
             residual=rng.random() < 0.5)
    c["bias"] = c["router"] == "sigmoid" or rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, std, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _codes(x):
    """Codes and scales of bf16 rows: 127 x / amax is decided in 64 bits, which the nearest ties of bf16 values need."""
    a = x.abs().amax(-1, keepdim=True).double()
    live = a > 0
    q = torch.round(x.double() * 127.0 / torch.where(live, a, 1.0))
    scale = torch.where(live, a / 127.0, 1.0)
    return q.to(torch.int8), scale.squeeze(-1).float()


def _nvfp4(w):
    """NVFP4 of [n, rows, cols]: nearest codes under one E4M3 scale per 16 values and one fp32 scale per matrix."""
    n, rows, cols = w.shape
    w = w.float()
    t = w.abs().amax((1, 2), keepdim=True) / 2688.0
    b = w.view(n, rows, cols // 16, 16)
    s = (b.abs().amax(-1) / (6.0 * t)).to(torch.float8_e4m3fn)
    y = (b / (s.float() * t).clamp_min(1e-30)[..., None]).view(n, rows, cols)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    c = torch.bucketize(y.abs(), edges).to(torch.uint8) | (y < 0).to(torch.uint8) << 3
    return c[..., 0::2] | c[..., 1::2] << 4, s.view(torch.uint8), t.view(n)


def _weights(gen, E, rows, cols, fmt):
    """Weights N(0, 0.02) of E experts in a format: a tuple of tensors."""
    parts = []
    for e in range(0, E, 16):
        w = _normal(gen, (min(16, E - e), rows, cols), 0.02)
        parts.append((w,) if fmt == BF16 else _codes(w) if fmt == INT8 else _nvfp4(w))
    return tuple(torch.cat(p) for p in zip(*parts))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    c = dict(case)
    st = {"case": c}
    if c["op"] == "quant":
        st["x"] = _normal(gen, (c["R"], c["C"]), 1.0)
    elif c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        rows = 2 * N if c["act"] == SWIGLU else N
        st["x"] = _codes(_normal(gen, (M, K), 1.0))
        st["w"] = _codes(_normal(gen, (rows, K), 0.02))
        st["bias"] = _normal(gen, (rows,), 0.1, torch.float32) if c["bias"] else None
        st["residual"] = _normal(gen, (M, N), 1.0) if c["residual"] else None
    else:
        T, d, E, k, f = c["T"], c["d"], c["E"], c["k"], c["d_ff"]
        fmt = INT8 if c["op"] == "experts" else c["weights"]
        st["x"] = _normal(gen, (T, d), 1.0)
        st["w1"] = _weights(gen, E, 2 * f, d, fmt)
        st["w2"] = _weights(gen, E, d, f, fmt)
        if c["op"] == "experts":
            key = torch.randn((T, E), generator=gen, device="cuda")
            key += c["skew"] * torch.randn((E,), generator=gen, device="cuda")
            ids = key.topk(k, dim=1).indices
            st["ids"] = ids.to(torch.int32).contiguous()
            st["order"] = torch.argsort(ids.reshape(-1), stable=True)
            st["counts"] = torch.bincount(ids.reshape(-1), minlength=E).tolist()
        else:
            st["router"] = _normal(gen, (E, d), d ** -0.5)
            st["bias"] = _normal(gen, (E,), 0.5, torch.float32) if c["bias"] else None
            st["residual"] = _normal(gen, (T, d), 1.0) if c["residual"] else None
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    import precision_moe_numerics_amd as nvq
    c = st["case"]
    if c["op"] == "quant":
        codes, scales = nvq.int8_quantize(st["x"])
        return nvq.int8_dequantize(codes, scales, out_dtype=torch.float32 if c["f32"] else torch.bfloat16), scales
    if c["op"] == "linear":
        act = {NONE: nvq.ACT_NONE, RELU: nvq.ACT_RELU, GELU: nvq.ACT_GELU, GELU_TANH: nvq.ACT_GELU_TANH,
               SILU: nvq.ACT_SILU, SWIGLU: nvq.ACT_SWIGLU}[c["act"]]
        return nvq.linear_act_int8(st["x"], st["w"], bias=st["bias"], act=act, residual=st["residual"],
                                   out_dtype=torch.float32 if c["f32"] else torch.bfloat16)
    if c["op"] == "experts":
        return nvq.moe_expert_fwd_int8(st["x"], st["ids"], st["w1"], st["w2"])
    router = nvq.ROUTER_SIGMOID if c["router"] == "sigmoid" else nvq.ROUTER_SOFTMAX
    args = dict(bias=st["bias"], router=router, residual=st["residual"])
    if c["weights"] == BF16:
        return nvq.moe_layer_decode_bf16(st["x"], st["router"], c["k"], st["w1"][0], st["w2"][0], **args)
    if c["weights"] == INT8:
        return nvq.moe_layer_decode_int8(st["x"], st["router"], c["k"], st["w1"], st["w2"], **args)
    return nvq.moe_layer_decode_nvfp4(st["x"], st["router"], c["k"], st["w1"], st["w2"], **args)


def _act(z, act):
    if act == RELU:
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == GELU:
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == GELU_TANH:
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == SILU:
        return z / (1 + torch.exp(-z))
    if act == SWIGLU:
        g, u = z.chunk(2, dim=-1)
        return g * u / (1 + torch.exp(-g))
    return z


def _values(w, ids, fmt):
    """fp32 values of the matrices `ids` (a slice or index tensor) of a stack in a format."""
    if fmt == BF16:
        return w[0][ids].float()
    if fmt == INT8:
        return w[0][ids].float() * w[1][ids][..., None]
    c = w[0][ids]
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=c.device)
    v = lut[torch.stack([c & 15, c >> 4], -1).flatten(-2).int()]
    s = w[1][ids].view(torch.float8_e4m3fn).float() * w[2][ids][:, None, None]
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _run_plain(st):
    c = st["case"]
    if c["op"] == "quant":
        codes, scales = _codes(st["x"])
        return (codes.float() * scales[:, None]).to(torch.float32 if c["f32"] else torch.bfloat16), scales
    if c["op"] == "linear":
        (xq, xs), (wq, ws) = st["x"], st["w"]
        z = (xq.float() @ wq.float().T) * xs[:, None] * ws
        if st["bias"] is not None:
            z = z + st["bias"]
        out = _act(z, c["act"])
        if st["residual"] is not None:
            out = out + st["residual"].float()
        return out if c["f32"] else out.to(torch.bfloat16)
    if c["op"] == "experts":
        return _plain_experts(st, c)
    ids, p = _plain_route(st, c)
    x, fmt = st["x"].float(), c["weights"]
    out = []
    for t in range(c["T"]):
        e = ids[t]
        z = _values(st["w1"], e, fmt) @ x[t]
        h = _act(z, SWIGLU)
        y = (_values(st["w2"], e, fmt) @ h[:, :, None]).squeeze(-1)
        out.append((p[t][:, None] * y).sum(0))
    out = torch.stack(out)
    if st["residual"] is not None:
        out = out + st["residual"].float()
    return out.to(torch.bfloat16), ids.to(torch.int32), p


def _plain_route(st, c):
    """The choice in 64 bits (of two close logits the larger one is chosen); the lower of equal keys first."""
    logits = st["x"].double() @ st["router"].double().T
    score = 1 / (1 + torch.exp(-logits)) if c["router"] == "sigmoid" else logits
    key = score if st["bias"] is None else score + st["bias"].double()
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    v = score.gather(1, ids)
    if c["router"] != "sigmoid":
        v = torch.exp(v - v.amax(1, keepdim=True))
    return ids, (v / v.sum(1, keepdim=True)).float()


def _plain_experts(st, c):
    T, k = c["T"], c["k"]
    xq, xs = _codes(st["x"])
    y = torch.empty((T * k, c["d"]), dtype=torch.bfloat16, device="cuda")
    a = 0
    for e, n in enumerate(st["counts"]):
        if n == 0:
            continue
        rows = st["order"][a:a + n]
        a += n
        src = rows // k
        z = (xq[src].float() @ st["w1"][0][e].float().T) * xs[src][:, None] * st["w1"][1][e]
        hq, hs = _codes(_act(z, SWIGLU).to(torch.bfloat16))
        y[rows] = ((hq.float() @ st["w2"][0][e].float().T) * hs[:, None] * st["w2"][1][e]).to(torch.bfloat16)
    return y.view(T, k, c["d"])


# ------------------------------------------------------------------ work and exact values
def _bytes_per_value(fmt):
    return {BF16: 2.0, INT8: 1.0, NVFP4: 0.5625}[fmt]


def work(case):
    c = case
    if c["op"] == "quant":
        n = c["R"] * c["C"]
        # bf16 in, codes and scales out and in again, values out
        return dict(bytes=n * (2 + 1 + 1 + (4 if c["f32"] else 2)) + 8 * c["R"], flops=4 * n)
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        R = 2 * N if c["act"] == SWIGLU else N
        return dict(bytes=M * K + R * K + 4 * (M + R) + (4 if c["f32"] else 2) * M * N + (2 * M * N if c["residual"] else 0)
                    + (4 * R if c["bias"] else 0), flops=2 * M * R * K)
    T, d, E, k, f = c["T"], c["d"], c["E"], c["k"], c["d_ff"]
    hit = E * (1 - (1 - k / E) ** T)       # experts with at least one row under even routing
    if c["op"] == "experts":
        return dict(bytes=2 * T * d + hit * (3 * f * d + 4 * (2 * f + d)) + 2 * T * k * d + 4 * T * k,
                    flops=6 * T * k * f * d)
    scales = 4 * hit * (2 * f + d) if c["weights"] == INT8 else 8 * hit if c["weights"] == NVFP4 else 0
    return dict(bytes=hit * 3 * f * d * _bytes_per_value(c["weights"]) + scales + 2 * E * d + 4 * T * d + 8 * T * k
                + (4 * E if c["bias"] else 0) + (2 * T * d if c["residual"] else 0),
                flops=6 * T * k * f * d + 2 * T * E * d)


def exact(case, seed):
    """The definitions in 64 bits, over the experts in turn and whole matrices."""
    c = case
    st = prepare(case, seed)
    if c["op"] == "quant":
        x = st["x"].to(torch.float64)
        top = torch.linalg.vector_norm(x, float("inf"), dim=1)
        step = torch.where(top == 0, torch.ones_like(top), top / 127)
        return _exact_rows(x), step
    if c["op"] == "linear":
        a = torch.mul(st["x"][0].to(torch.float64), st["x"][1].to(torch.float64).unsqueeze(1))
        b = torch.mul(st["w"][0].to(torch.float64), st["w"][1].to(torch.float64).unsqueeze(1))
        z = torch.mm(a, b.t().contiguous())
        if c["bias"]:
            z += st["bias"].to(torch.float64)[None, :]
        out = _exact_act(z, c["act"], c["N"])
        return out + st["residual"].to(torch.float64) if c["residual"] else out
    T, d, E, k, f = c["T"], c["d"], c["E"], c["k"], c["d_ff"]
    x = st["x"].to(torch.float64)
    if c["op"] == "experts":
        if T * k * f * d > 2 ** 40:
            return None
        rows = _exact_rows(x)
        res = torch.zeros((T, k, d), dtype=torch.float64, device="cuda")
        for e in torch.unique(st["ids"]).tolist():
            t, s = (st["ids"] == e).nonzero(as_tuple=True)
            h = _exact_act(torch.mm(rows[t], _exact_matrix(st["w1"], e, INT8).t().contiguous()), SWIGLU, f)
            h = _exact_rows(h.to(torch.bfloat16).to(torch.float64))
            res[t, s] = torch.mm(h, _exact_matrix(st["w2"], e, INT8).t().contiguous())
        return res
    lg = torch.mm(x, st["router"].to(torch.float64).t().contiguous())
    val = torch.sigmoid(lg) if c["router"] == "sigmoid" else lg
    key = (val + st["bias"].to(torch.float64)[None, :]) if c["bias"] else val.clone()
    ids = torch.empty((T, k), dtype=torch.int64, device="cuda")
    col = torch.arange(E, device="cuda")
    for s in range(k):
        # the lowest index among the largest keys
        best = torch.where(key == key.amax(dim=1, keepdim=True), col, E).amin(dim=1)
        ids[:, s] = best
        key[torch.arange(T, device="cuda"), best] = float("-inf")
    p = torch.take_along_dim(val, ids, 1)
    p = p / p.sum(dim=1, keepdim=True) if c["router"] == "sigmoid" else torch.softmax(p, dim=1)
    res = st["residual"].to(torch.float64).clone() if c["residual"] else torch.zeros((T, d), dtype=torch.float64,
                                                                                     device="cuda")
    for e in torch.unique(ids).tolist():
        t, s = (ids == e).nonzero(as_tuple=True)
        h = _exact_act(torch.mm(x[t], _exact_matrix(st["w1"], e, c["weights"]).t().contiguous()), SWIGLU, f)
        res[t] += p[t, s][:, None] * torch.mm(h, _exact_matrix(st["w2"], e, c["weights"]).t().contiguous())
    return res, ids.to(torch.int32), p


def _exact_rows(x):
    """Rows rounded to their 255 levels, in 64 bits."""
    top = x.abs().amax(dim=1, keepdim=True)
    step = torch.where(top == 0, torch.ones_like(top), top / 127)
    return step * torch.special.round(x * 127 / torch.where(top == 0, torch.ones_like(top), top))


def _exact_matrix(w, e, fmt):
    """Matrix e of a stack in 64 bits."""
    if fmt == BF16:
        return w[0][e].to(torch.float64)
    if fmt == INT8:
        return w[0][e].to(torch.float64).mul_(w[1][e].to(torch.float64).unsqueeze(1))
    c = w[0][e].to(torch.int64)
    c = torch.dstack([c % 16, c // 16]).reshape(c.shape[0], -1)
    m, x = c % 2, c // 2 % 4                      # one bit of mantissa, two of exponent
    v = torch.where(x == 0, m / 2, (1 + m / 2) * 2.0 ** (x - 1)).to(torch.float64)
    s = w[1][e].view(torch.float8_e4m3fn).to(torch.float64) * w[2][e].to(torch.float64)
    return torch.where(c >= 8, -v, v) * s.repeat_interleave(16, dim=1)


def _exact_act(z, act, N):
    if act == NONE:
        return z
    if act == RELU:
        return z.clamp_min(0)
    if act == GELU:
        return z * torch.special.ndtr(z)
    if act == GELU_TANH:
        # 0.5 (1 + tanh v) = sigmoid(2 v)
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == SILU:
        return z * torch.sigmoid(z)
    g, u = z[..., :N], z[..., N:]
    return g * torch.sigmoid(g) * u
