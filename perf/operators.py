"""The BF16 expert layer's operators and their plain forms, case by case.

Four operators of the unquantized expert layer, which stands beside the NVFP4 and MXFP8 ones: the
matrix products grouped by expert (forward with SwiGLU, forward with scatter, gradients of the rows
and of the weights), the dense product with bias, activation and residual in its epilogue (and its
backward), the weighted combine of the expert outputs (and its backward), and the backward of the
two routers. With `own` true `run` makes the library's calls; with `own` false it computes the same
in elementary torch operations: 32-bit products and sums, one rounding at the end.

A case is a dict; `op` names the path:
  fc1      h = silu(x W1g^T) * (x W1u^T) per expert, with g, u saved
  fc2      y[assignment] = h W2^T per expert, scattered to assignment order
  dgrad    dX rows = dA W1 per expert
  wgrad    dW2 = dY^T H per expert, fp32
  linear   out = act(x W^T + bias) + residual
  linear_bwd  dx, dw and dbias (fp32) of the same
  combine / combine_bwd   out = sum_s w_s y_s + residual; dy, dw
  router_bwd  dlogits of the softmax or sigmoid top-k weights
"""
import math

import torch

own = False

NONE, RELU, GELU, GELU_TANH, SILU, SWIGLU = "none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"
ACTS = (NONE, RELU, GELU, GELU_TANH, SILU, SWIGLU)


def listed():
    moe = dict(d=4096, E=384, k=8, d_ff=1024)   # the moe_layer workload's layer
    return [
        # serving: four sequences, one new token each; every chosen expert's weights are read once
        dict(name="fc1_decode", op="fc1", T=4, skew=0.0, **moe),
        # training: the whole moe_layer batch, experts of very different load
        dict(name="fc1_train", op="fc1", T=16384, skew=1.0, **moe),
        # training: the rows' gradient through W1, K = 2 d_ff
        dict(name="dgrad_train", op="dgrad", T=16384, skew=1.0, **moe),
        # training: the gradient of W2 of every expert, fp32
        dict(name="wgrad_train", op="wgrad", T=16384, skew=1.0, **moe),
        # serving: a shared SwiGLU expert on eight tokens, weights bound
        dict(name="linear_decode", op="linear", M=8, N=1024, K=4096, act=SWIGLU, bias=False, residual=False,
             f32=False),
        # the router's projection: fp32 logits over 384 experts
        dict(name="linear_router", op="linear", M=16384, N=384, K=4096, act=NONE, bias=True, residual=False,
             f32=True),
        # a dense feed-forward product with everything in its epilogue
        dict(name="linear_gelu", op="linear", M=8192, N=8192, K=4096, act=GELU, bias=True, residual=True,
             f32=False),
        # training: the shared expert's first product, a packed batch of odd length
        dict(name="linear_bwd", op="linear_bwd", M=4091, N=1024, K=4096, act=SWIGLU, bias=True, f32=False),
        # the unquantized form of the combine workload
        dict(name="combine", op="combine", T=16384, C=4096, E=384, k=8, drop=0.0, residual=True),
        # its gradient on a padded batch: the padding's assignments are dropped
        dict(name="combine_bwd", op="combine_bwd", T=4093, C=4096, E=384, k=8, drop=0.1),
        # the gradient of the routing weights, both routers
        dict(name="router_softmax_bwd", op="router_bwd", T=16384, E=384, k=8, sigmoid=False),
        dict(name="router_sigmoid_bwd", op="router_bwd", T=256, E=8, k=2, sigmoid=True),
    ]


def _log_int(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / mult)) * mult))


def draw(rng):
    op = rng.choice(["fc1", "fc1", "fc2", "dgrad", "wgrad", "linear", "linear", "linear_bwd", "combine",
                     "combine_bwd", "router_bwd"])
    if op in ("fc1", "fc2", "dgrad", "wgrad"):
        E = _log_int(rng, 4, 384)
        return dict(op=op, T=_log_int(rng, 1, 16384), d=_log_int(rng, 64, 4096, 8), E=E,
                    k=rng.randint(1, min(8, E)), d_ff=_log_int(rng, 64, 1024, 8), skew=rng.choice([0.0, 1.0]))
    if op == "linear":
        act = rng.choice(ACTS)
        return dict(op=op, M=_log_int(rng, 1, 16384), N=_log_int(rng, 8, 4096, 8), K=_log_int(rng, 64, 4096, 8),
                    act=act, bias=rng.random() < 0.5, residual=rng.random() < 0.5, f32=rng.random() < 0.3)
    if op == "linear_bwd":
        # with an activation the gradient of z is a bf16 operand of both products: dw is then asked for in bf16
        act = rng.choice(ACTS)
        return dict(op=op, M=_log_int(rng, 1, 8192), N=_log_int(rng, 8, 4096, 8), K=_log_int(rng, 64, 4096, 8),
                    act=act, bias=rng.random() < 0.5, f32=act == NONE)
    E = _log_int(rng, 8, 384)
    if op == "router_bwd":
        # (one chosen expert has weight 1 and no gradient)
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=rng.randint(2, 8), sigmoid=rng.random() < 0.5)
    c = dict(op=op, T=_log_int(rng, 1, 16384), C=_log_int(rng, 64, 4096, 8), E=E, k=rng.randint(1, 8),
             drop=rng.choice([0.0, 0.1]))
    if op == "combine":
        c["residual"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, std, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _weights(gen, E, rows, cols):
    w = torch.empty((E, rows, cols), dtype=torch.bfloat16, device="cuda")
    for e in range(0, E, 32):
        n = min(32, E - e)
        w[e:e + n] = _normal(gen, (n, rows, cols), 0.02)
    return w


def _route(gen, T, E, k, skew):
    """Top-k of N(0, 1) logits (+ a per-expert N(0, 1) load bias): ids, softmax weights, segments, order."""
    logits = torch.randn((T, E), generator=gen, device="cuda")
    if skew:
        key = logits + skew * torch.randn((E,), generator=gen, device="cuda")
    else:
        key = logits
    ids = key.topk(k, dim=1).indices
    weights = torch.softmax(logits.gather(1, ids).double(), 1).float()
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True).to(torch.int32)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return logits, ids.to(torch.int32).contiguous(), weights, offsets, order, offsets.tolist()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    c = dict(case)
    op = c["op"]
    st = {"case": c}
    if op in ("fc1", "fc2", "dgrad", "wgrad"):
        T, d, E, k, f = c["T"], c["d"], c["E"], c["k"], c["d_ff"]
        _, _, _, st["offsets"], st["order"], st["segments"] = _route(gen, T, E, k, c["skew"])
        if op == "fc1":
            st["x"] = _normal(gen, (T, d), 1.0)
            st["w"] = _weights(gen, E, 2 * f, d)
        elif op == "fc2":
            st["x"] = _normal(gen, (T * k, f), 0.5)
            st["w"] = _weights(gen, E, d, f)
        elif op == "dgrad":
            st["x"] = _normal(gen, (T * k, 2 * f), 1e-3)
            st["w"] = _weights(gen, E, 2 * f, d)
        else:
            st["x"] = _normal(gen, (T * k, d), 1e-3)       # dY in assignment order
            st["h"] = _normal(gen, (T * k, f), 0.5)        # H in sorted order
    elif op in ("linear", "linear_bwd"):
        M, N, K = c["M"], c["N"], c["K"]
        rows = 2 * N if c["act"] == SWIGLU else N
        st["x"] = _normal(gen, (M, K), 1.0)
        st["w"] = _normal(gen, (rows, K), 0.02)
        st["bias"] = _normal(gen, (rows,), 0.1, torch.float32) if c["bias"] else None
        if op == "linear":
            st["residual"] = _normal(gen, (M, N), 1.0) if c["residual"] else None
        else:
            z = st["x"].float() @ st["w"].float().T
            if c["bias"]:
                z += st["bias"]
            st["z"] = z.to(torch.bfloat16) if c["act"] != NONE else None
            st["dout"] = _normal(gen, (M, N), 1e-3)
    elif op in ("combine", "combine_bwd"):
        T, C, E, k = c["T"], c["C"], c["E"], c["k"]
        _, ids, st["weights"], _, _, _ = _route(gen, T, E, k, 0.0)
        st["y"] = torch.empty((T, k, C), dtype=torch.bfloat16, device="cuda")
        for t in range(0, T, 2048):
            n = min(2048, T - t)
            st["y"][t:t + n] = _normal(gen, (n, k, C), 1.0)
        if c["drop"]:
            pad = torch.rand((T,), generator=gen, device="cuda") < c["drop"]
            ids[pad] = -1
            st["y"][pad] = float("nan")      # what fc2 never wrote
        st["ids"] = ids
        if op == "combine":
            st["residual"] = _normal(gen, (T, C), 1.0) if c["residual"] else None
        else:
            st["dout"] = _normal(gen, (T, C), 1e-3)
    else:
        T, E, k = c["T"], c["E"], c["k"]
        st["logits"], st["ids"], st["weights"], _, _, _ = _route(gen, T, E, k, 0.0)
        if c["sigmoid"]:
            s = torch.sigmoid(st["logits"].double().gather(1, st["ids"].long()))
            st["weights"] = (s / s.sum(1, keepdim=True)).float()
        st["dweights"] = torch.randn((T, k), generator=gen, device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    import precision_moe_numerics_amd as nvq
    c = st["case"]
    op = c["op"]
    if op == "fc1":
        return nvq.moe_fc1_swiglu_bf16(st["x"], st["offsets"], st["order"], c["k"], st["w"], save_gu=True)
    if op == "fc2":
        return nvq.moe_grouped_gemm_bf16(nvq.FWD, st["x"], st["w"], st["offsets"], out_scatter=st["order"])
    if op == "dgrad":
        return nvq.moe_grouped_gemm_bf16(nvq.DGRAD, st["x"], st["w"], st["offsets"])
    if op == "wgrad":
        return nvq.moe_grouped_gemm_bf16(nvq.WGRAD, st["x"], st["h"], st["offsets"], a_gather=st["order"],
                                         out_dtype=torch.float32)
    if op in ("linear", "linear_bwd"):
        act = {NONE: nvq.ACT_NONE, RELU: nvq.ACT_RELU, GELU: nvq.ACT_GELU, GELU_TANH: nvq.ACT_GELU_TANH,
               SILU: nvq.ACT_SILU, SWIGLU: nvq.ACT_SWIGLU}[c["act"]]
        if op == "linear":
            return nvq.linear_act_bf16(st["x"], st["w"], bias=st["bias"], act=act, residual=st["residual"],
                                       out_dtype=torch.float32 if c["f32"] else torch.bfloat16)
        dx, dw, db = nvq.linear_act_bwd_bf16(st["dout"], st["x"], st["w"], z=st["z"], act=act,
                                             dw_dtype=torch.float32 if c["f32"] else torch.bfloat16,
                                             need_dbias=c["bias"])
        return (dx, dw, db) if c["bias"] else (dx, dw)
    if op == "combine":
        return nvq.moe_combine_bf16(st["y"], st["weights"], topk_ids=st["ids"], E=c["E"], residual=st["residual"])
    if op == "combine_bwd":
        return nvq.moe_combine_bwd_bf16(st["dout"], st["y"], st["weights"], topk_ids=st["ids"], E=c["E"])
    if c["sigmoid"]:
        return nvq.moe_router_sigmoid_topk_bwd(st["weights"], st["logits"], st["ids"], st["dweights"])
    return nvq.moe_router_softmax_topk_bwd(st["weights"], st["ids"], st["dweights"], c["E"])


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
        g, u = z.chunk(2, dim=1)
        return g * u / (1 + torch.exp(-g))
    return z


def _act_bwd(dout, z, act):
    if act == NONE:
        return dout
    if act == RELU:
        return torch.where(z > 0, dout, torch.zeros_like(dout))
    if act == GELU:
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return dout * (cdf + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    if act == GELU_TANH:
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return dout * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z))
    if act == SILU:
        s = 1 / (1 + torch.exp(-z))
        return dout * s * (1 + z * (1 - s))
    g, u = z.chunk(2, dim=1)
    s = 1 / (1 + torch.exp(-g))
    return torch.cat([dout * u * s * (1 + g * (1 - s)), dout * g * s], dim=1)


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op in ("fc1", "fc2", "dgrad", "wgrad"):
        return _plain_grouped(st, c, op)
    if op == "linear":
        z = st["x"].float() @ st["w"].float().T
        if st["bias"] is not None:
            z = z + st["bias"]
        out = _act(z, c["act"])
        if st["residual"] is not None:
            out = out + st["residual"].float()
        return out if c["f32"] else out.to(torch.bfloat16)
    if op == "linear_bwd":
        z = None if st["z"] is None else st["z"].float()
        dz = _act_bwd(st["dout"].float(), z, c["act"])
        dx = (dz @ st["w"].float()).to(torch.bfloat16)
        dw = dz.T @ st["x"].float()
        if not c["f32"]:
            dw = dw.to(torch.bfloat16)
        return (dx, dw, dz.sum(0)) if c["bias"] else (dx, dw)
    if op == "combine":
        live = (st["ids"] >= 0) & (st["ids"] < c["E"])
        out = (torch.where(live[:, :, None], st["y"].float(), 0.0) * st["weights"][:, :, None]).sum(1)
        if st["residual"] is not None:
            out = out + st["residual"].float()
        return out.to(torch.bfloat16)
    if op == "combine_bwd":
        live = (st["ids"] >= 0) & (st["ids"] < c["E"])
        do = st["dout"].float()[:, None, :]
        dy = (torch.where(live, st["weights"], 0.0)[:, :, None] * do).to(torch.bfloat16)
        return dy, (torch.where(live[:, :, None], st["y"].float(), 0.0) * do).sum(2)
    ids = st["ids"].long()
    lg = st["logits"].gather(1, ids)
    dwt = st["dweights"]
    if c["sigmoid"]:
        s = 1 / (1 + torch.exp(-lg))
        tot = s.sum(1, keepdim=True)
        g = (dwt - (dwt * s).sum(1, keepdim=True) / tot) / tot * s * (1 - s)
    else:
        p = torch.exp(lg - lg.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        g = p * (dwt - (dwt * p).sum(1, keepdim=True))
    return torch.zeros_like(st["logits"]).scatter_(1, ids, g)


def _plain_grouped(st, c, op):
    T, d, E, k, f = c["T"], c["d"], c["E"], c["k"], c["d_ff"]
    seg, order, x = st["segments"], st["order"].long(), st["x"]
    A = T * k
    dev = x.device
    if op == "fc1":
        h = torch.empty((A, f), dtype=torch.bfloat16, device=dev)
        gu = torch.empty((A, 2 * f), dtype=torch.bfloat16, device=dev)
    elif op == "wgrad":
        dw = torch.zeros((E, d, f), dtype=torch.float32, device=dev)
    else:
        out = torch.empty((A, d), dtype=torch.bfloat16, device=dev)
    for e in range(E):
        a, b = seg[e], seg[e + 1]
        if a == b:
            continue
        if op == "fc1":
            z = x[order[a:b] // k].float() @ st["w"][e].float().T
            h[a:b] = _act(z, SWIGLU).to(torch.bfloat16)
            gu[a:b] = z.to(torch.bfloat16)
        elif op == "fc2":
            out[order[a:b]] = (x[a:b].float() @ st["w"][e].float().T).to(torch.bfloat16)
        elif op == "dgrad":
            out[a:b] = (x[a:b].float() @ st["w"][e].float()).to(torch.bfloat16)
        else:
            dw[e] = x[order[a:b]].float().T @ st["h"][a:b].float()
    if op == "fc1":
        return h, gu
    return dw if op == "wgrad" else out


# ------------------------------------------------------------------ work and exact values
def work(case):
    c = case
    op = c["op"]
    if op in ("fc1", "fc2", "dgrad", "wgrad"):
        T, d, E, k, f = c["T"], c["d"], c["E"], c["k"], c["d_ff"]
        A = T * k
        hit = E * (1 - (1 - k / E) ** T)       # experts with at least one row under even routing
        idx = 4 * A + 4 * (E + 1)
        if op == "fc1":
            return dict(bytes=2 * T * d + hit * 4 * f * d + A * 6 * f + idx, flops=4 * A * d * f)
        if op == "fc2":
            return dict(bytes=2 * A * f + hit * 2 * f * d + 2 * A * d + idx, flops=2 * A * d * f)
        if op == "dgrad":
            return dict(bytes=4 * A * f + hit * 4 * f * d + 2 * A * d + idx, flops=4 * A * d * f)
        return dict(bytes=2 * A * (d + f) + 4 * E * d * f + idx, flops=2 * A * d * f)
    if op in ("linear", "linear_bwd"):
        M, N, K = c["M"], c["N"], c["K"]
        R = 2 * N if c["act"] == SWIGLU else N
        if op == "linear":
            return dict(bytes=2 * (M * K + R * K) + (4 if c["f32"] else 2) * M * N + (2 * M * N if c["residual"] else 0)
                        + (4 * R if c["bias"] else 0), flops=2 * M * R * K)
        return dict(bytes=2 * (M * N + M * K + R * K) + (2 * M * R if c["act"] != NONE else 0) + 2 * M * K
                    + (4 if c["f32"] else 2) * R * K + (4 * R if c["bias"] else 0), flops=4 * M * R * K)
    T, E, k = c["T"], c["E"], c["k"]
    if op == "combine":
        live = 1 - c["drop"]
        return dict(bytes=2 * T * c["C"] * (live * k + 1 + (1 if c["residual"] else 0)) + 8 * T * k,
                    flops=2 * T * k * c["C"])
    if op == "combine_bwd":
        live = 1 - c["drop"]
        return dict(bytes=2 * T * c["C"] * (live * k + k + 1) + 12 * T * k, flops=3 * T * k * c["C"])
    return dict(bytes=12 * T * k + 4 * T * E, flops=10 * T * k)


def exact(case, seed):
    """The definitions in 64 bits, over masks of the assignments and whole matrices."""
    c = case
    op = c["op"]
    st = prepare(case, seed)
    if op in ("fc1", "fc2", "dgrad", "wgrad"):
        T, d, E, k, f = c["T"], c["d"], c["E"], c["k"], c["d_ff"]
        if op == "wgrad" and E * d * f > 2 ** 29:
            return None
        A = T * k
        o64 = st["offsets"].long()
        expert_of = torch.bucketize(torch.arange(A, device="cuda"), o64[1:], right=True)
        dbl = lambda t: t.to(torch.float64)
        if op == "wgrad":
            res = torch.zeros((E, d, f), dtype=torch.float64, device="cuda")
            src = st["x"].index_select(0, st["order"].long())
        else:
            width = {"fc1": 2 * f, "fc2": d, "dgrad": d}[op]
            res = torch.zeros((A, width), dtype=torch.float64, device="cuda")
            src = st["x"]
            if op == "fc1":
                src = src.index_select(0, torch.div(st["order"].long(), k, rounding_mode="floor"))
        for e in torch.unique(expert_of).tolist():
            rows = (expert_of == e).nonzero(as_tuple=True)[0]
            if op == "wgrad":
                res[e] = torch.mm(dbl(src[rows]).t(), dbl(st["h"][rows]))
                continue
            m = dbl(st["w"][e])
            prod = torch.mm(dbl(src[rows]), m if op == "dgrad" else m.t().contiguous())
            res[st["order"].long()[rows] if op == "fc2" else rows] = prod
        if op == "fc1":
            g, u = res[:, :f], res[:, f:]
            return g * u * torch.sigmoid(g), res
        return res
    x64 = lambda name: st[name].to(torch.float64)
    if op in ("linear", "linear_bwd"):
        act = c["act"]
        N = c["N"]
        if op == "linear":
            z = torch.mm(x64("x"), x64("w").t().contiguous())
            if st["bias"] is not None:
                z += x64("bias")[None, :]
            out = _exact_act(z, act, N)[0]
            return out if st["residual"] is None else out + x64("residual")
        if act == NONE:
            dz = x64("dout")
        else:
            parts = _exact_act(x64("z"), act, N)[1]
            dz = torch.hstack([x64("dout") * p for p in parts])
        res = (torch.mm(dz, x64("w")), torch.mm(dz.t().contiguous(), x64("x")))
        return res + (dz.sum(dim=0),) if c["bias"] else res
    if op in ("combine", "combine_bwd"):
        used = ((st["ids"] >= 0) & (st["ids"] < c["E"])).to(torch.float64)
        w = x64("weights") * used
        if op == "combine":
            res = torch.zeros((c["T"], c["C"]), dtype=torch.float64, device="cuda")
            for t in range(0, c["T"], 1024):
                y = torch.nan_to_num(st["y"][t:t + 1024].to(torch.float64), nan=0.0)
                res[t:t + 1024] = (y * w[t:t + 1024, :, None]).sum(dim=1)
            return res if st["residual"] is None else res + x64("residual")
        dy = x64("dout")[:, None, :] * w[:, :, None]
        dw = torch.empty_like(w)
        for t in range(0, c["T"], 1024):
            y = torch.nan_to_num(st["y"][t:t + 1024].to(torch.float64), nan=0.0)
            dw[t:t + 1024] = (y * x64("dout")[t:t + 1024, None, :]).sum(dim=2)
        return dy, dw * used
    chosen = torch.zeros(st["logits"].shape, dtype=torch.bool, device="cuda").scatter_(1, st["ids"].long(), True)
    up = torch.zeros_like(x64("logits")).scatter_(1, st["ids"].long(), x64("dweights"))
    lg = x64("logits")
    if c["sigmoid"]:
        s = torch.sigmoid(lg) * chosen
        total = s.sum(dim=1, keepdim=True)
        w = s / total
        return torch.where(chosen, (up - (up * w).sum(dim=1, keepdim=True)) / total * s * torch.sigmoid(-lg), 0.0)
    w = torch.softmax(lg.masked_fill(~chosen, float("-inf")), dim=1)
    return w * (up - (up * w).sum(dim=1, keepdim=True))


def _exact_act(z, act, N):
    """(value, factors of dout in dz) in 64 bits."""
    if act == NONE:
        return z, (torch.ones_like(z),)
    if act == RELU:
        return z.clamp_min(0), ((z > 0).to(torch.float64),)
    if act == GELU:
        phi = torch.special.ndtr(z)
        return z * phi, (phi + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi),)
    if act == GELU_TANH:
        # 0.5 (1 + tanh v) = sigmoid(2 v)
        b = 2 * math.sqrt(2 / math.pi)
        q = torch.sigmoid(b * (z + 0.044715 * z ** 3))
        return z * q, (q + z * q * (1 - q) * b * (1 + 0.134145 * z ** 2),)
    if act == SILU:
        q = torch.sigmoid(z)
        return z * q, (q + z * q * torch.sigmoid(-z),)
    g, u = z[:, :N], z[:, N:]
    q = torch.sigmoid(g)
    return g * q * u, (u * (q + g * q * torch.sigmoid(-g)), g * q)
