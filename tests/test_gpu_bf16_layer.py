"""The dense product with its epilogue, the combine and the router gradients
against 64-bit references and differences, and a whole expert layer trained
one step through them."""
import pytest
import torch

import precision_moe_numerics_amd as nvq
from bf16_ref import (GELU, GELU_TANH, NONE, RELU, SILU, SWIGLU, U8, U23, act_bound, act_ref, check, d64,
                      matmul_bound, out_bound)
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ACTS = [NONE, RELU, GELU, GELU_TANH, SILU, SWIGLU]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rnd(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std).to(dtype).cuda()


def pre(x, w, bias):
    z, dz = matmul_bound(d64(x), d64(w).T)
    if bias is not None:
        z = z + d64(bias)
        dz = dz + z.abs() * U23
    return z, dz


# ------------------------------------------------------------------ linear forward
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (1, 1024, 4096), (8, 64, 512), (17, 72, 200), (129, 136, 64), (300, 264, 1032)])
@pytest.mark.parametrize("bias,residual,f32", [(True, True, False), (False, False, True), (True, False, True), (False, True, False)])
def test_linear(act, M, N, K, bias, residual, f32):
    rows = 2 * N if act == SWIGLU else N
    x, w = rnd(1, M, K), rnd(2, rows, K, std=2 * K ** -0.5)
    b = rnd(3, rows, dtype=F32) if bias else None
    r = rnd(4, M, N) if residual else None
    out, z = nvq.linear_act_bf16(x, w, bias=b, act=act, residual=r, out_dtype=F32 if f32 else BF16, save_z=True)
    zr, dz = pre(x, w, b)
    check(z, zr, out_bound(zr, dz, False), "z")
    ref, err = act_ref(zr, act, N)[0], act_bound(zr, dz, act, N)
    if residual:
        ref = ref + d64(r)
        err = err + ref.abs() * U23
    check(out, ref, out_bound(ref, err, f32), "out")
    assert torch.equal(nvq.linear_act_bf16(x, w, bias=b, act=act, residual=r, out_dtype=F32 if f32 else BF16), out)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("f32", [False, True])
def test_linear_large(act, f32):
    """Sizes that take the 256 x 256 tiles, with ragged edges on every side."""
    M, N, K = 2090, 7240, 72
    rows = 2 * N if act == SWIGLU else N
    x, w = rnd(8, M, K), rnd(9, rows, K, std=2 * K ** -0.5)
    b, r = rnd(3, rows, dtype=F32), rnd(4, M, N)
    out, z = nvq.linear_act_bf16(x, w, bias=b, act=act, residual=r, out_dtype=F32 if f32 else BF16, save_z=True)
    zr, dz = pre(x, w, b)
    check(z, zr, out_bound(zr, dz, False), "z")
    ref = act_ref(zr, act, N)[0] + d64(r)
    check(out, ref, out_bound(ref, act_bound(zr, dz, act, N) + ref.abs() * U23, f32), "out")


@pytest.mark.parametrize("act", ACTS)
def test_linear_extreme_pre_activations(act):
    """Pre-activations from -300 to 300 set by the bias: no overflow where the limit is finite."""
    N = 64
    vals = torch.linspace(-300, 300, N, dtype=F32)
    b = (vals if act != SWIGLU else torch.cat([vals, torch.full((N,), 3.0)])).cuda()
    x, w = torch.zeros((5, 8), dtype=BF16, device="cuda"), torch.zeros((b.numel(), 8), dtype=BF16, device="cuda")
    out = nvq.linear_act_bf16(x, w, bias=b, act=act, out_dtype=F32)
    z = d64(b)[None].expand(5, -1)
    ref = act_ref(z, act, N)[0]
    check(out, ref, act_bound(z, torch.zeros_like(z), act, N) + 2.0 ** -126, "out")


def test_linear_residual_in_place_and_no_rows():
    x, w, r = rnd(5, 70, 64), rnd(6, 72, 64), rnd(7, 70, 72)
    out = nvq.linear_act_bf16(x, w, residual=r)
    nvq.linear_act_bf16(x, w, residual=r, out=r)
    assert torch.equal(out, r)
    assert nvq.linear_act_bf16(x[:0], w).shape == (0, 72)
    dw, db = torch.ones((72, 64), device="cuda"), torch.ones(72, device="cuda")
    dx, dw, db = nvq.linear_act_bwd_bf16(r[:0], x[:0], w, dw=dw, dbias=db, accumulate=True)
    assert dx.shape == (0, 64) and (dw == 1).all() and (db == 1).all()
    dx, dw, db = nvq.linear_act_bwd_bf16(r[:0], x[:0], w, dw=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()


# ------------------------------------------------------------------ linear backward
def ref_dz(dout, z, act, N):
    """64-bit dz and a bound of the kernel's fp32 dz: dout times a factor made of exponentials and a few products
    (relative error as in act_bound, of terms no larger than 1 + |z|), which is what the saved bf16 z gives."""
    if act == NONE:
        return dout, torch.zeros_like(dout)
    zz = torch.zeros_like(z)
    parts = act_ref(z, act, N)[1]
    dz = torch.cat([dout * p for p in parts], 1)
    mag = z.abs() if act != SWIGLU else torch.cat([z[:, :N].abs()] * 2, 1)
    arg = mag if act != GELU_TANH else 1.6 * mag + 0.08 * mag ** 3
    size = 1 + mag if act != GELU_TANH else 1 + 1.6 * mag + 0.25 * mag ** 3
    scale = dout.abs() if act != SWIGLU else torch.cat([dout.abs() * z[:, N:].abs(), dout.abs()], 1)
    return dz, scale * size * (arg.clamp_max(40.0) + 16) * U23 + zz[:, :dz.shape[1]]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (5, 520, 64), (130, 72, 136), (300, 264, 200)])
@pytest.mark.parametrize("dout_f32,dw_f32", [(False, True), (True, False)])
def test_linear_bwd(act, M, N, K, dout_f32, dw_f32):
    rows = 2 * N if act == SWIGLU else N
    x, w = rnd(11, M, K), rnd(12, rows, K, std=K ** -0.5)
    z = rnd(13, M, rows, std=1.5) if act != NONE else None
    dout = rnd(14, M, N, dtype=F32 if dout_f32 else BF16)
    dx, dw, db = nvq.linear_act_bwd_bf16(dout, x, w, z=z, act=act, need_dbias=True,
                                         dw_dtype=F32 if dw_f32 else BF16)
    dz, ez = ref_dz(d64(dout), d64(z) if z is not None else None, act, N)
    check(db, dz.sum(0), ez.sum(0) + M * U23 * dz.abs().sum(0) + 2.0 ** -126, "dbias")
    # dz enters the products rounded to bf16: 2^-8 of each element (nothing for a bf16 dout without activation)
    er = ez if act == NONE and not dout_f32 else ez + U8 * (dz.abs() + ez)
    ref, err = matmul_bound(dz, d64(w))
    check(dx, ref, out_bound(ref, err + 1.01 * er @ d64(w).abs(), False), "dx")
    ref, err = matmul_bound(dz.T, d64(x))
    check(dw, ref, out_bound(ref, err + 1.01 * er.T @ d64(x).abs(), dw_f32), "dw")
    # parts of the call equal the whole; accumulation adds
    assert torch.equal(nvq.linear_act_bwd_bf16(dout, x, w, z=z, act=act, need_dw=False)[0], dx)
    assert torch.equal(nvq.linear_act_bwd_bf16(dout, x, w, z=z, act=act, need_dx=False,
                                               dw_dtype=dw.dtype)[1], dw)
    dw0, db0 = torch.full_like(dw, 2.0), torch.full_like(db, 3.0)
    _, dw2, db2 = nvq.linear_act_bwd_bf16(dout, x, w, z=z, act=act, need_dx=False, dw=dw0, dbias=db0, accumulate=True)
    check(dw2, ref + 2.0, out_bound(ref + 2.0, err + 1.01 * er.T @ d64(x).abs() + (ref.abs() + 2) * U23, dw_f32), "dw +=")
    check(db2, dz.sum(0) + 3.0, ez.sum(0) + (M + 1) * U23 * (dz.abs().sum(0) + 3.0), "dbias +=")


@pytest.mark.parametrize("act", ACTS)
def test_linear_bwd_against_differences(act):
    """<dout, act(z + h v)> differenced in 64 bits against the kernel's dz, read through dx with w = identity."""
    M, N = 40, 64
    rows = 2 * N if act == SWIGLU else N
    z = rnd(15, M, rows, std=1.5)
    dout = rnd(16, M, N)
    eye = torch.eye(rows, dtype=BF16, device="cuda")
    dz = d64(nvq.linear_act_bwd_bf16(dout, torch.zeros((M, rows), dtype=BF16, device="cuda"), eye,
                                     z=z if act != NONE else None, act=act, need_dw=False)[0])
    h, z64 = 2.0 ** -16, d64(z)
    for part in range(2 if act == SWIGLU else 1):
        v = torch.zeros_like(z64)
        v[:, part * N:(part + 1) * N] = 1.0
        num = d64(dout) * (act_ref(z64 + h * v, act, N)[0] - act_ref(z64 - h * v, act, N)[0]) / (2 * h)
        # the difference itself is off by h^2 |act'''| / 6 (below 2^-30 |dout|) and 2^-53 / h of |act|
        tol = 1.01 * U8 * num.abs() + 2.0 ** -19 * (1 + d64(dout).abs()) * (1 + z64.abs().amax())
        at_kink = (z64[:, :N].abs() <= h) if act == RELU else torch.zeros_like(num, dtype=torch.bool)
        got = dz[:, part * N:(part + 1) * N]
        assert (((got - num).abs() <= tol) | at_kink).all(), (act, part)


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("T,k,C", [(1, 1, 8), (3, 2, 64), (129, 8, 200), (40, 3, 4096), (7, 17, 1032), (5, 8, 8200)])
@pytest.mark.parametrize("drop", [False, True])
def test_combine_and_backward(T, k, C, drop):
    E = 12
    y, w, res, dout = rnd(21, T, k, C), rnd(22, T, k, dtype=F32), rnd(23, T, C), rnd(24, T, C)
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(25)).to(torch.int32).cuda()
    y64, w64 = d64(y), d64(w)
    kept = torch.ones((T, k), dtype=torch.bool)
    if drop:  # what a dropped slot holds does not matter: not in y, nor in w
        ids[::2, 0] = -1
        ids[T // 2] = E
        kept = ((ids >= 0) & (ids < E)).cpu()
        y[~kept.cuda()] = float("nan")
        w[~kept.cuda()] = float("inf")
        y64, w64 = torch.where(kept[..., None], y64, 0.0), torch.where(kept, w64, 0.0)
    args = dict(topk_ids=ids, E=E) if drop else {}
    for r in (None, res):
        out = nvq.moe_combine_bf16(y, w, residual=r, **args)
        terms = w64[..., None] * y64
        ref = terms.sum(1) + (d64(r) if r is not None else 0.0)
        err = (k + 1) * U23 * (terms.abs().sum(1) + (d64(r).abs() if r is not None else 0.0))
        check(out, ref, out_bound(ref, err, False), "out")
    inplace = res.clone()
    nvq.moe_combine_bf16(y, w, residual=inplace, out=inplace, **args)
    assert torch.equal(inplace, out)
    dy, dw = nvq.moe_combine_bwd_bf16(dout, y, w, **args)
    ref = w64[..., None] * d64(dout)[:, None]
    check(dy, ref, out_bound(ref, ref.abs() * U23, False), "dy")
    prod = y64 * d64(dout)[:, None]
    check(dw, prod.sum(2), C * U23 * prod.abs().sum(2) + 2.0 ** -126, "dw")
    assert (dy[~kept.cuda()] == 0).all() and (dw[~kept.cuda()] == 0).all()


# ------------------------------------------------------------------ router gradients
@pytest.mark.parametrize("T,E,k", [(1, 2, 2), (5, 8, 2), (130, 384, 8), (9, 1000, 64), (4, 64, 64)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_router_bwd(T, E, k, sigmoid):
    lg, dw = rnd(31, T, E, dtype=F32), rnd(32, T, k, dtype=F32)
    if sigmoid:
        ids, w = nvq.moe_router_sigmoid_topk(lg, torch.zeros(E, device="cuda"), k)
        got = nvq.moe_router_sigmoid_topk_bwd(w, lg, ids, dw)
    else:
        ids, w = nvq.moe_router_softmax_topk(lg, None, k)
        got = nvq.moe_router_softmax_topk_bwd(w, ids, dw, E)
    l64 = d64(lg).requires_grad_()
    c = l64.gather(1, ids.cpu().long())
    w64 = torch.sigmoid(c) / torch.sigmoid(c).sum(1, keepdim=True) if sigmoid else torch.softmax(c, 1)
    (w64 * d64(dw)).sum().backward()
    # w is rounded to fp32; D sums k terms, then three or four fp32 steps, an exponential of |logit| <= 6
    spread = (w64.detach() * d64(dw).abs()).sum(1, keepdim=True)
    tol = torch.zeros_like(l64).scatter_(1, ids.cpu().long(),
                                         w64.detach() * (d64(dw).abs() + spread) * (k + 30) * U23)
    check(got, l64.grad, tol + 2.0 ** -126, "dlogits")
    # against differences of the loss along one direction
    v = torch.randn(l64.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(33))
    h = 2.0 ** -17
    def loss(x):
        cc = x.gather(1, ids.cpu().long())
        ww = torch.sigmoid(cc) / torch.sigmoid(cc).sum(1, keepdim=True) if sigmoid else torch.softmax(cc, 1)
        return (ww * d64(dw)).sum(1)
    num = (loss(d64(lg) + h * v) - loss(d64(lg) - h * v)) / (2 * h)
    dirs = (d64(got) * v).sum(1)
    assert ((dirs - num).abs() <= (tol * v.abs()).sum(1) + 2.0 ** -30 * (1 + d64(dw).abs().sum(1)) * v.abs().amax(1) ** 3).all()


def test_router_bwd_ids_out_of_range_and_repeated():
    w = torch.tensor([[0.5, 0.3, 0.2], [0.6, 0.3, 0.1]], device="cuda")
    dw = torch.tensor([[1.0, 2.0, 0.0], [0.0, 1.0, 4.0]], device="cuda")
    ids = torch.tensor([[2, -1, 9], [1, 1, 0]], dtype=torch.int32, device="cuda")
    got = d64(nvq.moe_router_softmax_topk_bwd(w, ids, dw, 4))
    w64, d = d64(w), d64(dw)
    g = w64 * (d - (w64 * d).sum(1, keepdim=True))
    ref = torch.zeros((2, 4), dtype=torch.float64)
    ref[0, 2] = g[0, 0]
    ref[1, 1] = g[1, 0] + g[1, 1]
    ref[1, 0] = g[1, 2]
    assert ((got - ref).abs() <= 8 * U23 * 4).all()
    assert (got[0, [0, 1, 3]] == 0).all()


# ------------------------------------------------------------------ the layer as it is used
def layer_forward(x, wr, w1, w2, k):
    E = wr.shape[0]
    logits = nvq.linear_act_bf16(x, wr, out_dtype=F32)
    ids, w, (off, order, _) = nvq.moe_router_softmax_topk(logits, None, k, route=True)
    h, gu = nvq.moe_fc1_swiglu_bf16(x, off, order, k, w1, save_gu=True)
    y = torch.empty((x.shape[0], k, x.shape[1]), dtype=BF16, device=x.device)
    nvq.moe_grouped_gemm_bf16(nvq.FWD, h, w2, off, out_scatter=order, out=y.view(-1, x.shape[1]))
    return nvq.moe_combine_bf16(y, w, topk_ids=ids, E=E, residual=x), (logits, ids, w, off, order, h, gu, y)


def layer_backward(dout, x, wr, w1, w2, k, saved):
    logits, ids, w, off, order, h, gu, y = saved
    T, d = x.shape
    E = wr.shape[0]
    dy, dw = nvq.moe_combine_bwd_bf16(dout, y, w, topk_ids=ids, E=E)
    dy = dy.view(T * k, d)
    dh = nvq.moe_grouped_gemm_bf16(nvq.DGRAD, dy, w2, off, a_gather=order, out_dtype=F32)
    dw2 = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, dy, h, off, a_gather=order, out_dtype=F32)
    da = nvq.swiglu_bwd(dh, gu)
    dxr = torch.empty((T * k, d), dtype=BF16, device=x.device)
    nvq.moe_grouped_gemm_bf16(nvq.DGRAD, da, w1, off, out_scatter=order, out=dxr)
    dw1 = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, da, x, off, b_gather=order, b_div=k, out_dtype=F32)
    dlogits = nvq.moe_router_softmax_topk_bwd(w, ids, dw, E)
    dxl, dwr, _ = nvq.linear_act_bwd_bf16(dlogits, x, wr)
    ones = torch.ones((T, k), device=x.device)
    # x reaches the output through the experts, the router and, as the residual, directly
    dx = nvq.moe_combine_bf16(dxr.view(T, k, d), ones, residual=dxl + dout)
    return dx, dwr, dw1, dw2


def test_expert_layer_step_against_autograd():
    """Forward and every gradient of a routed layer, chained as a training step chains them, against 64-bit autograd
    on the same routing. Each bf16 intermediate adds a relative 2^-8; at most five follow one another on any path, and
    they add up like independent errors, so 5 * 2^-8 of the 2-norm bounds each output."""
    T, d, E, k, f = 200, 128, 8, 2, 192
    x, wr = rnd(41, T, d), rnd(42, E, d, std=d ** -0.5)
    w1, w2 = rnd(43, E, 2 * f, d, std=d ** -0.5), rnd(44, E, d, f, std=f ** -0.5)
    dout = rnd(45, T, d)
    out, saved = layer_forward(x, wr, w1, w2, k)
    grads = layer_backward(dout, x, wr, w1, w2, k, saved)
    X, WR, W1, W2 = (d64(t).requires_grad_() for t in (x, wr, w1, w2))
    ids = saved[1].cpu().long()
    w = torch.softmax((X @ WR.T).gather(1, ids), 1)
    ref = X.clone()
    for s in range(k):
        z = torch.bmm(W1[ids[:, s]], X[:, :, None]).squeeze(2)
        hh = torch.nn.functional.silu(z[:, :f]) * z[:, f:]
        ref = ref + w[:, s:s + 1] * torch.bmm(W2[ids[:, s]], hh[:, :, None]).squeeze(2)
    ref.backward(d64(dout))
    rel = lambda a, b: ((d64(a) - b).norm() / b.norm()).item()
    for name, got, want in (("out", out, ref.detach()), ("dx", grads[0], X.grad), ("dwr", grads[1], WR.grad),
                            ("dw1", grads[2], W1.grad), ("dw2", grads[3], W2.grad)):
        e = rel(got, want)
        print(f"[layer] {name} relative error {e:.2e}", flush=True)
        assert e <= 5 * U8, (name, e)


def test_layer_step_replayed_as_a_graph():
    """Forward and backward captured together; each replay on new inputs equals the eager step bit for bit."""
    T, d, E, k, f = 96, 64, 8, 2, 128
    wr, w1, w2 = rnd(52, E, d, std=0.1), rnd(53, E, 2 * f, d, std=0.1), rnd(54, E, d, f, std=0.1)
    data = [(rnd(60 + i, T, d), rnd(70 + i, T, d)) for i in range(3)]

    def step(x, dout):
        out, saved = layer_forward(x, wr, w1, w2, k)
        return (out, *layer_backward(dout, x, wr, w1, w2, k, saved))

    expect = [step(*p) for p in data]
    x, dout = data[0][0].clone(), data[0][1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, dout)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, dout)
    for r in (1, 0, 2, 2, 1):
        x.copy_(data[r][0])
        dout.copy_(data[r][1])
        eager = step(*data[(r + 1) % 3])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, expect[r]):
            assert torch.equal(a, b), f"replay {r}"
        for a, b in zip(eager, expect[(r + 1) % 3]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("E", [9])
def test_two_streams_at_once(E):
    """Two calls in flight on two streams, each with its own workspace, give what they give alone."""
    x = [rnd(80 + i, 260, 136) for i in range(2)]
    w = [rnd(82 + i, 264, 136, std=0.1) for i in range(2)]
    alone = [nvq.linear_act_bf16(x[i], w[i], act=nvq.ACT_SILU) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(E):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                outs[i].append(nvq.linear_act_bf16(x[i], w[i], act=nvq.ACT_SILU))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, alone[i])
