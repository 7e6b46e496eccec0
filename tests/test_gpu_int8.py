"""The int8 quantizer and products against 64-bit references: codes bit for bit, products within the bounds of
int8_ref.py, at sizes on both sides of each kernel's rule, on extreme codes and non-finite rows."""
import pytest
import torch

import precision_moe_numerics_amd as nvq
from bf16_ref import (GELU, GELU_TANH, NONE, RELU, SILU, SWIGLU, U8, U23, act_bound, act_ref, check, d64, out_bound,
                      segments)
from gpu_util import require_gpu
from int8_ref import product, quantize, with_bias

pytestmark = pytest.mark.gpu

BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8
ACTS = [NONE, RELU, GELU, GELU_TANH, SILU, SWIGLU]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rnd(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std).to(dtype).cuda()


def codes(seed, *shape, scale=0.01):
    """Codes over the whole type, -128 among them, and scales of any size."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)
    s = torch.rand(shape[:-1], generator=g).add(0.1).mul(scale)
    return q.cuda(), s.cuda()


def same_bits(a, b):
    return torch.equal(a.cpu().view(torch.int32), b.cpu().view(torch.int32))


def check_quantize(x):
    c, s = nvq.int8_quantize(x)
    rc, rs = quantize(x)
    assert c.shape == x.shape and s.shape == x.shape[:-1]
    assert torch.equal(c.cpu(), rc)
    nan = torch.isnan(rs)
    assert torch.equal(torch.isnan(s.cpu()), nan) and same_bits(s.cpu()[~nan], rs[~nan])


# ------------------------------------------------------------------ quantize
@pytest.mark.parametrize("shape", [(1, 16), (16,), (3, 48), (2, 3, 80), (1, 4096), (7, 4096), (5, 4112), (3, 2048), (2, 8192),
                                   (2, 8208), (2, 16400), (3, 65536), (4095, 64), (4096, 64), (4097, 528), (4099, 1040),
                                   (4098, 2064), (4097, 4096), (0, 64)])
def test_quantize(shape):
    x = rnd(1, *shape)
    if x.dim() > 1 and x.shape[0] > 1:  # rows of every size, the smallest subnormal
        e = torch.linspace(-132, 126, x.shape[0], dtype=torch.float64).round()
        x = (d64(x) / 8 * (2.0 ** e).view(-1, *[1] * (x.dim() - 1))).to(BF16).cuda()
    check_quantize(x)


@pytest.mark.parametrize("top", [1.0, 1.9921875, 127.0, 2.0 ** -126, 2.0 ** -133, 3.3895313892515355e38, 0.01, 254.0 * 2 ** 90])
def test_quantize_every_value_under_a_maximum(top):
    """All bf16 magnitudes up to the row's maximum, of both signs."""
    t = torch.tensor(top, dtype=BF16)
    bits = torch.arange(0, int(t.view(torch.int16)) + 1, dtype=torch.int32)
    x = torch.cat([bits, bits | 0x8000])
    x = torch.cat([x, torch.zeros(-len(x) % 16, dtype=torch.int32)]).to(torch.int16).view(BF16)
    check_quantize(x[None].cuda())


def test_quantize_ties_zeros_and_non_finite_rows():
    x = torch.zeros((8, 256), dtype=BF16)
    x[0, :255] = torch.arange(-127, 128) / 2.0               # maximum 63.5: codes x * 2
    x[1, :254] = torch.arange(-127, 127).add(0.5)            # with 127 below: all ties
    x[1, 254] = 127.0
    x[3, 5] = float("inf")
    x[4, 250] = float("nan")
    x[5, 0], x[5, 255] = -float("inf"), 1.0
    x[6] = -0.0
    x[7, 17] = -2.0 ** -133
    check_quantize(x.cuda())
    big = torch.zeros((2, 16400), dtype=BF16)
    big[0, 16399] = float("nan")
    big[1, 9000] = 3.0
    check_quantize(big.cuda())


@pytest.mark.parametrize("shape", [(1, 16), (5, 48), (2, 3, 4112), (4097, 528), (0, 64)])
def test_dequantize(shape):
    q, s = codes(2, *shape)
    if s.numel() > 1:
        s.view(-1)[0] = float("nan")
    ref = q.cpu().float() * s.cpu()[..., None]
    out = nvq.int8_dequantize(q, s)
    assert out.dtype == F32 and torch.equal(out.cpu().nan_to_num(7.0), ref.nan_to_num(7.0))
    assert torch.equal(nvq.int8_dequantize(q, s, out_dtype=BF16).cpu().nan_to_num(7.0), ref.to(BF16).nan_to_num(7.0))


def test_quantize_then_dequantize_is_within_half_a_step():
    x = rnd(3, 130, 1024)
    c, s = nvq.int8_quantize(x)
    # half a step of the exact maximum / 127, the scale's rounding times up to 127, the product's rounding
    step = d64(x).abs().amax(1, keepdim=True) / 127
    err = (d64(nvq.int8_dequantize(c, s)) - d64(x)).abs()
    assert (err <= step * 0.5 + step * 127 * 2.0 ** -23).all()


# ------------------------------------------------------------------ dense product
SIZES = [(1, 8, 16), (1, 1024, 4096), (8, 64, 512), (17, 72, 208), (33, 520, 48), (64, 2048, 1024), (129, 136, 64),
         (300, 264, 1040), (512, 1024, 4096), (513, 1032, 144)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("bias,residual,f32", [(True, True, False), (False, False, True)])
def test_linear(act, M, N, K, bias, residual, f32):
    linear_case(act, M, N, K, bias, residual, f32)


@pytest.mark.parametrize("act", [NONE, GELU, SWIGLU])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,N,K", [(2090, 7240, 80), (4096, 4096, 272), (257, 17000, 128)])
def test_linear_large(act, f32, M, N, K):
    """The 256 x 256 tiles, with ragged edges on every side, and many tiles per workgroup."""
    linear_case(act, M, N, K, True, True, f32)


def linear_case(act, M, N, K, bias, residual, f32):
    rows = 2 * N if act == SWIGLU else N
    xq, wq = codes(1, M, K, scale=0.02), codes(2, rows, K, scale=2 * K ** -0.5 / 40)
    b = rnd(3, rows, dtype=F32) if bias else None
    r = rnd(4, M, N) if residual else None
    out = nvq.linear_act_int8(xq, wq, bias=b, act=act, residual=r, out_dtype=F32 if f32 else BF16)
    z, dz = with_bias(*product(*xq, *wq), b)
    ref, err = act_ref(z, act, N)[0], act_bound(z, dz, act, N)
    if residual:
        ref = ref + d64(r)
        err = err + ref.abs() * U23
    check(out, ref, out_bound(ref, err, f32), "out")
    assert torch.equal(nvq.linear_act_int8(xq, wq, bias=b, act=act, residual=r, out_dtype=F32 if f32 else BF16), out)


@pytest.mark.parametrize("M,N", [(4, 16), (200, 136)])
def test_linear_largest_sums(M, N):
    """K at its limit with every code at -128 or 127: sums up to 2147221504, exact in int32."""
    K = 131056
    x, w = torch.full((M, K), -128, dtype=I8), torch.full((N, K), -128, dtype=I8)
    w[1::2] = 127
    x[1, ::2] = 127
    one, half = torch.ones(M, device="cuda"), torch.full((N,), 0.5, device="cuda")
    z, dz = product(x, one, w, half)
    out = nvq.linear_act_int8((x.cuda(), one), (w.cuda(), half), out_dtype=F32)
    check(out, z, dz, "out")


@pytest.mark.parametrize("M,N,K", [(5, 64, 128), (300, 264, 256), (2090, 7240, 80)])
def test_linear_non_finite_scales_stay_in_their_rows(M, N, K):
    (x, xs), wq = codes(5, M, K), codes(6, N, K)
    clean = nvq.linear_act_int8((x, xs), wq, out_dtype=F32)
    xs2 = xs.clone()
    xs2[M - 2] = float("nan")
    out = nvq.linear_act_int8((x, xs2), wq, out_dtype=F32)
    assert torch.isnan(out[M - 2]).all()
    keep = torch.arange(M, device="cuda") != M - 2
    assert torch.equal(out[keep], clean[keep])


def test_linear_in_place_residual_no_rows_and_streams():
    xq, wq, r = codes(5, 70, 64), codes(6, 72, 64), rnd(7, 70, 72)
    out = nvq.linear_act_int8(xq, wq, residual=r)
    keep = r.clone()
    nvq.linear_act_int8(xq, wq, residual=r, out=r)
    assert torch.equal(out, r)
    assert nvq.linear_act_int8((xq[0][:0], xq[1][:0]), wq).shape == (0, 72)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = nvq.linear_act_int8(xq, wq, residual=keep)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, again)


# ------------------------------------------------------------------ expert products
def order_of(lens, k, seed):
    """Random token slots in segments of the given lengths (assignments each used once), offsets and order."""
    A = sum(lens)
    T = -(-A // k)
    perm = torch.randperm(T * k, generator=torch.Generator().manual_seed(seed))[:A]
    full = torch.cat([perm, torch.full((T * k - A,), -1)])
    return T, torch.tensor(segments(lens), dtype=torch.int32).cuda(), full.to(torch.int32).cuda()


LENS = [[5], [0, 0, 3, 0], [1] * 40, [17, 0, 130, 1, 64, 0], [300, 0, 7, 513], [0, 0], [2000, 1, 900, 0, 1500]]


@pytest.mark.parametrize("lens", LENS, ids=lambda v: "x".join(map(str, v[:6])))
@pytest.mark.parametrize("d,f", [(64, 64), (512, 144), (144, 528)])
def test_fc1_and_fc2(lens, d, f):
    E = len(lens)
    k = min(3, E)
    T, off, order = order_of(lens, k, 1)
    A, n = T * k, sum(lens)
    xq, w1 = codes(2, T, d, scale=0.02), codes(3, E, 2 * f, d, scale=2 * d ** -0.5 / 40)
    h = torch.full((A, f), 7.0, dtype=BF16, device="cuda")
    nvq.moe_fc1_swiglu_int8(xq, off, order, k, w1, h=h)
    hq, w2 = codes(4, A, f, scale=0.02), codes(5, E, d, f, scale=2 * f ** -0.5 / 40)
    y = torch.full((A, d), 7.0, dtype=BF16, device="cuda")
    nvq.moe_fc2_int8(hq, off, order, w2, y=y)
    assert (h[n:] == 7.0).all()
    used = torch.zeros(A, dtype=torch.bool)
    used[order[:n].cpu().long()] = True
    assert (y.cpu()[~used] == 7.0).all()
    seg = off.tolist()
    for e in range(E):
        rows = slice(seg[e], seg[e + 1])
        if seg[e] == seg[e + 1]:
            continue
        src = (order[rows] // k).long()
        z, dz = product(xq[0][src], xq[1][src], w1[0][e], w1[1][e])
        ref = act_ref(z, SWIGLU, f)[0]
        check(h[rows], ref, out_bound(ref, act_bound(z, dz, SWIGLU, f), False), f"h of expert {e}")
        z, dz = product(hq[0][rows], hq[1][rows], w2[0][e], w2[1][e])
        check(y[order[rows].long()], z, out_bound(z, dz, False), f"y of expert {e}")


@pytest.mark.parametrize("T,d,E,k,f", [(1, 64, 4, 2, 64), (33, 256, 8, 2, 512), (256, 256, 8, 2, 512), (700, 128, 40, 8, 96)])
def test_expert_forward(T, d, E, k, f):
    """Staged: each intermediate against the reference of the one before it."""
    g = torch.Generator().manual_seed(T)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    ids[T // 2, k - 1] = -1
    ids[0, 0] = E
    x = rnd(1, T, d)
    w1 = nvq.int8_quantize(rnd(2, E, 2 * f, d, std=d ** -0.5))
    w2 = nvq.int8_quantize(rnd(3, E, d, f, std=f ** -0.5))
    y = torch.full((T, k, d), 7.0, dtype=BF16, device="cuda")
    nvq.moe_expert_fwd_int8(x, ids.cuda(), w1, w2, y=y)
    y2 = torch.full((T, k, d), 7.0, dtype=BF16, device="cuda")
    _, it = nvq.moe_expert_fwd_int8(x, ids.cuda(), w1, w2, export=True, y=y2)
    assert torch.equal(y, y2)
    xc, xs = quantize(x)
    assert torch.equal(it["xq_codes"].cpu(), xc) and same_bits(it["xq_tscale"], xs)
    flat = ids.view(-1)
    live = (flat >= 0) & (flat < E)
    n = int(live.sum())
    order = torch.argsort(torch.where(live, flat, E), stable=True)[:n]
    assert torch.equal(it["sorted2assign"][:n].cpu().long(), order) and int(it["offsets"][E]) == n
    hc, hs = quantize(it["h"][:n])
    assert torch.equal(it["hq_codes"][:n].cpu(), hc) and same_bits(it["hq_tscale"][:n], hs)
    assert (it["hq_codes"][n:] == 0).all() and (it["hq_tscale"][n:] == 0).all()
    yf = y.view(T * k, d)
    assert (yf[(~live).cuda()] == 7.0).all()
    for i, a in enumerate(order.tolist()):
        e = int(flat[a])
        if i % max(1, n // 97) and i != n - 1:
            continue
        z, dz = product(xc[a // k:a // k + 1], xs[a // k:a // k + 1], w1[0][e], w1[1][e])
        ref = act_ref(z, SWIGLU, f)[0]
        check(it["h"][i:i + 1], ref, out_bound(ref, act_bound(z, dz, SWIGLU, f), False), "h")
        z, dz = product(hc[i:i + 1], hs[i:i + 1], w2[0][e], w2[1][e])
        check(yf[a:a + 1], z, out_bound(z, dz, False), "y")


def test_expert_forward_of_no_tokens():
    w1, w2 = codes(1, 4, 64, 32), codes(2, 4, 32, 32)
    ids = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    y, it = nvq.moe_expert_fwd_int8(rnd(1, 0, 32), ids, w1, w2, export=True)
    assert y.shape == (0, 2, 32) and (it["offsets"] == 0).all()


def test_a_non_finite_token_stays_its_own():
    T, d, E, k, f = 40, 64, 4, 2, 64
    ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(i))[:k] for i in range(T)])
    ids = ids.to(torch.int32).cuda()
    x, w1, w2 = rnd(1, T, d), codes(2, E, 2 * f, d, scale=1e-3), codes(3, E, d, f, scale=1e-3)
    clean = nvq.moe_expert_fwd_int8(x, ids, w1, w2)
    x2 = x.clone()
    x2[7, 3], x2[20, 60] = float("nan"), -float("inf")
    y = nvq.moe_expert_fwd_int8(x2, ids, w1, w2)
    assert torch.isnan(y[7]).all() and torch.isnan(y[20]).all()
    keep = torch.ones(T, dtype=torch.bool)
    keep[[7, 20]] = False
    assert torch.equal(y[keep.cuda()], clean[keep.cuda()])


def test_graph_replays_match_eager():
    T, d, E, k, f = 64, 256, 8, 2, 512
    w1 = nvq.int8_quantize(rnd(2, E, 2 * f, d, std=0.02))
    w2 = nvq.int8_quantize(rnd(3, E, d, f, std=0.02))
    sets = []
    for s in range(2):
        g = torch.Generator().manual_seed(s)
        ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
        sets.append((rnd(10 + s, T, d), ids))
    expect = [nvq.moe_expert_fwd_int8(x, ids, w1, w2).clone() for x, ids in sets]
    dense = [nvq.linear_act_int8(nvq.int8_quantize(x), (w1[0][0], w1[1][0]), act=SWIGLU) for x, _ in sets]
    x, ids = sets[0][0].clone(), sets[0][1].clone()
    y = torch.empty((T, k, d), dtype=BF16, device="cuda")
    out = torch.empty((T, f), dtype=BF16, device="cuda")
    q = (torch.empty((T, d), dtype=I8, device="cuda"), torch.empty(T, device="cuda"))
    ws = torch.empty(nvq.lib().moe_expert_fwd_int8_workspace_size(T, d, k, E, f), dtype=torch.uint8, device="cuda")

    def step():
        nvq.moe_expert_fwd_int8(x, ids, w1, w2, y=y, ws=ws)
        nvq.int8_quantize(x, *q)
        nvq.linear_act_int8(q, (w1[0][0], w1[1][0]), act=SWIGLU, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for sel in (1, 0, 1, 1):
        x.copy_(sets[sel][0])
        ids.copy_(sets[sel][1])
        y.zero_()
        out.zero_()
        ws.zero_()
        assert torch.equal(nvq.moe_expert_fwd_int8(*sets[1 - sel], w1, w2), expect[1 - sel])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, expect[sel]) and torch.equal(out, dense[sel])


@pytest.mark.parametrize("shape", [(1024, 2064), (1025, 16), (1025, 1040), (1026, 2048), (1027, 2064), (1, 16400), (1030, 16400)])
def test_quantize_on_both_sides_of_long_and_many_rows(shape):
    test_quantize(shape)


@pytest.mark.parametrize("lens", [[1, 65, 127, 0, 200, 333, 64], [1000]], ids=lambda v: "x".join(map(str, v)))
@pytest.mark.parametrize("d,f", [(512, 2048), (2048, 256), (272, 2064)])
def test_fc1_and_fc2_of_few_tiles(lens, d, f):
    """Segments of some hundred rows and few columns: tiles of 64 rows, with every kind of last tile."""
    test_fc1_and_fc2(lens, d, f)
