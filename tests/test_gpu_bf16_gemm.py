"""The grouped BF16 products against 64-bit references: ragged and empty
segments, odd widths, gathers, scatters, accumulation, rows of no expert,
non-finite values next to what a product reads, other streams and replayed
graphs."""
import pytest
import torch

import precision_moe_numerics_amd as nvq
from bf16_ref import act_bound, act_ref, check, d64, matmul_bound, out_bound, segments, SWIGLU
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
RAGGED = [0, 1, 129, 0, 127, 128, 300, 7, 0]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rnd(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std).to(dtype).cuda()


def seg_of(lens):
    return torch.tensor(segments(lens), dtype=torch.int32, device="cuda")


def perm(seed, n):
    return torch.randperm(n, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()


def ref_rows(mode, a, b, off, R):
    """64-bit rows of FWD / DGRAD with the fp32 bound; a already gathered."""
    a, b = d64(a), d64(b)
    N = b.shape[1] if mode == nvq.FWD else b.shape[2]
    ref, err = torch.zeros((R, N), dtype=torch.float64), torch.zeros((R, N), dtype=torch.float64)
    for e in range(b.shape[0]):
        s, t = off[e], off[e + 1]
        ref[s:t], err[s:t] = matmul_bound(a[s:t], b[e].T if mode == nvq.FWD else b[e])
    return ref, err


SHAPES = [([5], 8, 8), ([1], 64, 64), ([0], 16, 16), (RAGGED, 128, 128), (RAGGED, 264, 200), (RAGGED, 120, 72),
          ([64] * 8, 136, 64), ([700, 0, 33], 520, 328), ([1] * 40, 256, 512), ([3, 2, 0, 1] * 16, 48, 1032)]


@pytest.mark.parametrize("mode", [nvq.FWD, nvq.DGRAD])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("lens,N,K", SHAPES)
def test_rows(mode, f32, lens, N, K):
    R, E = sum(lens), len(lens)
    a, b = rnd(1, R, K), rnd(2, E, *((N, K) if mode == nvq.FWD else (K, N)))
    out = nvq.moe_grouped_gemm_bf16(mode, a, b, seg_of(lens), out_dtype=F32 if f32 else BF16)
    ref, err = ref_rows(mode, a, b, segments(lens), R)
    check(out, ref, out_bound(ref, err, f32), "rows")


@pytest.mark.parametrize("mode", [nvq.FWD, nvq.DGRAD])
@pytest.mark.parametrize("lens", [RAGGED, [2, 0, 1, 3], [300, 260]])
def test_gather_scatter_and_rows_of_no_expert(mode, lens):
    """Rows past the last segment hold index and value traps: neither read nor written."""
    n, E, N, K, extra = sum(lens), len(lens), 72, 136, 5
    R = n + extra
    T = R
    src = rnd(3, T, K)
    g = perm(4, 3 * R)[:R] % (3 * T)        # entries / 3 name a source row
    g[n:] = 2 ** 30                          # never read
    dst = torch.full((R,), -7, dtype=torch.int32, device="cuda")
    dst[:n] = perm(5, R)[:n]
    b = rnd(6, E, *((N, K) if mode == nvq.FWD else (K, N)))
    out = torch.full((R, N), 77.0, dtype=BF16, device="cuda")
    nvq.moe_grouped_gemm_bf16(mode, src, b, seg_of(lens), a_gather=g, a_div=3, out_scatter=dst, out=out)
    ref, err = ref_rows(mode, src[(g[:n] // 3).long()], b, segments(lens), n)
    where = dst[:n].long().cpu()
    check(out.cpu()[where], ref, out_bound(ref, err, False), "scattered rows")
    rest = torch.ones(R, dtype=torch.bool)
    rest[where] = False
    assert (out.cpu()[rest] == 77.0).all()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("lens,M,N", [([5], 8, 8), ([0, 3], 16, 16), (RAGGED, 128, 128), (RAGGED, 264, 200),
                                      ([700, 0, 33], 328, 136), ([1] * 20, 72, 256)])
def test_wgrad(f32, lens, M, N):
    R, E = sum(lens), len(lens)
    a, b = rnd(11, R, M), rnd(12, R, N)
    out = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, seg_of(lens), out_dtype=F32 if f32 else BF16)
    off, A, B = segments(lens), d64(a), d64(b)
    for e in range(E):
        ref, err = matmul_bound(A[off[e]:off[e + 1]].T, B[off[e]:off[e + 1]])
        check(out[e], ref, out_bound(ref, err, f32), f"expert {e}")
    assert (out[[n == 0 for n in lens]] == 0).all()


@pytest.mark.parametrize("which", ["a", "b", "both"])
def test_wgrad_gathers_and_accumulates(which):
    lens, M, N, T = RAGGED, 136, 72, 400
    R = sum(lens)
    ga = (perm(21, 2 * R)[:R] % (2 * T)) if which != "b" else None
    gb = (perm(22, 3 * R)[:R] % (3 * T)) if which != "a" else None
    a = rnd(23, T if ga is not None else R, M)
    b = rnd(24, T if gb is not None else R, N)
    start = rnd(25, len(lens), M, N, dtype=F32)
    out = start.clone()
    nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, seg_of(lens), a_gather=ga, a_div=2 if ga is not None else 1,
                              b_gather=gb, b_div=3 if gb is not None else 1, out=out, accumulate=True)
    A = d64(a)[(ga // 2).long().cpu()] if ga is not None else d64(a)
    B = d64(b)[(gb // 3).long().cpu()] if gb is not None else d64(b)
    off = segments(lens)
    for e in range(len(lens)):
        ref, err = matmul_bound(A[off[e]:off[e + 1]].T, B[off[e]:off[e + 1]])
        ref = ref + d64(start[e])
        check(out[e], ref, out_bound(ref, err + U(ref), True), f"expert {e}")
        if lens[e] == 0:
            assert torch.equal(out[e], start[e])
    acc16 = start.to(BF16)
    before = d64(acc16)
    nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, seg_of(lens), a_gather=ga, a_div=2 if ga is not None else 1,
                              b_gather=gb, b_div=3 if gb is not None else 1, out=acc16, accumulate=True)
    for e in range(len(lens)):
        ref, err = matmul_bound(A[off[e]:off[e + 1]].T, B[off[e]:off[e + 1]])
        ref = ref + before[e]
        check(acc16[e], ref, out_bound(ref, err + U(ref), False), f"bf16, expert {e}")


def U(ref):
    return ref.abs() * 2.0 ** -23  # the fp32 addition to the old value


@pytest.mark.parametrize("mode", [nvq.FWD, nvq.DGRAD, nvq.WGRAD])
def test_neighbours_do_not_leak(mode):
    """K, N and the segments end inside tiles; everything outside what an expert reads is NaN."""
    lens, nan = [37, 0, 130, 5], float("nan")
    off, E, N, K = segments(lens), 4, 72, 104
    R = off[-1]
    for e in (0, 2, 3):
        s, t = off[e], off[e + 1]
        if mode == nvq.WGRAD:
            a, b = torch.full((R + 3, K), nan, dtype=BF16, device="cuda"), torch.full((R + 3, N), nan, dtype=BF16, device="cuda")
            a[s:t], b[s:t] = rnd(31, t - s, K), rnd(32, t - s, N)
            out = nvq.moe_grouped_gemm_bf16(mode, a, b, seg_of(lens), out_dtype=F32)[e]
            ref, err = matmul_bound(d64(a[s:t]).T, d64(b[s:t]))
        else:
            a = torch.full((R + 3, K), nan, dtype=BF16, device="cuda")
            b = torch.full((E, *((N, K) if mode == nvq.FWD else (K, N))), nan, dtype=BF16, device="cuda")
            a[s:t], b[e] = rnd(31, t - s, K), rnd(32, *b.shape[1:])
            out = nvq.moe_grouped_gemm_bf16(mode, a, b, seg_of(lens), out_dtype=F32)[s:t]
            ref, err = matmul_bound(d64(a[s:t]), d64(b[e]).T if mode == nvq.FWD else d64(b[e]))
        check(out, ref, out_bound(ref, err, True), f"expert {e}")


def test_non_finite_values_propagate():
    a, b = rnd(41, 40, 64), rnd(42, 1, 64, 64)
    a[3, 5], a[4, 0], a[5, 1] = float("inf"), float("-inf"), float("nan")
    out = d64(nvq.moe_grouped_gemm_bf16(nvq.FWD, a, b, seg_of([40]), out_dtype=F32))
    assert torch.equal(out[3], float("inf") * torch.sign(d64(b)[0, :, 5]))
    assert torch.equal(out[4], float("-inf") * torch.sign(d64(b)[0, :, 0]))
    assert out[5].isnan().all() and out[6:].isfinite().all() and out[:3].isfinite().all()


def test_bad_offsets_stay_in_bounds():
    """Offsets outside [0, R] are clamped and decreasing ones count as empty: no row outside [0, R) is touched."""
    R, N, K = 50, 64, 64
    a, b = rnd(51, R, K), rnd(52, 4, N, K)
    guard = torch.full((R + 100, N), 5.0, dtype=BF16, device="cuda")
    seg = torch.tensor([-20, 10, 2 ** 30, 7, -3], dtype=torch.int32, device="cuda")
    out = nvq.moe_grouped_gemm_bf16(nvq.FWD, a, b, seg, out=guard[:R])
    torch.cuda.synchronize()
    assert (guard[R:] == 5.0).all()
    ref, err = ref_rows(nvq.FWD, a, b[:2], [0, 10, R], R)
    check(out, ref, out_bound(ref, err, False), "clamped segments")


# ------------------------------------------------------------------ fc1 and the whole layer
def ref_fc1(x, w1, off, order, k):
    E, two, _ = w1.shape
    f, A = two // 2, order.numel()
    xs, w = d64(x)[(order // k).long().cpu()], d64(w1)
    z, dz = torch.zeros((A, two), dtype=torch.float64), torch.zeros((A, two), dtype=torch.float64)
    for e in range(E):
        z[off[e]:off[e + 1]], dz[off[e]:off[e + 1]] = matmul_bound(xs[off[e]:off[e + 1]], w[e].T)
    return z, dz, act_ref(z, SWIGLU, f)[0], act_bound(z, dz, SWIGLU, f)


def routed(seed, T, E, k, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    lg = torch.randn((T, E), generator=g) + skew * torch.randn((E,), generator=g)
    ids, w = nvq.moe_router_softmax_topk(lg.cuda(), None, k)
    return lg.cuda(), ids, w


@pytest.mark.parametrize("T,d,E,k,f", [(1, 64, 4, 2, 64), (3, 256, 8, 2, 512), (57, 72, 5, 3, 40), (300, 264, 8, 2, 136),
                                       (256, 256, 8, 2, 512), (700, 128, 3, 3, 200)])
def test_fc1_and_expert_forward(T, d, E, k, f):
    x, w1, w2 = rnd(61, T, d), rnd(62, E, 2 * f, d, std=d ** -0.5), rnd(63, E, d, f, std=f ** -0.5)
    _, ids, _ = routed(64, T, E, k, 1.0)
    off, order, _ = nvq.moe_route(ids, E)
    o = off.tolist()
    h, gu = nvq.moe_fc1_swiglu_bf16(x, off, order, k, w1, save_gu=True)
    z, dz, hr, dh = ref_fc1(x, w1, o, order, k)
    check(gu, z, out_bound(z, dz, False), "gu")
    check(h, hr, out_bound(hr, dh, False), "h")
    y, it = nvq.moe_expert_fwd_bf16(x, ids, w1, w2, export=True, save_gu=True)
    assert torch.equal(it["offsets"], off) and torch.equal(it["sorted2assign"], order)
    assert torch.equal(it["h"], h) and torch.equal(it["gu"], gu)
    ref, err = ref_rows(nvq.FWD, h, w2, o, T * k)
    got = y.view(T * k, d)[order.long()]
    check(got, ref, out_bound(ref, err, False), "y")
    assert torch.equal(nvq.moe_expert_fwd_bf16(x, ids, w1, w2), y)


def test_dropped_assignments_are_left_alone():
    T, d, E, k, f = 40, 64, 6, 2, 64
    x, w1, w2 = rnd(71, T, d), rnd(72, E, 2 * f, d, std=0.1), rnd(73, E, d, f, std=0.1)
    _, ids, _ = routed(74, T, E, k)
    full = nvq.moe_expert_fwd_bf16(x, ids, w1, w2)
    ids2 = ids.clone()
    ids2[::3] = -1
    ids2[1, 0] = E
    y = torch.full((T, k, d), 9.0, dtype=BF16, device="cuda")
    nvq.moe_expert_fwd_bf16(x, ids2, w1, w2, y=y)
    kept = (ids2 >= 0) & (ids2 < E)
    assert torch.equal(y[kept], full[kept]) and (y[~kept] == 9.0).all()


def test_no_rows():
    E, N, K = 3, 64, 64
    e0, b = torch.empty((0, K), dtype=BF16, device="cuda"), rnd(81, E, N, K)
    seg = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    assert nvq.moe_grouped_gemm_bf16(nvq.FWD, e0, b, seg).shape == (0, N)
    out = torch.full((E, K, K), 3.0, device="cuda")
    nvq.moe_grouped_gemm_bf16(nvq.WGRAD, e0, e0, seg, out=out, accumulate=True)
    assert (out == 3.0).all()
    nvq.moe_grouped_gemm_bf16(nvq.WGRAD, e0, e0, seg, out=out)
    assert (out == 0.0).all()
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    assert nvq.moe_expert_fwd_bf16(e0, ids, rnd(82, E, 2 * 64, K), rnd(83, E, K, 64)).shape == (0, 2, K)


def test_streams_and_graph_replays():
    """The layer captured once; replays on changing inputs, with eager work between them, equal the eager calls."""
    T, d, E, k, f = 130, 128, 8, 2, 192
    w1, w2 = rnd(91, E, 2 * f, d, std=0.1), rnd(92, E, d, f, std=0.1)
    xs = [rnd(93 + i, T, d) for i in range(3)]
    rt = [routed(97 + i, T, E, k)[1] for i in range(3)]
    expect = [nvq.moe_expert_fwd_bf16(x, i, w1, w2) for x, i in zip(xs, rt)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = nvq.moe_expert_fwd_bf16(xs[1], rt[1], w1, w2)
    side.synchronize()
    assert torch.equal(other, expect[1])
    x, ids = xs[0].clone(), rt[0].clone()
    y = torch.empty_like(expect[0])
    ws = torch.empty(int(nvq.lib().moe_expert_fwd_bf16_workspace_size(T, d, k, E, f)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nvq.moe_expert_fwd_bf16(x, ids, w1, w2, y=y, ws=ws)
    for r in (0, 1, 2, 1, 0):
        x.copy_(xs[r]); ids.copy_(rt[r]); y.zero_(); ws.fill_(r)
        assert torch.equal(nvq.moe_expert_fwd_bf16(xs[2], rt[2], w1, w2), expect[2])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, expect[r]), f"replay {r}"


# ------------------------------------------------------------------ many tiles
@pytest.mark.parametrize("mode", [nvq.FWD, nvq.DGRAD])
@pytest.mark.parametrize("lens,N,K", [([257, 0, 64, 511, 1], 16392, 72), ([700], 22008, 40), ([300, 200], 22000, 8),
                                      ([513, 129], 22016, 256), ([65, 320], 33000, 328)])
def test_rows_large(mode, lens, N, K):
    R, E = sum(lens), len(lens)
    T = R // 2 + 1
    a, b = rnd(101, T, K), rnd(102, E, *((N, K) if mode == nvq.FWD else (K, N)))
    g = perm(103, 2 * R)[:R] % (2 * T)
    dst = perm(104, R)
    out = torch.full((R + 1, N), 77.0, dtype=BF16, device="cuda")
    nvq.moe_grouped_gemm_bf16(mode, a, b, seg_of(lens), a_gather=g, a_div=2, out_scatter=dst, out=out)
    ref, err = ref_rows(mode, a[(g // 2).long()], b, segments(lens), R)
    check(out.cpu()[dst.long().cpu()], ref, out_bound(ref, err, False), "gathered and scattered")
    assert (out[R] == 77.0).all()
    plain = nvq.moe_grouped_gemm_bf16(mode, a[(g // 2).long()], b, seg_of(lens), out_dtype=F32)
    check(plain, ref, out_bound(ref, err, True), "plain")


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("lens,M,N", [([40, 0, 0, 1, 300, 33, 0, 64, 95], 1032, 1544), ([31], 4104, 4096),
                                      ([0, 5] * 40, 520, 264), ([0] * 300, 264, 8)])
def test_wgrad_large(gather, lens, M, N):
    R, E = sum(lens), len(lens)
    T = R // 2 + 1
    ga = perm(111, 2 * R)[:R] % (2 * T) if gather else None
    a, b = rnd(112, T if gather else R, M), rnd(113, R, N)
    start = rnd(114, E, M, N, dtype=F32)
    out = start.clone()
    nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, seg_of(lens), a_gather=ga, a_div=2 if gather else 1, out=out,
                              accumulate=gather)
    A, B, off = d64(a) if ga is None else d64(a)[(ga // 2).long().cpu()], d64(b), segments(lens)
    for e in range(E):
        ref, err = matmul_bound(A[off[e]:off[e + 1]].T, B[off[e]:off[e + 1]])
        if gather:
            ref = ref + d64(start[e])
        check(out[e], ref, out_bound(ref, err + U(ref), True), f"expert {e}")


def test_fc1_large():
    T, d, E, k, f = 1100, 104, 5, 2, 3304
    x, w1 = rnd(121, T, d), rnd(122, E, 2 * f, d, std=d ** -0.5)
    _, ids, _ = routed(123, T, E, k, 1.0)
    off, order, _ = nvq.moe_route(ids, E)
    h, gu = nvq.moe_fc1_swiglu_bf16(x, off, order, k, w1, save_gu=True)
    z, dz, hr, dh = ref_fc1(x, w1, off.tolist(), order, k)
    check(gu, z, out_bound(z, dz, False), "gu")
    check(h, hr, out_bound(hr, dh, False), "h")
