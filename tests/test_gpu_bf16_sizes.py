"""The BF16 products over the sizes at which they change kernel, rows per
workgroup, split of K or tile: from one row to many rounds of tiles over the
chip, each with K shorter than, equal to and past a stage, and with widths that
end inside a tile."""
import pytest
import torch

import precision_moe_numerics_amd as nvq
from bf16_ref import GELU, NONE, SWIGLU, act_bound, act_ref, check, d64, matmul_bound, out_bound, segments, U23
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rnd(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float32) * std).to(dtype).cuda()


def perm(seed, n):
    return torch.randperm(n, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()


def seg_of(lens):
    return torch.tensor(segments(lens), dtype=torch.int32, device="cuda")


def ref_rows(mode, a, b, off):
    a, b = d64(a), d64(b)
    N = b.shape[1] if mode == nvq.FWD else b.shape[2]
    ref, err = torch.zeros((a.shape[0], N), dtype=torch.float64), torch.zeros((a.shape[0], N), dtype=torch.float64)
    for e in range(b.shape[0]):
        s, t = off[e], off[e + 1]
        ref[s:t], err[s:t] = matmul_bound(a[s:t], b[e].T if mode == nvq.FWD else b[e])
    return ref, err


MIXED = [600, 0, 64, 1023, 1, 400]
ROWS = [([3, 1, 0], 200, 136), ([5], 8200, 200), ([1] * 9 + [16], 2056, 264), ([9] * 16, 520, 64), ([1], 16392, 72),
        ([20], 72, 1032), ([17] * 8, 584, 200), ([30, 25, 17] * 4, 520, 392), ([19] * 8, 1160, 200), ([31], 10072, 336),
        ([50], 4104, 456), ([33], 8200, 8), ([175], 2280, 808), ([350], 1160, 576),
        ([63, 60], 2056, 520), ([40, 35, 50, 63], 1160, 72), ([64] * 8, 136, 64),
        ([400, 300], 1032, 456), ([1000, 0, 500], 2056, 64), (MIXED, 5512, 8), (MIXED, 5512, 64),
        (MIXED, 5512, 136), ([2000], 8072, 40), (MIXED, 11016, 328), ([256] * 8, 4096, 256), ([257] * 8, 4104, 128),
        ([1, 0, 2, 0] * 1024, 24, 16)]


@pytest.mark.parametrize("mode", [nvq.FWD, nvq.DGRAD])
@pytest.mark.parametrize("lens,N,K", ROWS)
def test_rows(mode, lens, N, K):
    R, E = sum(lens), len(lens)
    T = R // 2 + 1
    a, b = rnd(1, T, K), rnd(2, E, *((N, K) if mode == nvq.FWD else (K, N)))
    g, dst = perm(3, 2 * R)[:R] % (2 * T), perm(4, R)
    rows = a[(g // 2).long()]
    out = torch.full((R + 3, N), 77.0, dtype=BF16, device="cuda")
    nvq.moe_grouped_gemm_bf16(mode, a, b, seg_of(lens), a_gather=g, a_div=2, out_scatter=dst, out=out)
    ref, err = ref_rows(mode, rows, b, segments(lens))
    check(out[:R].cpu()[dst.long().cpu()], ref, out_bound(ref, err, False), "gathered and scattered")
    assert (out[R:] == 77.0).all()
    plain = nvq.moe_grouped_gemm_bf16(mode, rows, b, seg_of(lens), out_dtype=F32)
    check(plain, ref, out_bound(ref, err, True), "plain")


DENSE = [(1, 16392, 72), (3, 8200, 200), (16, 4096, 1032), (31, 16392, 8), (20, 10072, 336), (25, 72, 1032),
         (50, 4104, 456), (100, 8200, 8), (175, 2280, 808), (163, 7688, 8), (450, 1256, 200), (4751, 120, 16),
         (2000, 1032, 520), (2000, 8072, 40), (2048, 8192, 64), (2090, 12000, 136)]


@pytest.mark.parametrize("act", [NONE, GELU, SWIGLU])
@pytest.mark.parametrize("M,N,K", DENSE)
def test_linear(act, M, N, K):
    wide = 2 * N if act == SWIGLU else N
    x, w, b, r = rnd(11, M, K), rnd(12, wide, K, std=2 * K ** -0.5), rnd(13, wide, dtype=F32), rnd(14, M, N)
    out, z = nvq.linear_act_bf16(x, w, bias=b, act=act, residual=r, save_z=True)
    zr, dz = matmul_bound(d64(x), d64(w).T)
    zr = zr + d64(b)
    dz = dz + zr.abs() * U23
    check(z, zr, out_bound(zr, dz, False), "z")
    v = act_ref(zr, act, N)[0] + d64(r)
    check(out, v, out_bound(v, act_bound(zr, dz, act, N) + v.abs() * U23, False), "out")
    plain = nvq.linear_act_bf16(x, w, act=act, out_dtype=F32)
    zr, dz = matmul_bound(d64(x), d64(w).T)
    v = act_ref(zr, act, N)[0]
    check(plain, v, out_bound(v, act_bound(zr, dz, act, N), True), "plain")


FC1 = [([3, 1, 0], 200, 136), ([34], 8216, 8), ([1] * 20, 1024, 72), ([17] * 14 + [3], 856, 8),
       ([1] * 9 + [16], 2056, 264), ([1], 8200, 72), ([7] * 30, 264, 72), ([2] * 40, 104, 136),
       ([17] * 8, 584, 72), ([30, 25, 17] * 4, 264, 264), ([20] * 16, 440, 8), ([50], 2056, 456), ([40, 35, 50, 63], 584, 72),
       ([64, 33] * 2, 1160, 8), ([400, 300], 520, 456), (MIXED, 2696, 72), (MIXED, 5512, 136), ([2000], 4040, 40)]


@pytest.mark.parametrize("lens,f,d", FC1)
def test_fc1(lens, f, d):
    R, E = sum(lens), len(lens)
    k = min(2, E)
    T = (R + k - 1) // k
    x, w1, order = rnd(21, T, d), rnd(22, E, 2 * f, d, std=d ** -0.5), perm(23, k * T)
    off = seg_of(lens)
    h, gu = nvq.moe_fc1_swiglu_bf16(x, off, order, k, w1, save_gu=True)
    rows = x[(order // k).long()][:R]
    z, dz = ref_rows(nvq.FWD, rows, w1, segments(lens))
    check(gu[:R], z, out_bound(z, dz, False), "gate and up")
    ref = act_ref(z, SWIGLU, f)[0]
    check(h[:R], ref, out_bound(ref, act_bound(z, dz, SWIGLU, f), False), "h")


WGRAD = [([9], 1000, 200), ([31], 4088, 4096), ([0, 5] * 40, 504, 256), ([100, 0, 0, 1, 300, 33, 0, 64, 129], 1000, 1280),
         ([64, 128, 0, 1] * 4, 1000, 2040), ([70, 0, 3] * 30, 520, 264), ([0] * 200 + [65], 264, 8)]


@pytest.mark.parametrize("gather", ["", "a", "b", "ab"])
@pytest.mark.parametrize("lens,M,N", WGRAD)
def test_wgrad(gather, lens, M, N):
    R, E = sum(lens), len(lens)
    T = R // 2 + 1
    ga = perm(31, 2 * R)[:R] % (2 * T) if "a" in gather else None
    gb = perm(32, 3 * R)[:R] % (3 * T) if "b" in gather else None
    a, b = rnd(33, R if ga is None else T, M), rnd(34, R if gb is None else T, N)
    kw = dict(a_gather=ga, a_div=1 if ga is None else 2, b_gather=gb, b_div=1 if gb is None else 3)
    f32 = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, seg_of(lens), out_dtype=F32, **kw)
    b16 = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, seg_of(lens), **kw)
    start = rnd(35, E, M, N)
    acc16 = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, seg_of(lens), out=start.clone(), accumulate=True, **kw)
    acc32 = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, seg_of(lens), out=start.float(), accumulate=True, **kw)
    A = d64(a) if ga is None else d64(a)[(ga // 2).long().cpu()]
    B = d64(b) if gb is None else d64(b)[(gb // 3).long().cpu()]
    off = segments(lens)
    for e in range(E):
        if lens[e] == 0:
            assert (f32[e] == 0).all() and (b16[e] == 0).all() and torch.equal(acc16[e], start[e])
            continue
        ref, err = matmul_bound(A[off[e]:off[e + 1]].T, B[off[e]:off[e + 1]])
        check(f32[e], ref, out_bound(ref, err, True), f"expert {e}")
        check(b16[e], ref, out_bound(ref, err, False), f"bf16, expert {e}")
        ref = ref + d64(start[e])
        check(acc16[e], ref, out_bound(ref, err + ref.abs() * U23, False), f"added to bf16, expert {e}")
        check(acc32[e], ref, out_bound(ref, err + ref.abs() * U23, True), f"added to fp32, expert {e}")


# ------------------------------------------------------------------ past 32 bits
def test_outputs_past_32_bits():
    """40000 x 65536 outputs: rows at both ends and on both sides of element 2^31, with a residual and z."""
    M, N, K = 40000, 65536, 8
    x, w = rnd(41, M, K), rnd(42, N, K)
    res = torch.zeros((M, N), dtype=BF16, device="cuda")
    at = [0, 1, 2 ** 31 // N - 1, 2 ** 31 // N, M - 2, M - 1]
    res[at] = rnd(43, len(at), N)
    out, z = nvq.linear_act_bf16(x, w, residual=res, save_z=True)
    ref, err = matmul_bound(d64(x[at]), d64(w).T)
    check(z[at], ref, out_bound(ref, err, False), "z")
    ref = ref + d64(res[at])
    check(out[at], ref, out_bound(ref, err + ref.abs() * U23, False), "out")
    del out, z, res
    got = nvq.moe_grouped_gemm_bf16(nvq.DGRAD, x, w.T.contiguous()[None], seg_of([M]))
    ref, err = matmul_bound(d64(x[at]), d64(w).T)
    check(got[at], ref, out_bound(ref, err, False), "grouped")


@pytest.mark.parametrize("N", [8, 264])
def test_rows_past_4_gib(N):
    """70000 x 32768 rows: the products along K and, with the last rows alone not zero, along the rows."""
    M, K = 70000, 32768
    x = torch.zeros((M, K), dtype=BF16, device="cuda")
    at = [0, 65535, 65536, M - 130, M - 1]
    x[at] = rnd(51, len(at), K)
    w = rnd(52, N, K)
    out = nvq.linear_act_bf16(x, w, out_dtype=F32)
    ref, err = matmul_bound(d64(x[at]), d64(w).T)
    check(out[at], ref, out_bound(ref, err, True), "rows")
    dz = rnd(53, M, N)
    dw = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, dz, x, seg_of([65536, M - 65536]), out_dtype=F32)
    for e, rows in enumerate((at[:2], at[2:])):
        ref, err = matmul_bound(d64(dz[rows]).T, d64(x[rows]))
        check(dw[e], ref, out_bound(ref, err, True), f"weights {e}")


def test_many_tiles_replayed_as_a_graph():
    """Products of many tiles, their tile tables in one workspace, captured once; replays on other rows and segments,
    with eager calls between them, equal the eager results."""
    N, d, E = 5512, 72, len(MIXED)
    R = sum(MIXED)
    w, lw = rnd(61, E, N, d), rnd(62, 2000, d)
    xs, gs = [rnd(63 + i, R, d) for i in range(2)], [rnd(65 + i, R, N) for i in range(2)]
    segs = [seg_of(MIXED), seg_of(MIXED[::-1])]

    def layer(x, g, seg, ws=None):
        return (nvq.moe_grouped_gemm_bf16(nvq.FWD, x, w, seg, ws=ws), nvq.moe_grouped_gemm_bf16(nvq.DGRAD, g, w, seg, ws=ws),
                nvq.moe_grouped_gemm_bf16(nvq.WGRAD, g, x, seg, ws=ws), nvq.linear_act_bf16(x, lw, act=GELU))

    expect = [layer(*a) for a in zip(xs, gs, segs)]
    x, g, seg = xs[0].clone(), gs[0].clone(), segs[0].clone()
    size = int(nvq.lib().moe_grouped_gemm_bf16_workspace_size(nvq.FWD, E, R))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, g, seg, ws)
    for r in (0, 1, 1, 0):
        x.copy_(xs[r]); g.copy_(gs[r]); seg.copy_(segs[r]); ws.fill_(255)
        again = layer(xs[1 - r], gs[1 - r], segs[1 - r])
        graph.replay()
        torch.cuda.synchronize()
        for got, ref, other, eager in zip(out, expect[r], again, expect[1 - r]):
            assert torch.equal(got, ref) and torch.equal(other, eager), f"replay {r}"
