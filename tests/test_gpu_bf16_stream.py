"""The persistent 256 x 256 form of the BF16 products over many tiles per
workgroup, as a layer with hundreds of experts runs it: some eight to sixteen
tiles a workgroup, of full, short and empty segments in no order, so that every
pairing of one tile's loads, waits and stores with the next one's occurs.
References in 64 bits, bounds as in bf16_ref, both on the GPU."""
import pytest
import torch

import precision_moe_numerics_amd as nvq
from bf16_ref import GELU_TANH, RELU, SILU, SWIGLU, U8, U23, act_bound, act_ref, segments
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rnd(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def lengths(seed, E, of):
    g = torch.Generator().manual_seed(seed)
    return [of[int(i)] for i in torch.randint(0, len(of), (E,), generator=g)]


def perm(seed, n):
    return torch.randperm(n, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()


def seg_of(lens):
    return torch.tensor(segments(lens), dtype=torch.int32, device="cuda")


def product(a, b):
    """a @ b in 64 bits and the bound of its fp32 sum."""
    a, b = a.double().contiguous(), b.double().contiguous()
    return a @ b, a.shape[1] * U23 * (a.abs() @ b.abs())


def check(got, ref, err, what):
    bound = err + (0.0 if got.dtype is F32 else U8 * (ref.abs() + err)) + 2.0 ** -126
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist())


# 200 experts: 3200 tiles of 256 x 256; 90 of [0, 2, 1, ..]: long runs without a row
WGRAD = [(lengths(1, 200, [0, 0, 1, 7, 63, 64, 65, 128, 130, 300, 511]), 1024, 1024),
         (lengths(2, 200, [0, 0, 1, 64, 65, 129, 320]), 1000, 1016),
         (lengths(3, 300, [0, 0, 0, 0, 0, 2, 70]), 1024, 768),
         ([341] * 160, 1024, 1024)]


@pytest.mark.parametrize("gather", ["", "a", "b", "ab"])
@pytest.mark.parametrize("case", range(len(WGRAD)))
def test_weight_gradients(case, gather):
    lens, M, N = WGRAD[case]
    R, E, off = sum(lens), len(lens), segments(lens)
    T = R // 2 + 1
    ga = perm(31, 2 * R)[:R] % (2 * T) if "a" in gather else None
    gb = perm(32, 3 * R)[:R] % (3 * T) if "b" in gather else None
    a, b = rnd(33, R if ga is None else T, M), rnd(34, R if gb is None else T, N)
    kw = dict(a_gather=ga, a_div=1 if ga is None else 2, b_gather=gb, b_div=1 if gb is None else 3)
    seg = seg_of(lens)
    f32 = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, seg, out_dtype=F32, **kw)
    b16 = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, seg, **kw)
    start = rnd(35, E, M, N)
    acc16 = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, seg, out=start.clone(), accumulate=True, **kw)
    acc32 = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, seg, out=start.float(), accumulate=True, **kw)
    again = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, seg, out_dtype=F32, **kw)
    assert torch.equal(f32, again)
    A = a if ga is None else a[(ga // 2).long()]
    B = b if gb is None else b[(gb // 3).long()]
    for e in range(E):
        ref, err = product(A[off[e]:off[e + 1]].T, B[off[e]:off[e + 1]])
        check(f32[e], ref, err, f"expert {e}")
        check(b16[e], ref, err, f"bf16, expert {e}")
        ref = ref + start[e].double()
        check(acc16[e], ref, err + ref.abs() * U23, f"added to bf16, expert {e}")
        check(acc32[e], ref, err + ref.abs() * U23, f"added to fp32, expert {e}")


ROWS = lengths(4, 64, [0, 1, 64, 65, 128, 129, 190, 256, 257, 300, 511, 512])


@pytest.mark.parametrize("mode", [nvq.FWD, nvq.DGRAD])
@pytest.mark.parametrize("K", [8, 64, 136, 200])
def test_rows(mode, K):
    lens, N = ROWS, 4104
    R, E, off = sum(lens), len(lens), segments(lens)
    T = R // 2 + 1
    a, b = rnd(1, T, K), rnd(2, E, *((N, K) if mode == nvq.FWD else (K, N)))
    g, dst = perm(3, 2 * R)[:R] % (2 * T), perm(4, R)
    rows = a[(g // 2).long()]
    out = torch.full((R + 3, N), 77.0, dtype=BF16, device="cuda")
    nvq.moe_grouped_gemm_bf16(mode, a, b, seg_of(lens), a_gather=g, a_div=2, out_scatter=dst, out=out)
    assert (out[R:] == 77.0).all()
    plain = nvq.moe_grouped_gemm_bf16(mode, rows, b, seg_of(lens), out_dtype=F32)
    back = out[dst.long()]
    for e in range(E):
        s, t = off[e], off[e + 1]
        ref, err = product(rows[s:t], b[e].T if mode == nvq.FWD else b[e])
        check(back[s:t], ref, err, f"gathered and scattered, expert {e}")
        check(plain[s:t], ref, err, f"plain, expert {e}")


@pytest.mark.parametrize("d", [8, 72, 200])
def test_fc1(d):
    lens, f, k = ROWS, 2056, 2
    R, E, off = sum(lens), len(lens), segments(lens)
    T = (R + k - 1) // k
    x, w1, order = rnd(21, T, d), rnd(22, E, 2 * f, d, std=d ** -0.5), perm(23, k * T)
    h, gu = nvq.moe_fc1_swiglu_bf16(x, seg_of(lens), order, k, w1, save_gu=True)
    rows = x[(order // k).long()]
    for e in range(E):
        s, t = off[e], off[e + 1]
        z, dz = product(rows[s:t], w1[e].T)
        check(gu[s:t], z, dz, f"gate and up, expert {e}")
        check(h[s:t], act_ref(z, SWIGLU, f)[0], act_bound(z, dz, SWIGLU, f), f"h, expert {e}")


@pytest.mark.parametrize("mode", [nvq.FWD, nvq.DGRAD, nvq.WGRAD])
@pytest.mark.parametrize("odd", [0, 1])
def test_neighbours_do_not_leak(mode, odd):
    """Every other expert's rows (and weights) are NaN; the others' results have none. K ends inside a stage."""
    lens, N, K = [n for n in ROWS if n], 4104, 104
    R, E, off = sum(lens), len(lens), segments(lens)
    if mode == nvq.WGRAD:
        lens, N, K = [n % 130 for n in ROWS] * 4, 1016, 1000
        R, E, off = sum(lens), len(lens), segments(lens)
    a = rnd(41, R, K)
    b = rnd(42, R, N) if mode == nvq.WGRAD else rnd(42, E, *((N, K) if mode == nvq.FWD else (K, N)))
    for e in range(odd, E, 2):
        a[off[e]:off[e + 1]] = float("nan")
        if mode == nvq.WGRAD:
            b[off[e]:off[e + 1]] = float("nan")
        else:
            b[e] = float("nan")
    out = nvq.moe_grouped_gemm_bf16(mode, a, b, seg_of(lens), out_dtype=F32)
    for e in range(1 - odd, E, 2):
        s, t = off[e], off[e + 1]
        if mode == nvq.WGRAD:
            ref, err = product(a[s:t].T, b[s:t])
            check(out[e], ref, err, f"expert {e}")
        else:
            ref, err = product(a[s:t], b[e].T if mode == nvq.FWD else b[e])
            check(out[s:t], ref, err, f"expert {e}")


@pytest.mark.parametrize("act", [RELU, GELU_TANH, SILU, SWIGLU])
@pytest.mark.parametrize("M,N,K", [(2090, 12000, 136), (8200, 7240, 40)])
def test_dense(act, M, N, K):
    """The activations that no size of the other files takes to this kernel, with every part of the epilogue."""
    wide = 2 * N if act == SWIGLU else N
    x, w, b, r = rnd(11, M, K), rnd(12, wide, K, std=2 * K ** -0.5), rnd(13, wide, dtype=F32), rnd(14, M, N)
    out, z = nvq.linear_act_bf16(x, w, bias=b, act=act, residual=r, save_z=True)
    plain = nvq.linear_act_bf16(x, w, act=act, out_dtype=F32)
    z0, d0 = product(x, w.T)
    zr = z0 + b.double()
    dz = d0 + zr.abs() * U23
    check(z, zr, dz, "z")
    v = act_ref(zr, act, N)[0] + r.double()
    check(out, v, act_bound(zr, dz, act, N) + v.abs() * U23, "out")
    check(plain, act_ref(z0, act, N)[0], act_bound(z0, d0, act, N), "plain")
    nvq.linear_act_bf16(x, w, bias=b, act=act, residual=r, out=r)
    assert torch.equal(out, r)
