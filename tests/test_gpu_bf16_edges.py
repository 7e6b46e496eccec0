"""The BF16 expert layer where its values and sizes are extreme: infinities, NaN
and tails of the activations, empty batches and segments, offsets that
contradict each other."""
import pytest
import torch

import precision_moe_numerics_amd as nvq
from bf16_ref import GELU, GELU_TANH, NONE, RELU, SILU, SWIGLU, act_ref, check
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ACTS = [NONE, RELU, GELU, GELU_TANH, SILU, SWIGLU]
INF, NAN = float("inf"), float("nan")
# rows, outputs, K: the products of a few rows, of 128 x 128 tiles (one per CU, two) and of 256 x 256 tiles
KERNELS = [(5, 64, 8), (2000, 1032, 520), (2090, 7240, 72), (2048, 12008, 8)]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def act_of(vals, up, act, M, N, K, dtype):
    """act at the pre-activations vals (fp32, cycled over N columns; SwiGLU: of the gate, with `up` beside them), set by
    the bias of a product of zeros: one row, which all M have to equal bit for bit."""
    reps = -(-N // vals.numel())
    b = vals.repeat(reps)[:N]
    if act == SWIGLU:
        b = torch.cat([b, up.repeat(reps)[:N]])
    x = torch.zeros((M, K), dtype=BF16, device="cuda")
    w = torch.zeros((b.numel(), K), dtype=BF16, device="cuda")
    out = nvq.linear_act_bf16(x, w, bias=b.cuda(), act=act, out_dtype=dtype)
    raw = out.view(torch.int16 if dtype is BF16 else torch.int32)
    assert torch.equal(raw, raw[:1].expand(M, N))
    return out[0].cpu(), b.double()[None]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", KERNELS)
def test_infinite_and_nan_pre_activations(M, N, K, act, dtype):
    """What the formulas give in 64 bits: +inf stays, z Phi(z), z sigmoid(z) at -inf are -inf * 0, relu(-inf) is 0."""
    vals = torch.tensor([INF, -INF, NAN, 1.0, -1.0, INF, 0.0, 3.0])
    up = torch.tensor([2.0, 2.0, 2.0, INF, INF, -2.0, NAN, -INF])
    got, z = act_of(vals, up, act, M, N, K, dtype)
    ref = z[0].clamp_min(0.0) if act == RELU else act_ref(z, act, N)[0][0]
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.isinf(), ref.isinf())
    assert torch.equal(got[got.isinf()].double(), ref[ref.isinf()])


# Relative errors of the fp32 forms, in u = 2^-23. An exponential's argument a is rounded a few times (tanh GELU: eight,
# of 2^-24 each; else at most two), which moves the result by that part of |a|; the reciprocal, the exponential, the
# products and the polynomial of Phi (fitted to 1e-7, nine steps) stay within 16 u, a derivative's further products within
# 24 u of its terms taken absolutely. Results and factors below 2^-126 may be flushed.
U = 2.0 ** -23


def tail_ref(z, act, n):
    """act_ref with the two GELU forms written without a difference: Phi(z) = erfc(-z / sqrt(2)) / 2 and, by the sigmoid,
    0.5 (1 + tanh v) = sigmoid(2 v). In 64 bits ndtr and 1 + tanh(v) are off by 2^-53 absolutely, which leaves them no
    digits where they are 1e-17."""
    if act == GELU:
        phi = torch.special.erfc(-z * 0.5 ** 0.5) / 2
        return z * phi, (phi + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5,)
    if act == GELU_TANH:
        a = 2 * (2 / torch.pi) ** 0.5
        v = a * (z + 0.044715 * z ** 3)
        q, p = torch.sigmoid(v), torch.sigmoid(-v)
        return z * q, (q + z * q * p * a * (1 + 3 * 0.044715 * z * z),)
    return act_ref(z, act, n)


def argument(z, act):
    if act == GELU:
        return z * z / 2
    return 4 * (1.6 * z.abs() + 0.0715 * z.abs() ** 3) if act == GELU_TANH else z.abs()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", KERNELS)
def test_values_relative_to_themselves(M, N, K, act, dtype):
    """Pre-activations over [-10, 10], every 1/400: tails as exact as the rest."""
    vals = torch.linspace(-10, 10, 8001, dtype=F32)[torch.randperm(8001, generator=torch.Generator().manual_seed(1))]
    vals = vals[vals != 0]
    for part in vals.split(N):
        got, z = act_of(part, torch.full_like(part, 3.0), act, M, N, K, dtype)
        ref = tail_ref(z, act, N)[0][0]
        err = (argument(z[0, :N], act) + 16) * U * ref.abs() + 2.0 ** -120
        if act in (NONE, RELU):
            err = torch.zeros_like(ref)  # a bias and zeros
        check(got, ref, err + (2.0 ** -8 * (ref.abs() + err) if dtype is BF16 else 0.0), "value")


@pytest.mark.parametrize("act", ACTS)
def test_gradients_relative_to_their_terms(act):
    """The pre-activation's gradient at every bf16 z with 2^-8 <= |z| <= 10: in fp32 as the bias gradient of one row, in
    bf16 as dx through the identity."""
    z = torch.arange(0x3B80, 0x4121, dtype=torch.int32).to(torch.int16).view(BF16)
    z = torch.cat([z, -z])[:2 * (z.numel() // 8 * 8)]
    N = z.numel() // 8 * 8
    z = z[:N]
    full = torch.cat([z, torch.full_like(z, 3.0)]) if act == SWIGLU else z
    dout = torch.full((1, N), 0.75, dtype=BF16, device="cuda")
    eye = torch.eye(full.numel(), dtype=BF16, device="cuda")
    dx, _, db = nvq.linear_act_bwd_bf16(dout, torch.zeros((1, full.numel()), dtype=BF16, device="cuda"), eye,
                                        z=full[None].cuda() if act != NONE else None, act=act, need_dw=False, need_dbias=True)
    z64 = full.double()[None]
    parts = tail_ref(z64, act, N)[1]
    ref = 0.75 * torch.cat([p.expand(1, N) for p in parts], 1)
    g = z64[:, :N]
    s = torch.sigmoid(g)
    if act in (NONE, RELU):
        terms = torch.zeros_like(g)
    elif act == GELU:
        terms = torch.special.erfc(-g * 0.5 ** 0.5) / 2 + g.abs() * torch.exp(-g * g / 2) / (2 * torch.pi) ** 0.5
    elif act == GELU_TANH:
        q = torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3))
        terms = q * (1 + 1.6 * g.abs() * (1 + 0.135 * g * g))
    elif act == SILU:
        terms = s * (1 + g.abs())
    else:
        terms = torch.cat([3 * s * (1 + g.abs()), g.abs() * s], 1)
    a = torch.cat([argument(g, act)] * (2 if act == SWIGLU else 1), 1)
    err = 0.75 * terms * (a + 24) * U + 2.0 ** -120
    check(db[None], ref, err, "fp32")
    check(dx, ref, err + 2.0 ** -8 * (ref.abs() + err), "bf16")


@pytest.mark.parametrize("act", ACTS)
def test_values_and_gradients_of_huge_pre_activations(act):
    """Every power of two up to 2^127 with both signs: finite, and what the formulas give (past |z| = 100 exactly z or 0,
    and dout or 0)."""
    p = 2.0 ** torch.arange(4, 128, dtype=torch.float64)
    z = torch.cat([p, -p]).to(BF16)
    N = z.numel()
    got, z64 = act_of(z.float(), torch.ones(N), act, 5, N, 8, F32)
    g = z64[:, :N]
    ref, parts = tail_ref(z64, act, N)
    # of a positive argument past 40 only that it is past 40 matters
    a = argument(g, act)
    err = (torch.where(g > 0, a.clamp_max(40.0), a.clamp_max(1e6)) + 24) * U
    check(got[None], ref, err * ref.abs() + 2.0 ** -110, "value")
    full = z64.to(BF16).cuda()
    rows = full.shape[1]
    dx, _, db = nvq.linear_act_bwd_bf16(torch.full((1, N), 0.75, dtype=BF16, device="cuda"),
                                        torch.zeros((1, 8), dtype=BF16, device="cuda"),
                                        torch.zeros((rows, 8), dtype=BF16, device="cuda"),
                                        z=full if act != NONE else None, act=act, need_dw=False, need_dbias=True)
    ref = 0.75 * torch.cat([q.expand(1, N) for q in parts], 1)
    # (the terms of a derivative are at most 1 + argument times its sigmoid or tail, and cancel by less than that)
    slack = torch.cat([err * (1 + torch.where(g < 0, a.clamp_max(1e6), 0.0))] * len(parts), 1)
    check(db[None], ref, slack * ref.abs() + 2.0 ** -100, "gradient")
    assert (dx == 0).all()


# ------------------------------------------------------------------ nothing to add, nothing to do
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,M,N", [([0, 5, 0], 264, 136), ([0, 40] * 40, 1032, 1544)])
def test_accumulating_nothing_keeps_every_bit(lens, M, N, dtype):
    """An empty segment leaves its matrix as it was: -0 stays -0 (adding a sum of 0 would make it +0), NaN payloads stay.
    The two sizes take 128 x 128 and 256 x 256 tiles."""
    off = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    R, E = sum(lens), len(lens)
    g = torch.Generator().manual_seed(3)
    a, b = (torch.randn((R, c), generator=g).to(BF16).cuda() for c in (M, N))
    out = torch.full((E, M, N), -0.0, dtype=dtype, device="cuda")
    out[0, 0, :4] = NAN
    raw = out.view(torch.int16 if dtype is BF16 else torch.int32)
    raw[0, 1, :4] = raw[0, 0, :4] + 1
    before = raw.clone()
    nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, b, off, out=out, accumulate=True)
    empty = torch.tensor([n == 0 for n in lens], device="cuda")
    assert torch.equal(raw[empty], before[empty])
    assert (out[~empty].abs().amax((1, 2)) > 0).all()


def test_accumulating_no_rows_keeps_every_bit():
    """The dense form: no rows add nothing to dw and dbias."""
    x, w = torch.zeros((0, 64), dtype=BF16, device="cuda"), torch.zeros((72, 64), dtype=BF16, device="cuda")
    dw, db = torch.full((72, 64), -0.0, device="cuda"), torch.full((72,), -0.0, device="cuda")
    nvq.linear_act_bwd_bf16(torch.zeros((0, 72), dtype=BF16, device="cuda"), x, w, dw=dw, dbias=db, accumulate=True)
    assert (dw.view(torch.int32) == -2 ** 31).all() and (db.view(torch.int32) == -2 ** 31).all()


def test_offsets_of_an_empty_batch():
    """The exported offsets of no tokens are all 0, in new tensors and in a caller's buffer that holds an older batch's."""
    E, d, f = 5, 64, 72
    w1, w2 = torch.zeros((E, 2 * f, d), dtype=BF16, device="cuda"), torch.zeros((E, d, f), dtype=BF16, device="cuda")
    x, ids = torch.zeros((0, d), dtype=BF16, device="cuda"), torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    dirty = [torch.full((E + 1,), 77, dtype=torch.int32, device="cuda") for _ in range(8)]
    del dirty  # what torch.empty may give next
    y, it = nvq.moe_expert_fwd_bf16(x, ids, w1, w2, export=True, save_gu=True)
    assert y.shape == (0, 2, d) and it["h"].shape == (0, f) and it["gu"].shape == (0, 2 * f)
    assert (it["offsets"] == 0).all()
    own = torch.full((E + 1,), 77, dtype=torch.int32, device="cuda")
    ws = torch.empty(int(nvq.lib().moe_expert_fwd_bf16_workspace_size(0, d, 2, E, f)), dtype=torch.uint8, device="cuda")
    rc = nvq.lib().moe_expert_fwd_bf16(None, 0, d, None, 2, E, f, w1.data_ptr(), w2.data_ptr(), None,
                                       nvq.C.byref(nvq.MoeBuffers(offsets=own.data_ptr())), ws.data_ptr(), ws.numel(),
                                       torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and (own == 0).all()


@pytest.mark.parametrize("act", [NONE, SILU, SWIGLU])
def test_dense_backward_of_no_rows_for_dx_alone(act):
    rows = 144 if act == SWIGLU else 72
    w, x = torch.zeros((rows, 64), dtype=BF16, device="cuda"), torch.zeros((0, 64), dtype=BF16, device="cuda")
    z = torch.zeros((0, rows), dtype=BF16, device="cuda")
    dx, dw, db = nvq.linear_act_bwd_bf16(torch.zeros((0, 72), device="cuda"), x, w, z=z, act=act, need_dw=False)
    assert dx.shape == (0, 64) and dw is None and db is None


@pytest.mark.parametrize("mode", [nvq.FWD, nvq.DGRAD])
def test_offsets_whose_tiles_pass_32_bits(mode):
    """Offsets that go up to R and down to 0 again by turns, 2048 times: 2^31 and more tiles of clamped segments. No
    tile is taken from outside the table, no row from outside [0, R). (All rows are row 0, stored to row 1.)"""
    R, E, N, K = 5 << 26, 4096, 264, 8
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1::2] = R
    src = torch.zeros(R, dtype=torch.int32, device="cuda")
    dst = torch.ones(R, dtype=torch.int32, device="cuda")
    a = torch.ones((1, K), dtype=BF16, device="cuda")
    b = torch.ones((E, N, K) if mode == nvq.FWD else (E, K, N), dtype=BF16, device="cuda")
    out = torch.full((3, N), 5.0, dtype=BF16, device="cuda")
    nvq.moe_grouped_gemm_bf16(mode, a, b, off, a_gather=src, out_scatter=dst, out=out)
    torch.cuda.synchronize()
    assert (out[0] == 5.0).all() and (out[2] == 5.0).all()
    assert ((out[1] == 5.0) | (out[1] == K)).all()


@pytest.mark.parametrize("act", [NONE, GELU, SWIGLU])
def test_dense_backward_without_the_operand_of_a_gradient_not_asked_for(act):
    """dx needs w, dw needs x, dbias neither, as in the C call; what a gradient needs may not be missing."""
    M, N, K = 50, 72, 64
    rows = 2 * N if act == SWIGLU else N
    g = torch.Generator().manual_seed(5)
    x, w, z, dout = (torch.randn(s, generator=g).to(BF16).cuda() for s in ((M, K), (rows, K), (M, rows), (M, N)))
    z = None if act == NONE else z
    dx, dw, db = nvq.linear_act_bwd_bf16(dout, x, w, z=z, act=act, need_dbias=True)
    assert torch.equal(nvq.linear_act_bwd_bf16(dout, None, w, z=z, act=act, need_dw=False)[0], dx)
    assert torch.equal(nvq.linear_act_bwd_bf16(dout, x, None, z=z, act=act, need_dx=False)[1], dw)
    only = nvq.linear_act_bwd_bf16(dout, None, None, z=z, act=act, need_dx=False, need_dw=False, need_dbias=True)
    assert only[0] is None and only[1] is None and torch.equal(only[2], db)
    for bad in (dict(x=None, w=w), dict(x=x, w=None), dict(x=x, w=w[:-8]), dict(x=x[:-1], w=w), dict(x=x.float(), w=w)):
        with pytest.raises(nvq.NvqError):
            nvq.linear_act_bwd_bf16(dout, bad["x"], bad["w"], z=z, act=act)


def test_dense_backward_of_an_fp32_dout_in_two_parts():
    """dz is a bf16 operand: 2^-8 of it is lost. An fp32 dout split into bf16 hi + lo and given in two calls, the second
    accumulating, leaves 2^-16 (lo is off by half a step of itself, and |lo| <= 2^-8 |dout|)."""
    M, N, K = 300, 72, 64
    g = torch.Generator().manual_seed(6)
    x, w = (torch.randn(s, generator=g).to(BF16).cuda() for s in ((M, K), (N, K)))
    dout = torch.randn((M, N), generator=g).cuda()
    hi = dout.to(BF16)
    lo = (dout - hi.float()).to(BF16)
    _, dw, db = nvq.linear_act_bwd_bf16(hi, x, w, need_dx=False, need_dbias=True)
    nvq.linear_act_bwd_bf16(lo, x, w, need_dx=False, dw=dw, dbias=db, accumulate=True)
    d, x64 = dout.double().cpu(), x.double().cpu()
    s = d.abs().T @ x64.abs()
    check(dw, d.T @ x64, (1.01 * 2.0 ** -16 + (M + 1) * U) * s, "dw")
    check(db, d.sum(0), (1.01 * 2.0 ** -16 + (M + 1) * U) * d.abs().sum(0), "dbias")
    # one call loses what the contract says and no more
    _, one, _ = nvq.linear_act_bwd_bf16(dout, x, w, need_dx=False)
    check(one, d.T @ x64, (1.01 * 2.0 ** -8 + M * U) * s, "dw in one call")


# ------------------------------------------------------------------ calls at once
def test_calls_with_scratch_on_two_streams_at_once():
    """Calls that keep tables, routing or partial sums in scratch memory, interleaved on two streams with different
    segments: each gives what it gives alone. Tile tables of 256 x 256 and 128 x 128 tiles, the whole expert forward, the
    dense backward's dz and bias sums."""
    def rnd(seed, *shape, std=1.0):
        return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(BF16).cuda()

    def side(i):
        lens = [[600, 0, 64, 1023, 1, 400], [1, 700, 300, 0, 87, 1000]][i]
        off = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        R, E, T, k = sum(lens), len(lens), 700, 2
        x, w, ws = rnd(10 + i, R, 72), rnd(20 + i, E, 5512, 72), rnd(22 + i, E, 72, 1032)
        ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(50 + 1000 * i + t))[:k]
                           for t in range(T)]).to(torch.int32).cuda()
        xt, w1, w2 = rnd(30 + i, T, 136), rnd(32 + i, E, 2 * 264, 136, std=0.1), rnd(34 + i, E, 136, 264, std=0.1)
        lx, lw, lz, lg = rnd(40 + i, 900, 136), rnd(42 + i, 2 * 520, 136), rnd(44 + i, 900, 2 * 520), rnd(46 + i, 900, 520)
        return [lambda: nvq.moe_grouped_gemm_bf16(nvq.FWD, x, w, off),
                lambda: nvq.moe_grouped_gemm_bf16(nvq.DGRAD, x, ws, off),
                lambda: nvq.moe_expert_fwd_bf16(xt, ids, w1, w2),
                lambda: torch.cat([t.flatten().float() for t in nvq.linear_act_bwd_bf16(lg, lx, lw, z=lz, act=SWIGLU,
                                                                                        need_dbias=True)])]

    calls = [side(0), side(1)]
    alone = [[c() for c in calls[i]] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for rep in range(8):
        for j in range(4):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    got[i].append((j, calls[i][j]()))
    torch.cuda.synchronize()
    for i in range(2):
        for j, out in got[i]:
            assert torch.equal(out, alone[i][j]), (i, j)


def test_gather_divisors_are_32_bit():
    """A divisor past 32 bits is refused, not cut to its low bits (2^32 + 2 would divide by 2)."""
    a, b = torch.zeros((8, 64), dtype=BF16, device="cuda"), torch.zeros((1, 64, 64), dtype=BF16, device="cuda")
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    g = torch.zeros(8, dtype=torch.int32, device="cuda")
    for div in (0, -1, 2 ** 31, 2 ** 32 + 2):
        with pytest.raises(nvq.NvqError):
            nvq.moe_grouped_gemm_bf16(nvq.FWD, a, b, off, a_gather=g, a_div=div)
        with pytest.raises(nvq.NvqError):
            nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, a, off, b_gather=g, b_div=div)
    nvq.moe_grouped_gemm_bf16(nvq.FWD, a, b, off, a_gather=g, a_div=2 ** 31 - 1)


@pytest.mark.parametrize("lens,N,K", [([3, 0, 2], 200, 72), ([400, 0, 300], 1032, 456), ([600, 0, 64, 1023, 1, 400], 5512, 72)])
def test_rows_before_the_first_and_behind_the_last_segment_are_left(lens, N, K):
    """Segments that start past row 0 and end before the last row: the rows outside, whose gather and scatter entries are
    traps, are neither read nor written, by the products of a few rows, of 128 x 128 and of 256 x 256 tiles."""
    def rnd(seed, *shape):
        return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()

    before, behind, E, k = 5, 9, len(lens), 1
    n = sum(lens)
    R = before + n + behind
    off = (torch.tensor([0] + lens, dtype=torch.int32).cumsum(0) + before).to(torch.int32).cuda()
    inner = slice(before, before + n)
    trap = torch.full((R,), 2 ** 30, dtype=torch.int32, device="cuda")
    idx = trap.clone()
    idx[inner] = torch.randperm(R, generator=torch.Generator().manual_seed(1))[:n].to(torch.int32).cuda()
    a, plain = rnd(2, R, K), off - before
    for mode in (nvq.FWD, nvq.DGRAD):
        b = rnd(3, E, *((N, K) if mode == nvq.FWD else (K, N)))
        out = torch.full((R, N), 77.0, dtype=BF16, device="cuda")
        nvq.moe_grouped_gemm_bf16(mode, a, b, off, a_gather=idx, out_scatter=idx, out=out)
        want = torch.full_like(out, 77.0)
        want[idx[inner].long()] = nvq.moe_grouped_gemm_bf16(mode, a[idx[inner].long()], b, plain)
        assert torch.equal(out, want)
    w1 = rnd(4, E, 2 * N, K)
    h, gu = torch.full((R, N), 77.0, dtype=BF16, device="cuda"), torch.full((R, 2 * N), 77.0, dtype=BF16, device="cuda")
    nvq.moe_fc1_swiglu_bf16(a, off, idx, k, w1, h=h, gu=gu)
    h2, gu2 = nvq.moe_fc1_swiglu_bf16(a[idx[inner].long()], plain, torch.arange(n, dtype=torch.int32, device="cuda"), k, w1,
                                      save_gu=True)
    for got, ref in ((h, h2), (gu, gu2)):
        assert torch.equal(got[inner], ref) and (got[:before] == 77.0).all() and (got[before + n:] == 77.0).all()
    dw = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a, h, off, a_gather=idx)
    ref = nvq.moe_grouped_gemm_bf16(nvq.WGRAD, a[idx[inner].long()], h[inner].contiguous(), plain)
    assert torch.equal(dw, ref)
