"""The whole expert layer for a few tokens against a 64-bit reference, in every weight format: sizes from one token of a
tiny layer up, experts that many tokens or one token chose, ties, non-finite weights and tokens, both routers."""
import pytest
import torch

import precision_moe_numerics_amd as nvq
from bf16_ref import check, out_bound
from decode_ref import check_choice, layer, route, values
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
FORMATS = ["bf16", "int8", "nvfp4"]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def rnd(seed, *shape, std=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std).to(dtype).cuda()


def nvfp4_weights(seed, E, rows, cols):
    """Codes and scale bytes over their whole ranges (every finite E4M3 magnitude): sizes need no multiple of 128."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 256, (E, rows, cols // 2), generator=g, dtype=torch.int32).to(torch.uint8)
    s = torch.randint(0, 127, (E, rows, cols // 16), generator=g, dtype=torch.int32).to(torch.uint8)
    t = torch.rand(E, generator=g).add(0.5).mul(2.0 ** -7 * cols ** -0.5)
    return c.cuda(), s.cuda(), t.cuda()


def weights(seed, E, rows, cols, fmt):
    if fmt == "nvfp4":
        return nvfp4_weights(seed, E, rows, cols)
    w = rnd(seed, E, rows, cols, std=cols ** -0.5)
    return w if fmt == "bf16" else nvq.int8_quantize(w)


def call(fmt, *args, **kw):
    return getattr(nvq, "moe_layer_decode_" + fmt)(*args, **kw)


def case(fmt, T, d, E, k, f, sigmoid=False, bias=True, residual=True, seed=0, hot=0.0):
    x, wr = rnd(seed + 1, T, d), rnd(seed + 2, E, d, std=d ** -0.5)
    w1, w2 = weights(seed + 3, E, 2 * f, d, fmt), weights(seed + 4, E, d, f, fmt)
    b = rnd(seed + 5, E, dtype=F32, std=0.5) if bias else None
    if hot:  # an expert that every token chooses
        b[E // 2] += hot
    r = rnd(seed + 6, T, d) if residual else None
    return dict(x=x, w_router=wr, k=k, bias=b, router=nvq.ROUTER_SIGMOID if sigmoid else nvq.ROUTER_SOFTMAX, residual=r), w1, w2


def run_case(fmt, a, w1, w2):
    names = dict(bf16=("w1", "w2")).get(fmt, ("w1q", "w2q"))
    return call(fmt, **a, **dict(zip(names, (w1, w2))))


def verify(fmt, a, w1, w2):
    out, ids, wts = run_case(fmt, a, w1, w2)
    sigmoid = a["router"] == nvq.ROUTER_SIGMOID
    key, lg, dl = route(a["x"], a["w_router"], a["bias"], a["k"], sigmoid)
    idc, w, dw = check_choice(ids, wts, key, lg, dl, a["k"], sigmoid)
    ref, err = layer(a["x"], idc, w, dw, values(w1, fmt), values(w2, fmt), a["residual"],
                     w1[2] if fmt == "nvfp4" else None)
    check(out, ref, out_bound(ref, err, False), "out")
    again = run_case(fmt, a, w1, w2)
    assert all(torch.equal(p, q) for p, q in zip((out, ids, wts), again))


# T, d, E, k, f
SIZES = [(1, 32, 1, 1, 32), (1, 256, 8, 2, 512), (2, 64, 4, 4, 96), (3, 1056, 16, 3, 160), (5, 96, 130, 8, 64),
         (8, 512, 24, 8, 256), (16, 288, 5, 2, 352), (17, 128, 3, 1, 128), (33, 160, 9, 3, 96), (64, 256, 8, 2, 128),
         (64, 64, 64, 64, 32), (1, 4096, 12, 8, 1024), (4, 2080, 40, 8, 544), (7, 64, 600, 8, 64), (2, 32, 1024, 5, 32)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,d,E,k,f", SIZES)
def test_layer(fmt, T, d, E, k, f):
    sigmoid = (T + k) % 2 == 1
    verify(fmt, *case(fmt, T, d, E, k, f, sigmoid=sigmoid, bias=sigmoid or k % 2 == 0, residual=T % 3 != 0))


@pytest.mark.parametrize("T,d,E,k,f,fmt", [(1, 8, 2, 1, 8, "bf16"), (3, 40, 4, 2, 24, "bf16"), (5, 16, 3, 2, 16, "int8"),
                                           (9, 48, 4, 3, 80, "int8"), (6, 264, 7, 2, 136, "bf16")])
def test_smallest_multiples(fmt, T, d, E, k, f):
    verify(fmt, *case(fmt, T, d, E, k, f))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [15, 16, 17, 32, 47, 48, 49, 63])
def test_an_expert_of_every_token(fmt, T):
    """Blocks of 16 tokens of one expert: full, one short, one over."""
    verify(fmt, *case(fmt, T, 96, 20, 3, 64, hot=50.0))


@pytest.mark.parametrize("fmt", FORMATS)
def test_equal_keys_choose_the_lower_expert(fmt):
    a, w1, w2 = case(fmt, 6, 64, 150, 5, 32, bias=False)
    a["w_router"][:] = a["w_router"][:1]
    out, ids, wts = run_case(fmt, a, w1, w2)
    assert (ids.cpu() == torch.arange(5, dtype=torch.int32)).all() and torch.allclose(wts.cpu(), torch.full((6, 5), 0.2))
    a["w_router"][70:] = -a["w_router"][70:]
    verify(fmt, a, w1, w2)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_tokens_result_does_not_depend_on_the_others(fmt):
    a, w1, w2 = case(fmt, 24, 256, 12, 4, 128)
    out, ids, wts = run_case(fmt, a, w1, w2)
    for t in (0, 11, 23):
        one = dict(a, x=a["x"][t:t + 1].contiguous(), residual=a["residual"][t:t + 1].contiguous())
        o, i, w = run_case(fmt, one, w1, w2)
        assert torch.equal(i[0], ids[t]) and torch.equal(w[0], wts[t])
        # the order in which the experts' parts are added differs: a few roundings of fp32 before the one to bf16
        verify(fmt, one, w1, w2)


@pytest.mark.parametrize("fmt", FORMATS)
def test_non_finite_weights_reach_only_tokens_that_chose_them(fmt):
    a, w1, w2 = case(fmt, 20, 64, 6, 2, 64)
    clean, ids, wts = run_case(fmt, a, w1, w2)
    bad = 3
    if fmt == "bf16":
        w1, w2 = w1.clone(), w2.clone()
        w1[bad, 5] = float("inf")
        w2[bad, 7] = float("nan")
    elif fmt == "int8":
        w1[1][bad, 5], w2[1][bad] = float("nan"), float("nan")
    else:
        w2[1][bad, :, 0] = 0x7F
    out, ids2, wts2 = run_case(fmt, a, w1, w2)
    hit = (ids == bad).any(1)
    assert 0 < int(hit.sum()) < 20
    assert torch.equal(ids, ids2) and torch.equal(wts, wts2) and torch.equal(out[~hit], clean[~hit])
    assert torch.isnan(out[hit]).any(1).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_non_finite_token_stays_its_own(fmt):
    a, w1, w2 = case(fmt, 20, 64, 6, 2, 64)
    clean, ids, wts = run_case(fmt, a, w1, w2)
    x = a["x"].clone()
    x[4, 3], x[17, 60] = float("nan"), float("inf")
    out, ids2, _ = run_case(fmt, dict(a, x=x), w1, w2)
    keep = torch.ones(20, dtype=torch.bool, device="cuda")
    keep[[4, 17]] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(ids[keep], ids2[keep])
    assert torch.isnan(out[4]).all()
    assert ((ids2 >= 0) & (ids2 < 6)).all() and (ids2[:, 0] != ids2[:, 1]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_residual_in_place_no_tokens_and_a_dirty_workspace(fmt):
    a, w1, w2 = case(fmt, 10, 128, 8, 2, 64)
    out, ids, wts = run_case(fmt, a, w1, w2)
    ws = torch.full((nvq.lib().moe_layer_decode_workspace_size(10, 128, 2, 8, 64),), 255, dtype=torch.uint8, device="cuda")
    res = a["residual"].clone()
    o, _, _ = run_case(fmt, dict(a, residual=res, out=res, ws=ws), w1, w2)
    assert torch.equal(o, out) and o.data_ptr() == res.data_ptr()
    o, i, w = run_case(fmt, dict(a, x=a["x"][:0], residual=None), w1, w2)
    assert o.shape == (0, 128) and i.shape == (0, 2) and w.shape == (0, 2)


@pytest.mark.parametrize("fmt", FORMATS)
def test_two_streams_at_once(fmt):
    """Calls in flight on two streams, each with its own workspace."""
    cases = [case(fmt, T, 256, 16, 4, 128, seed=10 * T) for T in (3, 20)]
    expect = [run_case(fmt, *c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run_case(fmt, *cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(g, expect[i]))


@pytest.mark.parametrize("fmt", FORMATS)
def test_graph_replays_match_eager(fmt):
    a, w1, w2 = case(fmt, 9, 256, 16, 4, 128)
    xs = [rnd(50 + i, 9, 256) for i in range(2)]
    expect = [run_case(fmt, dict(a, x=x), w1, w2) for x in xs]
    x = xs[0].clone()
    o = dict(out=torch.empty_like(expect[0][0]), ids=torch.empty_like(expect[0][1]), weights=torch.empty_like(expect[0][2]),
             ws=torch.empty(nvq.lib().moe_layer_decode_workspace_size(9, 256, 4, 16, 128), dtype=torch.uint8, device="cuda"))
    args = dict(a, x=x, **o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_case(fmt, args, w1, w2)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_case(fmt, args, w1, w2)
    for sel in (1, 0, 1, 1, 0):
        x.copy_(xs[sel])
        for t in o.values():
            t.fill_(77)
        assert torch.equal(run_case(fmt, dict(a, x=xs[1 - sel]), w1, w2)[0], expect[1 - sel][0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o["out"], expect[sel][0]) and torch.equal(o["ids"], expect[sel][1])
        assert torch.equal(o["weights"], expect[sel][2])


@pytest.mark.parametrize("fmt", FORMATS)
def test_agrees_with_the_layer_in_parts(fmt):
    """As a served model uses them: the same weights through the few-token call and through router, expert forward and
    combine. Relative 2-norms: bf16 differs by the roundings of y and of out, 2^-8 each at most; int8 by the rounding of x
    and h to amax / 127, a row's step / sqrt(12) with amax up to 4 (x) and 8 (h) of their deviations, 0.9 % and 1.8 %;
    NVFP4 by that of x and h to E2M1, half a step of at most a third of a value."""
    T, d, E, k, f = 40, 256, 8, 2, 512
    x, wr, b = rnd(1, T, d), rnd(2, E, d, std=d ** -0.5), rnd(5, E, dtype=F32, std=0.5)
    w1, w2 = rnd(3, E, 2 * f, d, std=d ** -0.5), rnd(4, E, d, f, std=f ** -0.5)
    logits = nvq.linear_act_bf16(x, wr, out_dtype=F32)
    ids, wts = nvq.moe_router_softmax_topk(logits, b, k)
    if fmt == "bf16":
        y = nvq.moe_expert_fwd_bf16(x, ids, w1, w2)
        out, i2, w2_ = nvq.moe_layer_decode_bf16(x, wr, k, w1, w2, bias=b)
        tol = 2.0 ** -7
    elif fmt == "int8":
        w1q, w2q = nvq.int8_quantize(w1), nvq.int8_quantize(w2)
        y = nvq.moe_expert_fwd_int8(x, ids, w1q, w2q)
        out, i2, w2_ = nvq.moe_layer_decode_int8(x, wr, k, w1q, w2q, bias=b)
        tol = 2.0 ** -5
    else:
        w1q, w2q = nvq.nvfp4_quantize(w1, batched=True), nvq.nvfp4_quantize(w2, batched=True)
        y = nvq.moe_expert_fwd_nvfp4(x, ids, w1q, w2q)
        out, i2, w2_ = nvq.moe_layer_decode_nvfp4(x, wr, k, w1q, w2q, bias=b)
        tol = 0.3
    assert torch.equal(ids, i2) and torch.allclose(wts, w2_, rtol=1e-5)
    ref = nvq.moe_combine_bf16(y, wts).double()
    assert (out.double() - ref).norm() <= tol * ref.norm()


# Steps are 64 bytes of a weight row: several a wave in fc1 (d 8192), a last part of a wave (d 1152), whole groups of four of
# them in one product only (d 160 and f 512, d 128 and f 640), blocks of 12 and 16 that the waves share unevenly.
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,d,E,k,f", [(3, 8192, 3, 2, 64), (2, 1152, 5, 3, 1536), (10, 160, 6, 2, 512), (9, 128, 6, 4, 640),
                                       (1, 384, 3, 1, 2048), (20, 256, 7, 3, 1024)])
def test_steps_of_long_and_uneven_rows(fmt, T, d, E, k, f):
    verify(fmt, *case(fmt, T, d, E, k, f, sigmoid=True))


# More tasks than 24 per workgroup: the last ones are taken from a counter.
@pytest.mark.parametrize("fmt", FORMATS)
def test_many_tasks(fmt):
    verify(fmt, *case(fmt, 64, 64, 100, 3, 2048))
    verify(fmt, *case(fmt, 5, 32, 100, 64, 2048, sigmoid=True))


@pytest.mark.parametrize("fmt", FORMATS)
def test_most_experts_and_choices(fmt):
    verify(fmt, *case(fmt, 64, 32, 1024, 64, 32, bias=False))
    verify(fmt, *case(fmt, 64, 32, 64, 64, 32, sigmoid=True))


@pytest.mark.parametrize("d,f", [(128, 512), (384, 1024)])
def test_non_finite_nvfp4_scales_reach_only_their_rows(d, f):
    """A scale that is not finite, in the middle of a row and next to other rows' and experts'."""
    a, w1, w2 = case("nvfp4", 12, d, 6, 2, f)
    clean, ids, wts = run_case("nvfp4", a, w1, w2)
    w1, w2 = tuple(t.clone() for t in w1), tuple(t.clone() for t in w2)
    w2[1][2, 9, f // 32], w2[1][4, d - 1, f // 16 - 1] = 0x7F, 0x7F
    out, ids2, wts2 = run_case("nvfp4", a, w1, w2)
    bad = torch.zeros_like(clean, dtype=torch.bool)
    bad[(ids == 2).any(1), 9] = True
    bad[(ids == 4).any(1), d - 1] = True
    assert bad.any() and torch.equal(ids, ids2) and torch.equal(out[~bad], clean[~bad]) and torch.isnan(out[bad]).all()
    w1[1][2, f - 1, d // 16 - 1] = 0x7F  # a gate row: all of what expert 2's tokens get
    out, _, _ = run_case("nvfp4", a, w1, w2)
    hit = (ids == 2).any(1)
    assert hit.any() and torch.isnan(out[hit]).all() and torch.equal(out[~hit & ~bad.any(1)], clean[~hit & ~bad.any(1)])


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_workspace_for_two_captured_graphs(fmt):
    """Two graphs of other sizes that share a workspace, replayed in turn, with eager calls in it between them."""
    sizes = [(3, 256, 16, 4, 128), (20, 128, 8, 2, 512)]
    cases = [case(fmt, *s, seed=20 * i) for i, s in enumerate(sizes)]
    expect = [run_case(fmt, *c) for c in cases]
    need = max(nvq.lib().moe_layer_decode_workspace_size(T, d, k, E, f) for T, d, E, k, f in sizes)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for (a, w1, w2), e in zip(cases, expect):
        o = dict(out=torch.empty_like(e[0]), ids=torch.empty_like(e[1]), weights=torch.empty_like(e[2]), ws=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run_case(fmt, dict(a, **o), w1, w2)
        graphs.append(g)
        outs.append(o)
    for i in (0, 1, 1, 0, 1, 0, 0):
        for n in ("out", "ids", "weights"):
            outs[i][n].fill_(77)
        graphs[i].replay()
        eager = run_case(fmt, dict(cases[1 - i][0], ws=ws), *cases[1 - i][1:])
        torch.cuda.synchronize()
        assert all(torch.equal(outs[i][n], e) for n, e in zip(("out", "ids", "weights"), expect[i]))
        assert all(torch.equal(p, e) for p, e in zip(eager, expect[1 - i]))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("s", [2.0 ** 40, 2.0 ** -40])
def test_large_and_small_activations(fmt, s):
    """x times a power of two, the router's weights divided by it, so that the choice is an ordinary one."""
    a, w1, w2 = case(fmt, 6, 256, 8, 2, 512)
    verify(fmt, dict(a, x=a["x"] * s, w_router=a["w_router"] / s, residual=None), w1, w2)


@pytest.mark.parametrize("fmt", FORMATS)
def test_tokens_of_zeros_and_of_far_apart_values(fmt):
    a, w1, w2 = case(fmt, 5, 256, 8, 2, 512, sigmoid=True)
    x = a["x"].clone()
    x[1] = 0.0
    x[3, 1:] *= 2.0 ** -30
    x[4, ::2] *= 2.0 ** -20
    verify(fmt, dict(a, x=x), w1, w2)
