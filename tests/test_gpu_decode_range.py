"""The few-token layer on NVFP4 weights whose tensor scale says little about what they hold: block scales far below E4M3's
largest, single large weights, tokens with single large values, negative scales. The bound is the other formats' (h to 2^-16
of itself), which knows nothing of the tensor scale."""
import pytest
import torch

import precision_moe_numerics_amd as nvq
from bf16_ref import check, out_bound
from decode_ref import check_choice, layer, route, values
from gpu_util import require_gpu
from test_gpu_decode import SIZES, case, rnd, run_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def verify(a, w1, w2):
    out, ids, wts = run_case("nvfp4", a, w1, w2)
    key, lg, dl = route(a["x"], a["w_router"], a["bias"], a["k"], a["router"] == nvq.ROUTER_SIGMOID)
    idc, w, dw = check_choice(ids, wts, key, lg, dl, a["k"], a["router"] == nvq.ROUTER_SIGMOID)
    ref, err = layer(a["x"], idc, w, dw, values(w1, "nvfp4"), values(w2, "nvfp4"), a["residual"])
    check(out, ref, out_bound(ref, err, False), "out")
    return out


def scales_between(w, lo, hi, seed):
    """The weights with block scale bytes drawn anew from lo .. hi - 1 (eight to a power of two)."""
    g = torch.Generator().manual_seed(seed)
    return w[0], torch.randint(lo, hi, w[1].shape, generator=g, dtype=torch.int32).to(torch.uint8).cuda(), w[2]


def loosened(w, n):
    """The same values: the tensor scale times 2^n, block scales divided by it (exponents from 1 up: normal)."""
    assert int(w[1].min()) >= 8 * n + 8
    return w[0], w[1] - 8 * n, w[2] * 2.0 ** n


@pytest.mark.parametrize("T,d,E,k,f", [(1, 4096, 3, 2, 1024), (20, 160, 5, 2, 96), (33, 256, 3, 2, 512), (7, 96, 4, 3, 640)])
def test_block_scales_far_below_the_largest(T, d, E, k, f):
    """Powers of two moved between tensor scale and block scales change no bit: every factor is exact."""
    a, w1, w2 = case("nvfp4", T, d, E, k, f, residual=False)
    w1, w2 = scales_between(w1, 72, 120, 1), scales_between(w2, 72, 120, 2)
    first = verify(a, w1, w2)
    for n in (3, 6, 8):
        assert torch.equal(verify(a, loosened(w1, n), loosened(w2, n)), first), n


@pytest.mark.parametrize("dev", [200, 1000, 20000])
@pytest.mark.parametrize("seen", [False, True])
def test_a_single_large_weight(dev, seen):
    """As the quantizer leaves it: N(0, 0.02) with one gate weight of `dev` deviations in each expert, at a channel where
    x is zero, or not."""
    T, d, E, k, f = 6, 1024, 4, 2, 512
    a, _, _ = case("nvfp4", T, d, E, k, f, residual=False)
    if not seen:
        a["x"][:, 77] = 0.0
    w1, w2 = rnd(3, E, 2 * f, d, std=0.02), rnd(4, E, d, f, std=0.02)
    w1[:, 5, 77] = 0.02 * dev
    verify(a, nvq.nvfp4_quantize(w1, batched=True), nvq.nvfp4_quantize(w2, batched=True))


@pytest.mark.parametrize("T,d,f", [(1, 256, 512), (12, 160, 96)])
def test_a_single_large_value_of_a_token(T, d, f):
    """A channel of x that is 2^34 times the others and that no weight reads."""
    a, w1, w2 = case("nvfp4", T, d, 4, 2, f, residual=False)
    a["x"][:, 6] = 2.0 ** 34
    a["w_router"][:, 6] = 0.0
    w1[0][:, :, 3] &= 0xF0
    verify(a, w1, w2)


@pytest.mark.parametrize("T,d,f", [(3, 256, 512), (17, 160, 96)])
def test_every_finite_scale_byte_of_both_signs(T, d, f):
    a, w1, w2 = case("nvfp4", T, d, 4, 2, f)
    w1, w2 = scales_between(w1, 0, 254, 1), scales_between(w2, 0, 254, 2)
    for w in (w1, w2):
        w[1][w[1] >= 127] += 1  # 0x7F is NaN; the last byte is then 0xFE
    verify(a, w1, w2)


@pytest.mark.parametrize("T,d,E,k,f", SIZES)
def test_every_size_within_the_other_formats_bound(T, d, E, k, f):
    verify(*case("nvfp4", T, d, E, k, f, sigmoid=k % 2 == 1, bias=True, residual=T % 2 == 0))


@pytest.mark.parametrize("T", [8, 9, 15, 16, 17, 24, 25, 31, 64])
@pytest.mark.parametrize("f", [96, 512])
def test_blocks_of_eight_tokens(T, f):
    """One expert of every token beside others of a few: blocks of eight that are full, one short, one over."""
    verify(*case("nvfp4", T, 128, 12, 3, f, hot=50.0, residual=False))
