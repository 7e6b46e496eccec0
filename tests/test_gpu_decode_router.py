"""The few-token layer's choice against 64-bit logits: products far apart within one logit, logits that differ by less than
fp32 resolves, and weights to fp32's rounding."""
import pytest
import torch

import precision_moe_numerics_amd as nvq
from bf16_ref import d64
from gpu_util import require_gpu
from test_gpu_decode import FORMATS, rnd, run_case, weights

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def args(x, wr, k, bias=None, sigmoid=False):
    return dict(x=x.cuda(), w_router=wr.cuda(), k=k, bias=bias, residual=None,
                router=nvq.ROUTER_SIGMOID if sigmoid else nvq.ROUTER_SOFTMAX)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("small", [2.0 ** -27, 2.0 ** -28, 2.0 ** -30])
@pytest.mark.parametrize("T", [1, 9, 17])
def test_small_products_beside_a_large_one_decide(fmt, small, T):
    """Expert 0: 1. Expert 1: 1 and 31 small products. Expert 2: 1, -1 and small products that add up to less than expert
    3's. All are exact in 64 bits: 1, 3, 2 in the order of the choice after expert 4, whose logit is 2."""
    d = 96
    x, wr = torch.ones((T, d), dtype=BF16), torch.zeros((5, d), dtype=BF16)
    wr[0, 40] = 1.0
    wr[1, 32:64] = small
    wr[1, 63] = 1.0
    wr[2, 0], wr[2, 9], wr[2, 1:9] = 1.0, -1.0, small
    wr[3, 0], wr[3, 9], wr[3, 10:19] = 1.0, -1.0, small
    wr[4, 3] = 2.0
    w1, w2 = weights(3, 5, 64, d, fmt), weights(4, 5, d, 32, fmt)
    _, ids, wts = run_case(fmt, args(x, wr, 5), w1, w2)
    assert (ids.cpu() == torch.tensor([4, 1, 0, 3, 2], dtype=torch.int32)).all()
    p = torch.exp(torch.tensor([2.0, 1.0 + 31 * small, 1.0, 9 * small, 8 * small], dtype=torch.float64))
    assert (d64(wts) / (p / p.sum()) - 1).abs().max() <= 2.0 ** -24 + 2.0 ** -45


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,d,E,k", [(1, 4096, 384, 8), (5, 1000, 40, 6), (8, 512, 130, 4), (33, 264, 1000, 8), (64, 2080, 384, 8)])
def test_far_apart_products_choose_as_64_bits(T, d, E, k, sigmoid):
    """x and w over forty powers of two. A sum in 64 bits is off by at most d 2^-53 of the magnitudes, kernel and reference
    alike: keys further apart than that are in one order only, and the weights are a rounding to fp32 off (2^-24) and what
    the logits' error makes of them, twice its relative size."""
    g = torch.Generator().manual_seed(T)
    e = torch.randint(-20, 21, (d,), generator=g).double()
    x = (d64(rnd(1, T, d)) * 2.0 ** e).to(BF16)
    wr = (d64(rnd(2, E, d, std=d ** -0.5)) * 2.0 ** -(e + torch.randint(0, 13, (E, d), generator=g))).to(BF16)
    bias = rnd(5, E, dtype=F32, std=0.5)
    fmt = "bf16"
    w1, w2 = rnd(3, 1, 32, d).expand(E, 32, d).contiguous(), rnd(4, 1, d, 16).expand(E, d, 16).contiguous()
    _, ids, wts = run_case(fmt, args(x, wr, k, bias, sigmoid), w1, w2)
    lg = d64(x) @ d64(wr).T
    dl = 2 * d * 2.0 ** -53 * (d64(x).abs() @ d64(wr).abs().T) + 2.0 ** -50
    key = (torch.sigmoid(lg) if sigmoid else lg) + d64(bias)
    order = key.argsort(1, descending=True)
    top = key.gather(1, order[:, :k + 1])
    assert (top[:, :-1] - top[:, 1:] > 2 * dl.amax(1, keepdim=True)).all(), "inputs: a tie"
    assert torch.equal(ids.cpu().long(), order[:, :k])
    v = lg.gather(1, order[:, :k])
    w = torch.sigmoid(v) if sigmoid else torch.exp(v - v.amax(1, keepdim=True))
    w = w / w.sum(1, keepdim=True)
    assert ((d64(wts) - w).abs() <= w * (2.0 ** -24 + 4.2 * dl.amax(1, keepdim=True)) + 2.0 ** -149).all()
