"""The BF16 expert layer where its values and sizes are extreme: infinities, NaN
and tails of the activations, empty batches and segments, offsets that
contradict each other."""
import pytest
import torch

import precision_moe_numerics_amd as nvq
from bf16_ref import GELU, GELU_TANH, NONE, RELU, SILU, SWIGLU, act_ref, d64
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
