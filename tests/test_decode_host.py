"""The few-token layer's entry points without a GPU: what they refuse before any device work (addresses that are never
dereferenced), and the binding's own checks."""
import ctypes as C

import pytest
import torch

import precision_moe_numerics_amd as nvq

OK, NULL, DIM, WORKSPACE, UNSUPPORTED, ALIGN = 0, -1, -2, -3, -5, -6
BIG = 1 << 40


def _p(i):
    return C.c_void_p(0x100000 + 0x1000 * i)


MIS = C.c_void_p(0x100008)
FORMATS = {"bf16": ("w1", "w2"), "int8": ("w1", "s1", "w2", "s2"), "nvfp4": ("w1", "s1", "t1", "w2", "s2", "t2")}


def call(fmt, x=_p(0), T=4, d=64, wr=_p(1), bias=_p(2), router=0, k=2, E=8, f=64, res=None, out=_p(3), ids=_p(4),
         wts=_p(5), ws=_p(6), wsb=BIG, **w):
    wp = [w.get(n, _p(10 + i)) for i, n in enumerate(FORMATS[fmt])]
    return getattr(nvq.lib(), "moe_layer_decode_" + fmt)(x, T, d, wr, bias, router, k, E, f, *wp, res, out, ids, wts, ws, wsb,
                                                         None)


@pytest.mark.parametrize("fmt", FORMATS)
def test_refusals(fmt):
    for n in ("x", "wr", "out", "ids", "wts", "ws") + FORMATS[fmt]:
        assert call(fmt, **{n: None}) == NULL, n
    for n in ("x", "wr", "bias", "res", "out", "ids", "wts", "ws") + FORMATS[fmt]:
        assert call(fmt, **{n: MIS}) == ALIGN, n
    m = {"bf16": 8, "int8": 16, "nvfp4": 32}[fmt]
    for bad in (dict(T=-1), dict(T=65), dict(d=0), dict(d=m // 2), dict(d=64 + m // 2), dict(f=0), dict(f=64 + m // 2),
                dict(d=(1 << 22) + 32), dict(f=(1 << 22) + 32), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(k=65, E=128),
                dict(d=1 << 17, f=1 << 17), dict(d=1 << 21, E=1024), dict(T=64, k=64, E=64, f=1 << 20)):
        assert call(fmt, **bad) == DIM, bad
    assert call(fmt, router=2) == UNSUPPORTED and call(fmt, router=-1) == UNSUPPORTED
    need = nvq.lib().moe_layer_decode_workspace_size(4, 64, 2, 8, 64)
    assert call(fmt, wsb=need - 1) == WORKSPACE
    assert call(fmt, T=0, x=None, out=None, ids=None, wts=None) == OK


def test_workspace_sizes():
    size = nvq.lib().moe_layer_decode_workspace_size
    assert 0 < size(1, 64, 2, 8, 64) <= size(64, 64, 2, 8, 64)
    for bad in ((-1, 64, 2, 8, 64), (65, 64, 2, 8, 64), (1, 64, 0, 8, 64), (1, 64, 65, 80, 64), (1, 64, 2, 0, 64),
                (1, 64, 2, 1025, 64), (1, 64, 2, 8, -1)):
        assert size(*bad) == 0


def test_the_binding_refuses_host_tensors_and_wrong_arguments():
    bf = torch.bfloat16
    x, wr, w1, w2 = (torch.zeros(s, dtype=bf) for s in ((2, 64), (4, 64), (4, 128, 64), (4, 64, 64)))
    q1, q2 = (torch.zeros((4, 128, 64), dtype=torch.int8), torch.zeros((4, 128))), (torch.zeros((4, 64, 64), dtype=torch.int8),
                                                                                   torch.zeros((4, 64)))
    for fn in (lambda: nvq.moe_layer_decode_bf16(x, wr, 2, w1, w2), lambda: nvq.moe_layer_decode_int8(x, wr, 2, q1, q2),
               lambda: nvq.moe_layer_decode_int8(x, wr, 2, w1, w2), lambda: nvq.moe_layer_decode_nvfp4(x, wr, 2, q1, q2),
               lambda: nvq.moe_layer_decode_bf16(x[0], wr, 2, w1, w2), lambda: nvq.moe_layer_decode_bf16(x, wr, 2, q1, q2)):
        with pytest.raises(nvq.NvqError):
            fn()
