"""The int8 products' entry points without a GPU: what they refuse before any device work (addresses that are never
dereferenced), the binding's own checks, and the tests' own reference quantizer."""
import ctypes as C
from fractions import Fraction

import pytest
import torch

import precision_moe_numerics_amd as nvq
from int8_ref import quantize

OK, NULL, DIM, WORKSPACE, UNSUPPORTED, ALIGN = 0, -1, -2, -3, -5, -6
BIG = 1 << 40


def _p(i):
    return C.c_void_p(0x100000 + 0x1000 * i)


MIS = C.c_void_p(0x100008)


def test_quantize_refusals():
    L = nvq.lib()

    def quant(x=_p(0), R=4, Cc=64, c=_p(1), s=_p(2)):
        return L.int8_quantize(x, R, Cc, c, s, None)

    def deq(c=_p(0), s=_p(1), R=4, Cc=64, o=_p(2), dt=0):
        return L.int8_dequantize(c, s, R, Cc, o, dt, None)

    for fn, names in ((quant, "xcs"), (deq, "cso")):
        for n in names:
            assert fn(**{n: None}) == NULL and fn(**{n: MIS}) == ALIGN, n
        for bad in (dict(R=-1), dict(R=1 << 24), dict(Cc=0), dict(Cc=8), dict(Cc=24), dict(Cc=(1 << 22) + 16)):
            assert fn(**bad) == DIM, bad
        assert fn(R=0) == OK
    assert deq(dt=2) == UNSUPPORTED and deq(dt=-1) == UNSUPPORTED
    assert deq(R=1 << 16, Cc=1 << 20) == DIM


def test_linear_refusals():
    def lin(x=_p(0), xs=_p(1), w=_p(2), ws=_p(3), b=None, r=None, M=16, N=64, K=64, act=0, out=_p(4), dt=0):
        return nvq.lib().linear_act_int8(x, xs, w, ws, b, r, M, N, K, act, out, dt, None)

    for n in ("x", "xs", "w", "ws", "out"):
        assert lin(**{n: None}) == NULL, n
    for n in ("x", "xs", "w", "ws", "b", "r", "out"):
        assert lin(**{n: MIS}) == ALIGN, n
    for bad in (dict(M=-1), dict(M=1 << 31), dict(M=1 << 30, N=1 << 11), dict(N=12), dict(N=0), dict(N=(1 << 22) + 8),
                dict(K=8), dict(K=0), dict(K=24), dict(K=1 << 17), dict(N=1 << 16, K=65536), dict(M=(1 << 31) - 512, N=8, K=16)):
        assert lin(**bad) == DIM, bad
    assert lin(act=6) == UNSUPPORTED and lin(act=-1) == UNSUPPORTED and lin(dt=2) == UNSUPPORTED
    assert lin(r=_p(4), dt=1) == UNSUPPORTED
    # the largest K and weights just below 4 GiB are within the limits (refused here for a missing operand)
    assert lin(x=None, K=(1 << 17) - 16) == NULL
    assert lin(x=None, N=32760, K=131056) == NULL and lin(x=None, N=32760, K=131056, act=5) == DIM


def test_layer_refusals():
    L = nvq.lib()

    def fc1(x=_p(0), xs=_p(1), T=16, d=64, off=_p(2), s2a=_p(3), k=2, E=4, f=64, w=_p(4), wsc=_p(5), h=_p(6), ws=_p(7),
            wsb=BIG):
        return L.moe_fc1_swiglu_int8(x, xs, T, d, off, s2a, k, E, f, w, wsc, h, ws, wsb, None)

    def fc2(h=_p(0), hs=_p(1), A=32, f=64, off=_p(2), s2a=_p(3), E=4, d=64, w=_p(4), wsc=_p(5), y=_p(6), ws=_p(7), wsb=BIG):
        return L.moe_fc2_int8(h, hs, A, f, off, s2a, E, d, w, wsc, y, ws, wsb, None)

    def fwd(x=_p(0), T=16, d=64, ids=_p(1), k=2, E=4, f=64, w1=_p(2), w1s=_p(3), w2=_p(4), w2s=_p(5), y=_p(6), bufs=None,
            ws=_p(7), wsb=BIG):
        return L.moe_expert_fwd_int8(x, T, d, ids, k, E, f, w1, w1s, w2, w2s, y, bufs, ws, wsb, None)

    for fn, nulls, mis in ((fc1, ("x", "xs", "off", "s2a", "w", "wsc", "h", "ws"), ("x", "xs", "w", "wsc", "h", "ws")),
                           (fc2, ("h", "hs", "off", "s2a", "w", "wsc", "y", "ws"), ("h", "hs", "w", "wsc", "y", "ws")),
                           (fwd, ("x", "ids", "w1", "w1s", "w2", "w2s", "y", "ws"),
                            ("x", "w1", "w1s", "w2", "w2s", "y", "ws"))):
        for n in nulls:
            assert fn(**{n: None}) == NULL, n
        for n in mis:
            assert fn(**{n: MIS}) == ALIGN, n
        for bad in (dict(d=68), dict(d=0), dict(f=20), dict(f=0), dict(E=0), dict(E=4097)):
            assert fn(**bad) == DIM, bad
        assert fn is fc1 or fn(f=24) == DIM and fn(f=1 << 17) == DIM  # fc2 contracts over d_ff
        assert fn is fc2 or fn(d=72) == DIM                                # fc1 over d
        assert fn(wsb=16) == WORKSPACE
    for fn in (fc1, fwd):
        for bad in (dict(T=-1), dict(k=0), dict(k=5), dict(T=1 << 31), dict(T=1 << 23, d=4096), dict(d=1 << 17)):
            assert fn(**bad) == DIM, bad
    assert fc2(A=-1) == DIM and fc2(A=1 << 31) == DIM
    assert fwd(T=0, x=None, ids=None, y=None) == OK
    for field in ("xq_scales", "hq_scales", "gu"):
        assert fwd(bufs=C.byref(nvq.MoeBuffers(**{field: 0x1000}))) == UNSUPPORTED
    assert fwd(bufs=C.byref(nvq.MoeBuffers(gemm_workgroups=3))) == UNSUPPORTED
    for field in ("xq_codes", "xq_tscale", "h", "hq_codes", "hq_tscale"):
        assert fwd(bufs=C.byref(nvq.MoeBuffers(**{field: 0x1008}))) == ALIGN, field


def test_the_binding_refuses_host_tensors_and_wrong_arguments():
    x, q, s = torch.zeros((16, 64), dtype=torch.bfloat16), torch.zeros((16, 64), dtype=torch.int8), torch.zeros(16)
    off = torch.zeros(2, dtype=torch.int32)
    calls = [lambda: nvq.int8_quantize(x), lambda: nvq.int8_dequantize(q, s), lambda: nvq.linear_act_int8((q, s), (q, s)),
             lambda: nvq.linear_act_int8(q, (q, s)), lambda: nvq.linear_act_int8((q, s), None),
             lambda: nvq.moe_fc1_swiglu_int8((q, s), off, off, 1, (q[None], s[None])),
             lambda: nvq.moe_fc2_int8((q, s), off, off, (q[None], s[None])),
             lambda: nvq.moe_expert_fwd_int8(x, off[None], (q[None], s[None]), (q[None], s[None]))]
    for call in calls:
        with pytest.raises(nvq.NvqError):
            call()


def test_reference_quantizer_against_fractions():
    """Every decision of the tests' quantizer against exact rational arithmetic, on rows whose values are random, ties
    (127 x / amax = n + 1/2 exactly) and their bf16 neighbours."""
    g = torch.Generator().manual_seed(0)
    rows = [torch.randn(64, generator=g), torch.randn(64, generator=g) * 2.0 ** -128, torch.arange(-127, 128) / 2.0]
    for a in (127.0, 254.0, 63.5, 1.9921875 * 2 ** 20):
        x = torch.arange(-127, 127).float().add(0.5).mul(a / 127.0)
        rows.append(torch.cat([x, torch.tensor([a])]))
    for row in rows:
        x = row.to(torch.bfloat16)
        codes, scale = quantize(x)
        vals = [Fraction(v) for v in x.double().tolist()]
        top = max(abs(v) for v in vals)
        for v, c in zip(vals, codes.tolist()):
            assert round(v * 127 / top) == c      # (Fraction rounds halves to even)
        assert scale.item() == (torch.tensor(float(top), dtype=torch.float32) / 127.0).item()
