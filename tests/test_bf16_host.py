"""The BF16 expert layer's entry points without a GPU: what they refuse, on
the host, before any device work (addresses that are never dereferenced), and
the binding's own checks."""
import ctypes as C

import pytest
import torch

import precision_moe_numerics_amd as nvq
from bf16_ref import act_ref

OK, NULL, DIM, WORKSPACE, UNSUPPORTED, ALIGN = 0, -1, -2, -3, -5, -6
BIG = 1 << 40


def _p(i):
    return C.c_void_p(0x100000 + 0x1000 * i)


MIS = C.c_void_p(0x100008)


def gemm(mode=0, a=_p(0), a_rows=64, ag=None, ad=1, b=_p(1), b_rows=64, bg=None, bd=1, seg=_p(2), E=4, R=64, M=64, N=64,
         K=64, out=_p(3), sc=None, dt=0, acc=0, ws=_p(4), wsb=BIG):
    return nvq.lib().moe_grouped_gemm_bf16(mode, a, a_rows, ag, ad, b, b_rows, bg, bd, seg, E, R, M, N, K, out, sc, dt,
                                           acc, ws, wsb, None)


def test_grouped_refusals():
    for mode in (nvq.FWD, nvq.DGRAD, nvq.WGRAD):
        for null in ("a", "b", "seg", "out", "ws"):
            assert gemm(mode, **{null: None}) == NULL, null
        for mis in ("a", "b", "out", "ws"):
            assert gemm(mode, **{mis: MIS}) == ALIGN, mis
        for bad in (dict(N=4), dict(N=60), dict(N=0), dict(N=(1 << 22) + 8), dict(E=0), dict(E=4097), dict(R=-1),
                    dict(R=2 ** 31 - 200, a_rows=2 ** 31, b_rows=2 ** 31), dict(a_rows=63), dict(ag=_p(5), ad=0),
                    dict(ag=_p(5), a_rows=1 << 40)):
            assert gemm(mode, **bad) == DIM, bad
        assert gemm(mode, dt=2) == UNSUPPORTED
    for mode in (nvq.FWD, nvq.DGRAD):
        for bad in (dict(K=4), dict(K=63), dict(K=0), dict(N=1 << 17, K=1 << 17)):
            assert gemm(mode, **bad) == DIM, bad
        assert gemm(mode, acc=1) == UNSUPPORTED
        assert gemm(mode, bg=_p(5)) == UNSUPPORTED
        need = nvq.lib().moe_grouped_gemm_bf16_workspace_size(mode, 4, 64)
        assert gemm(mode, wsb=need - 1) == WORKSPACE
    assert gemm(nvq.WGRAD, M=12) == DIM
    assert gemm(nvq.WGRAD, b_rows=63) == DIM
    assert gemm(nvq.WGRAD, bg=_p(5), bd=0) == DIM
    assert gemm(nvq.WGRAD, sc=_p(5)) == UNSUPPORTED
    assert gemm(3) == UNSUPPORTED and gemm(-1) == UNSUPPORTED


def test_layer_refusals():
    L = nvq.lib()

    def fc1(x=_p(0), T=16, d=64, off=_p(1), s2a=_p(2), k=2, E=4, f=64, w=_p(3), h=_p(4), gu=None, ws=_p(5), wsb=BIG):
        return L.moe_fc1_swiglu_bf16(x, T, d, off, s2a, k, E, f, w, h, gu, ws, wsb, None)

    def fwd(x=_p(0), T=16, d=64, ids=_p(1), k=2, E=4, f=64, w1=_p(2), w2=_p(3), y=_p(4), bufs=None, ws=_p(5), wsb=BIG):
        return L.moe_expert_fwd_bf16(x, T, d, ids, k, E, f, w1, w2, y, bufs, ws, wsb, None)

    for fn, nulls, mis in ((fc1, ("x", "off", "s2a", "w", "h", "ws"), ("x", "w", "h", "gu", "ws")),
                           (fwd, ("x", "ids", "w1", "w2", "y", "ws"), ("x", "w1", "w2", "y", "ws"))):
        for n in nulls:
            assert fn(**{n: None}) == NULL, n
        for n in mis:
            assert fn(**{n: MIS}) == ALIGN, n
        for bad in (dict(T=-1), dict(d=60), dict(f=0), dict(f=12), dict(k=0), dict(k=5), dict(E=0), dict(E=5000),
                    dict(T=1 << 31), dict(T=1 << 22, d=4096), dict(d=1 << 16, f=1 << 16)):
            assert fn(**bad) == DIM, bad
        assert fn(wsb=16) == WORKSPACE
    assert fwd(bufs=C.byref(nvq.MoeBuffers(gemm_workgroups=3))) == UNSUPPORTED
    assert fwd(bufs=C.byref(nvq.MoeBuffers(xq_codes=0x1000))) == UNSUPPORTED
    assert fwd(bufs=C.byref(nvq.MoeBuffers(h=0x1008))) == ALIGN
    assert fwd(T=0, x=None, ids=None, y=None) == OK


def test_linear_refusals():
    L = nvq.lib()

    def lin(x=_p(0), w=_p(1), b=None, r=None, M=16, N=64, K=64, act=0, out=_p(2), dt=0, z=None):
        return L.linear_act_bf16(x, w, b, r, M, N, K, act, out, dt, z, None)

    def bwd(g=_p(0), gt=0, x=_p(1), w=_p(2), z=_p(3), M=16, N=64, K=64, act=4, dx=_p(4), dw=_p(5), wt=1, acc=0,
            db=_p(6), ws=_p(7), wsb=BIG):
        return L.linear_act_bwd_bf16(g, gt, x, w, z, M, N, K, act, dx, dw, wt, acc, db, ws, wsb, None)

    for fn, nulls, mis in ((lin, ("x", "w", "out"), ("x", "w", "b", "r", "out", "z")),
                           (bwd, ("g", "x", "w", "z", "ws"), ("g", "x", "w", "z", "dx", "dw", "db", "ws"))):
        for n in nulls:
            assert fn(**{n: None}) == NULL, n
        for n in mis:
            assert fn(**{n: MIS}) == ALIGN, n
        for bad in (dict(M=-1), dict(M=1 << 31), dict(M=1 << 30, N=1 << 11), dict(N=12), dict(N=0), dict(K=4), dict(K=1 << 23),
                    dict(N=1 << 20, K=1 << 20)):
            assert fn(**bad) == DIM, bad
        assert fn(act=6) == UNSUPPORTED and fn(act=-1) == UNSUPPORTED
    assert bwd(wsb=16) == WORKSPACE
    assert lin(dt=5) == UNSUPPORTED and bwd(gt=2) == UNSUPPORTED and bwd(wt=2) == UNSUPPORTED
    assert bwd(dx=None, dw=None, db=None) == NULL


def test_combine_and_router_refusals():
    L = nvq.lib()

    def com(y=_p(0), w=_p(1), ids=_p(2), E=4, r=None, T=8, k=2, Cc=64, out=_p(3)):
        return L.moe_combine_bf16(y, w, ids, E, r, T, k, Cc, out, None)

    def cbw(g=_p(0), y=_p(1), w=_p(2), ids=_p(3), E=4, T=8, k=2, Cc=64, dy=_p(4), dw=_p(5)):
        return L.moe_combine_bwd_bf16(g, y, w, ids, E, T, k, Cc, dy, dw, None)

    for fn, nulls, mis in ((com, ("y", "w", "out"), ("y", "r", "out")), (cbw, ("g", "y", "w", "dy", "dw"), ("g", "y", "dy"))):
        for n in nulls:
            assert fn(**{n: None}) == NULL, n
        for n in mis:
            assert fn(**{n: MIS}) == ALIGN, n
        for bad in (dict(T=-1), dict(k=0), dict(k=1025), dict(Cc=0), dict(Cc=12), dict(Cc=(1 << 20) + 8), dict(E=0),
                    dict(T=1 << 30, k=2), dict(k=1024, Cc=1 << 20)):
            assert fn(**bad) == DIM, bad
        assert fn(T=0) == OK
    for fn in (lambda T, E, k, w=_p(0), d=_p(3): L.moe_router_softmax_topk_bwd(w, _p(1), _p(2), T, E, k, d, None),
               lambda T, E, k, w=_p(0), d=_p(3): L.moe_router_sigmoid_topk_bwd(w, _p(4), _p(1), _p(2), T, E, k, d, None)):
        for bad in ((-1, 8, 2), (4, 0, 1), (4, 8, 9), (4, 8, 0), (4, 1025, 8), (4, 512, 65), (1 << 22, 1024, 8)):
            assert fn(*bad) == DIM, bad
        assert fn(4, 8, 2, w=None) == NULL and fn(4, 8, 2, d=None) == NULL
        assert fn(0, 8, 2) == OK


def test_launches_of_2_to_the_32_work_items_are_refused():
    """Sizes within every other limit; the sizes below them are not run here, only refused for a missing operand."""
    L = nvq.lib()
    assert L.linear_act_bf16(_p(0), _p(1), None, None, (1 << 31) - 512, 8, 8, 0, _p(2), 0, None, None) == DIM
    assert L.linear_act_bf16(None, _p(1), None, None, 1 << 30, 8, 8, 0, _p(2), 0, None, None) == NULL
    assert gemm(mode=nvq.WGRAD, a=None, R=64, M=1 << 22, N=1 << 22, E=1) == DIM
    assert gemm(mode=nvq.FWD, a=None, R=1 << 30, N=1 << 10, E=1, a_rows=1 << 30) == DIM
    for T, C in ((1 << 24, 1 << 11), (1 << 16, 1 << 19)):
        assert L.moe_combine_bf16(_p(0), _p(1), None, 0, None, T, 1, C, _p(2), None) == DIM
        assert L.moe_combine_bf16(None, _p(1), None, 0, None, T // 2, 1, C, _p(2), None) == NULL
    for T, C in ((1 << 26, 64), (1 << 24, 2048)):
        assert L.moe_combine_bwd_bf16(_p(0), _p(1), _p(2), None, 0, T, 1, C, _p(3), _p(4), None) == DIM
    assert L.moe_router_softmax_topk_bwd(_p(0), _p(1), _p(2), 1 << 26, 8, 2, _p(3), None) == DIM
    assert L.linear_act_bwd_bf16(_p(0), 0, _p(1), _p(2), _p(3), 1 << 30, 8, 8, 4, _p(4), None, 1, 0, None, _p(7), BIG,
                                 None) == DIM


def test_the_binding_refuses_host_tensors_and_wrong_arguments():
    x, w = torch.zeros((8, 64), dtype=torch.bfloat16), torch.zeros((64, 64), dtype=torch.bfloat16)
    seg = torch.zeros(2, dtype=torch.int32)
    calls = [lambda: nvq.linear_act_bf16(x, w), lambda: nvq.linear_act_bwd_bf16(x, x, w),
             lambda: nvq.moe_grouped_gemm_bf16(nvq.FWD, x, w[None], seg),
             lambda: nvq.moe_fc1_swiglu_bf16(x, seg, seg, 1, w[None]),
             lambda: nvq.moe_expert_fwd_bf16(x, seg[None], w[None], w[None]),
             lambda: nvq.moe_combine_bf16(x[None], torch.zeros((1, 8))),
             lambda: nvq.moe_combine_bwd_bf16(x, x[None], torch.zeros((1, 8))),
             lambda: nvq.moe_router_softmax_topk_bwd(torch.zeros((1, 8)), seg[None], torch.zeros((1, 8)), 8),
             lambda: nvq.moe_router_sigmoid_topk_bwd(torch.zeros((1, 8)), torch.zeros((1, 8)), seg[None], torch.zeros((1, 8)))]
    for call in calls:
        with pytest.raises(nvq.NvqError):
            call()


@pytest.mark.parametrize("act", range(6))
def test_reference_gradients_against_differences(act):
    """The oracle of the GPU tests itself: its factors of dout against differences of its values."""
    n, h = 32, 2.0 ** -18
    z = torch.randn((50, 2 * n if act == 5 else n), dtype=torch.float64, generator=torch.Generator().manual_seed(act))
    for part, f in enumerate(act_ref(z, act, n)[1]):
        v = torch.zeros_like(z)
        v[:, part * n:(part + 1) * n] = 1.0
        num = (act_ref(z + h * v, act, n)[0] - act_ref(z - h * v, act, n)[0]) / (2 * h)
        kink = (z.abs() <= h) if act == 1 else torch.zeros_like(num, dtype=torch.bool)
        # h^2 / 6 |act'''| with |act'''| <= 3 (1 + |u|), and 2^-52 / h of the values
        assert (((f - num).abs() <= 2.0 ** -30 * (1 + z.abs().amax())) | kink).all()


def test_dense_backward_of_no_rows():
    """With no rows dx has no storage and so no address: not a missing output."""
    L = nvq.lib()

    def bwd(M, dx=None, w=_p(0), ws=_p(1)):
        return L.linear_act_bwd_bf16(None, 0, None, w, None, M, 64, 64, 4, dx, None, 1, 0, None, ws, BIG, None)

    assert bwd(0) == OK and bwd(0, dx=_p(2)) == OK
    assert bwd(16) == NULL and bwd(0, ws=None) == NULL and bwd(0, dx=_p(2), w=None) == NULL


def test_a_residual_in_place_has_the_outputs_type():
    """residual == out is for bf16 outputs: an fp32 out over a bf16 residual would overwrite rows not yet read."""
    L = nvq.lib()
    assert L.linear_act_bf16(_p(0), _p(1), None, _p(2), 16, 64, 64, 0, _p(2), 1, None, None) == UNSUPPORTED
    assert L.linear_act_bf16(None, _p(1), None, _p(2), 16, 64, 64, 0, _p(2), 0, None, None) == NULL


def test_fc1_is_not_refused_for_the_size_of_fc2():
    """2^24 tiles of 128 x 128 in fc2's output, 2^17 in fc1's: within fc1's limits (refused here for a missing operand)."""
    L = nvq.lib()
    T, d, k, E, f = (1 << 17) - 1, 1 << 14, 128, 128, 64
    assert L.moe_fc1_swiglu_bf16(None, T, d, _p(1), _p(2), k, E, f, _p(3), _p(4), None, _p(5), BIG, None) == NULL
    assert L.moe_expert_fwd_bf16(None, T, d, _p(1), k, E, f, _p(2), _p(3), _p(4), None, _p(5), BIG, None) == DIM
    assert L.moe_fc1_swiglu_bf16(None, T + 1, d, _p(1), _p(2), k, E, f, _p(3), _p(4), None, _p(5), BIG, None) == DIM
