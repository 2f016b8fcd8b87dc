"""Refusals of the operators around the quantizer, on the host: every check
runs before a device is touched (made-up addresses stand in for buffers)."""
import ctypes

import pytest
import torch

import nvfp4_adaptive_block_amd as fos

P = ctypes.c_void_p
INVALID, DTYPE, SHAPE, ALIGN = 1, 2, 3, 4
X, C, S, D, Y, O, B = (0x10000 * i for i in range(1, 8))


def operand(data=X, block_scales=S, scale=D, type=4, gran=0):
    return fos._Operand(data, block_scales, scale, type, gran)


def linear(x=None, w=None, M=4, N=8, K=32, epi=None, y=Y, out=0, work=None, room=0, offs=None, G=None):
    lib = fos.load_library()
    x, w = x or operand(type=0), w or operand(C)
    e = None if epi is None else ctypes.byref(epi)
    if G is None:
        rc = lib.fos_linear(ctypes.byref(x), ctypes.byref(w), M, N, K, e, P(y), out, work, room, None)
    else:
        rc = lib.fos_linear_grouped(ctypes.byref(x), ctypes.byref(w), offs, G, M, N, K, e, P(y), out, work, room,
                                    None, None)
    assert rc == 0 or lib.fos_last_error()
    return rc


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(K=40)), (INVALID, dict(M=-1)), (INVALID, dict(N=-3)), (SHAPE, dict(M=2 ** 31)),
    (SHAPE, dict(M=2 ** 30, K=2 ** 20)), (SHAPE, dict(M=2 ** 25, N=2 ** 25)), (DTYPE, dict(out=3)),
    (INVALID, dict(y=0)), (ALIGN, dict(y=Y + 8)),
    (DTYPE, dict(x=operand(type=2))), (DTYPE, dict(x=operand(type=9))), (INVALID, dict(x=operand(0, type=0))),
    (ALIGN, dict(x=operand(X + 2, type=0))), (ALIGN, dict(x=operand(X + 8, type=3))),
    (ALIGN, dict(x=operand(X + 4, type=4))), (INVALID, dict(x=operand(type=3, scale=0))),
    (ALIGN, dict(x=operand(type=3, scale=D + 2))), (INVALID, dict(x=operand(type=4, block_scales=0))),
    (INVALID, dict(x=operand(type=3, gran=2))), (INVALID, dict(x=operand(type=3, gran=5))),
    (DTYPE, dict(w=operand(C, type=0))), (DTYPE, dict(w=operand(C, type=3))), (INVALID, dict(w=operand(0))),
    (INVALID, dict(w=operand(C, scale=0))), (INVALID, dict(w=operand(C, gran=2))),
    (INVALID, dict(epi=fos._Epilogue(0, 0, 0, 5))), (INVALID, dict(epi=fos._Epilogue(0, 0, 0, -1))),
    (DTYPE, dict(epi=fos._Epilogue(B, 0, 3, 0))), (ALIGN, dict(epi=fos._Epilogue(B + 4, 0, 0, 0))),
    (ALIGN, dict(epi=fos._Epilogue(0, B + 2, 0, 0))),
    (INVALID, dict(G=0, offs=P(O))), (INVALID, dict(G=2, offs=None)), (ALIGN, dict(G=2, offs=P(O + 2))),
    (SHAPE, dict(G=1 << 20, offs=P(O), N=2 ** 20, K=2 ** 10)),
])
def test_linear_refusals(want, kw):
    assert linear(**kw) == want


def test_linear_needs_its_operands():
    lib = fos.load_library()
    w = operand()
    assert lib.fos_linear(None, ctypes.byref(w), 1, 1, 16, None, P(Y), 0, None, 0, None) == INVALID
    assert lib.fos_linear(ctypes.byref(w), None, 1, 1, 16, None, P(Y), 0, None, 0, None) == INVALID


def test_linear_workspace():
    lib = fos.load_library()
    assert lib.fos_linear_workspace(4, 4, 40, 0) == -1
    assert lib.fos_linear_workspace(4, 4, 64, -1) == -1
    with pytest.raises(ValueError):
        fos.fos_linear_workspace(-1, 4, 64)
    for M in (1, 16, 64, 200, 5000):
        for N in (16, 100, 4096):
            for K in (16, 4096, 14336):
                need = fos.fos_linear_workspace(M, N, K)
                assert need >= 0
                if need:  # too small, missing or misaligned
                    kw = dict(M=M, N=N, K=K)
                    assert linear(work=P(X), room=need - 1, **kw) == INVALID
                    assert linear(work=None, room=need, **kw) == INVALID
                    assert linear(work=P(X + 8), room=need, **kw) == ALIGN


def norm(x=X, dtype=0, M=4, K=64, res=None, w=C, wdt=2, eps=1e-6, q=Y, s=S, h=None, y=None):
    return fos.load_library().fos_rmsnorm_quantize(P(x), dtype, M, K, res, P(w), wdt, eps, P(q), P(s), h, y, None)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dtype=3)), (DTYPE, dict(wdt=-1)), (INVALID, dict(M=-1)), (INVALID, dict(K=-1)), (SHAPE, dict(K=0)),
    (SHAPE, dict(M=2 ** 31)), (SHAPE, dict(K=2 ** 31)), (SHAPE, dict(M=2 ** 30, K=2 ** 20)),
    (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(eps=float("inf"))),
    (INVALID, dict(w=0)), (INVALID, dict(x=0)), (INVALID, dict(q=0)), (INVALID, dict(s=0)),
    (ALIGN, dict(x=X + 2)), (ALIGN, dict(res=P(B + 8))), (ALIGN, dict(w=C + 4)), (ALIGN, dict(q=Y + 1)),
    (ALIGN, dict(s=S + 2)), (ALIGN, dict(h=P(O + 8))), (ALIGN, dict(y=P(O + 4))),
])
def test_norm_refusals(want, kw):
    assert norm(**kw) == want


def balance(logits=X, dtype=2, T=8, E=16, idx=C, ib=8, k=2, mask=None, align=16, loss=Y, counts=O, offs=None,
            slope=S, work=B, room=1 << 30):
    return fos.load_library().fos_balance_loss(P(logits), dtype, T, E, P(idx), ib, k, mask, 0.01, align, P(loss),
                                               P(counts), offs, P(slope), P(work), room, None, None)


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dtype=3)), (SHAPE, dict(T=-1)), (SHAPE, dict(T=2 ** 31)), (SHAPE, dict(E=0)), (SHAPE, dict(E=1025)),
    (DTYPE, dict(ib=2)), (INVALID, dict(k=0)), (INVALID, dict(align=0)), (SHAPE, dict(T=2 ** 30, k=2)),
    (SHAPE, dict(E=1024, align=2 ** 22)), (INVALID, dict(logits=0)), (INVALID, dict(idx=0)), (INVALID, dict(loss=0)),
    (INVALID, dict(counts=0)), (INVALID, dict(slope=0)), (INVALID, dict(work=0)), (INVALID, dict(room=16)),
    (ALIGN, dict(logits=X + 4)), (ALIGN, dict(idx=C + 4)), (ALIGN, dict(work=B + 4)), (ALIGN, dict(loss=Y + 2)),
    (ALIGN, dict(offs=P(O + 1))),
])
def test_balance_refusals(want, kw):
    assert balance(**kw) == want


@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dtype=5)), (SHAPE, dict(T=-2)), (SHAPE, dict(E=2000)), (INVALID, dict(d=0)), (INVALID, dict(x=0)),
    (INVALID, dict(slope=0)), (INVALID, dict(out=0)), (ALIGN, dict(x=X + 8)), (ALIGN, dict(out=Y + 8)),
    (ALIGN, dict(d=D + 2)),
])
def test_balance_backward_refusals(want, kw):
    a = dict(d=D, x=X, dtype=2, T=8, E=16, slope=S, out=Y) | kw
    rc = fos.load_library().fos_balance_loss_backward(P(a["d"]), P(a["x"]), a["dtype"], a["T"], a["E"], None,
                                                      P(a["slope"]), P(a["out"]), None)
    assert rc == want


def test_balance_workspace():
    assert fos.load_library().fos_balance_workspace(8, 0) == -1
    with pytest.raises(ValueError):
        fos.fos_balance_workspace(-1, 8)
    assert fos.fos_balance_workspace(0, 1) > 0


def test_python_refuses_host_tensors():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    w = (torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8), torch.ones(1))
    with pytest.raises(ValueError, match="device tensor"):
        fos.fos_linear(x, w)
    with pytest.raises(ValueError, match="device tensor"):
        fos.fos_linear_grouped(x, w, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        fos.fos_rmsnorm_quantize(x, torch.ones(32))
    with pytest.raises(ValueError, match="device tensor"):
        fos.fos_balance_loss(x, torch.zeros(4, 2, dtype=torch.int64))
    with pytest.raises(ValueError, match="device tensor"):
        fos.fos_balance_loss_backward(torch.ones(1), x, torch.ones(32))
