"""Refusals of the operators around the FP8 linears, before any device is touched: the same
argument checks run with and without a GPU, and no kernel is launched here."""
import ctypes

import pytest
import torch

from fp8_dynamic_scaled_b200 import binding as b

L = b._lib
P = 0x10000          # a 16-byte aligned fake device address; never dereferenced on these paths
INV, ALIGN = b.FP8_ERR_INVALID_ARG, b.FP8_ERR_ALIGNMENT


def norm(x=P, rows=4, cols=64, ldx=64, res=None, ldr=0, s=None, lds=0, w=P, eps=1e-5, fmt=0, mode=1, amax=None, q=P,
         scale=P, y=None):
    return L.fp8_rmsnorm_quantize(x, rows, cols, ldx, res, ldr, s, lds, w, eps, fmt, mode, amax, q, scale, y, None, None)


@pytest.mark.parametrize("kw", [
    dict(mode=3), dict(mode=5), dict(mode=9), dict(fmt=2), dict(mode=4, fmt=1), dict(cols=24, ldx=24),
    dict(mode=4, cols=48, ldx=48), dict(cols=32784, ldx=32784), dict(rows=-1), dict(rows=1 << 31), dict(ldx=56),
    dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(q=None),
    dict(scale=None), dict(mode=0), dict(mode=1, amax=P), dict(s=P, lds=64), dict(res=P, ldr=56),
    dict(res=P, ldr=64, s=P, lds=56), dict(res=P, ldr=64, s=P, lds=72), dict(res=2 * P, ldr=64, s=P, lds=72)])
def test_rmsnorm_invalid(kw):
    assert norm(**kw) == INV


@pytest.mark.parametrize("kw", [
    dict(x=P + 2), dict(ldx=68), dict(q=P + 8), dict(scale=P + 2), dict(w=P + 2), dict(y=P + 4), dict(mode=0, amax=P + 2),
    dict(res=P + 8, ldr=64), dict(res=P, ldr=68), dict(res=P, ldr=64, s=2 * P + 8, lds=64),
    dict(res=P, ldr=64, s=2 * P, lds=68)])
def test_rmsnorm_alignment(kw):
    assert norm(**kw) == ALIGN


def gemm(act=0, res=None, ldres=0, y=P, ldy=16, yq=None, linear=False):
    base = b.fp8_epilogue_t(None, None, yq, P if yq else None, 0, 16)
    epi = ctypes.byref(b.fp8_epilogue_act_t(base, act, res, ldres))
    if linear:
        return L.fp8_linear_forward_act(P, 16, 32, 32, 0, 1, None, P, P, 1, 0, 16, y, ldy, epi, None, P, 1 << 20, None)
    return L.fp8_scaled_gemm_act(P, P, 1, 0, P, P, 1, 0, 16, 16, 32, y, ldy, epi, None, None, 0, None)


@pytest.mark.parametrize("linear", [False, True])
def test_gemm_act_refusals(linear):
    for act in (-1, 5, 100):
        assert gemm(act=act, linear=linear) == INV
    assert gemm(res=2 * P, ldres=15, linear=linear) == INV
    assert gemm(res=P, ldres=24, linear=linear) == INV                # y itself with another stride
    assert gemm(res=2 * P + 1, ldres=16, linear=linear) == ALIGN
    assert gemm(act=1, y=None, linear=linear) == INV                  # nowhere to write
    assert gemm(act=1, ldy=8, linear=linear) == INV
    assert L.fp8_linear_forward_act(P, 16, 32, 32, 0, 1, None, P, P, 1, 0, 16, P, 16, None, None, None, 0, None) \
        == b.FP8_ERR_WORKSPACE


def test_binding_type_checks():
    x = torch.empty((4, 64), dtype=torch.bfloat16)
    q, s = torch.empty((4, 64), dtype=torch.uint8), torch.empty(4)
    bad = [dict(x=x.float()), dict(weight=torch.empty(32, dtype=torch.bfloat16)), dict(q=q[:, :32]), dict(scale=s[:3]),
           dict(scale=s.double()), dict(residual=x[:2]), dict(sum_out=x.t()), dict(y=x[:, ::2])]
    for kw in bad:
        args = dict(x=x, weight=None, q=q, scale=s) | kw
        with pytest.raises(TypeError):
            b.fp8_rmsnorm_quantize(args["x"], args["weight"], 1e-5, 0, 1, args["q"], args["scale"],
                                   **{k: v for k, v in kw.items() if k in ("residual", "sum_out", "y")})
    a, w = torch.empty((4, 32), dtype=torch.uint8), torch.empty((8, 32), dtype=torch.uint8)
    y = torch.empty((4, 8), dtype=torch.bfloat16)
    for res in (y.float(), y[:3], torch.empty((8, 4), dtype=torch.bfloat16).t()):
        with pytest.raises(TypeError):
            b.fp8_scaled_gemm_act(a, s, 1, 0, w, s, 1, 0, y, residual=res)
