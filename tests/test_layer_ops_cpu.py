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


def kv_cache(**kw):
    d = dict(k_dev=P, v_dev=P, k_scale_dev=P, v_scale_dev=P, num_pages=4, page_size=16, kv_heads=2, head_dim=64, fmt=0,
             page_table_dev=P, table_stride=4, max_pages=4, kv_lens_dev=P, batch=2) | kw
    return b.fp8_kv_cache_t(**d)


def append(k=P, ldk=128, v=P, ldv=128, tokens=2, cu=None, max_q=1, **kw):
    return L.fp8_kv_append(ctypes.byref(kv_cache(**kw)), k, ldk, v, ldv, tokens, cu, max_q, None, None)


def attend(q=P, ldq=256, heads=4, tokens=2, cu=None, max_q=1, max_kv=64, scale=0.1, out=P, ldo=256, ws=P, ws_bytes=1 << 30,
           **kw):
    return L.fp8_kv_attention(ctypes.byref(kv_cache(**kw)), q, ldq, heads, tokens, cu, max_q, max_kv, scale, out, ldo, None,
                              ws, ws_bytes, None)


BAD_CACHE = [dict(fmt=2), dict(page_size=48), dict(page_size=0), dict(page_size=256), dict(head_dim=96),
             dict(head_dim=256), dict(kv_heads=0), dict(batch=-1), dict(num_pages=-1), dict(max_pages=5), dict(max_pages=-1),
             dict(k_dev=None), dict(v_scale_dev=None), dict(kv_lens_dev=None), dict(page_table_dev=None), dict(tokens=-1),
             dict(max_q=-1), dict(tokens=3), dict(max_q=2)]


@pytest.mark.parametrize("kw", BAD_CACHE)
def test_kv_cache_refusals(kw):
    assert append(**kw) == INV
    assert attend(**kw) == INV


def test_kv_append_refusals():
    assert L.fp8_kv_append(None, P, 128, P, 128, 2, None, 1, None, None) == INV
    for kw in (dict(ldk=120), dict(ldv=64), dict(k=None), dict(v=None)):
        assert append(**kw) == INV
    for kw in (dict(ldk=132), dict(k=P + 2), dict(v=P + 8), dict(k_dev=P + 8), dict(v_scale_dev=P + 2),
               dict(kv_lens_dev=P + 1), dict(cu=P + 2, max_q=5)):
        assert append(**kw) == ALIGN


def test_kv_attention_refusals():
    for kw in (dict(heads=3), dict(heads=0), dict(ldq=248), dict(ldo=248), dict(q=None), dict(out=None), dict(max_kv=-1),
               dict(max_kv=1 << 30), dict(scale=float("nan")), dict(scale=float("inf")), dict(max_q=1 << 24, cu=P)):
        assert attend(**kw) == INV
    for kw in (dict(q=P + 2), dict(ldq=260), dict(out=P + 8), dict(ldo=260), dict(ws=P + 4, max_kv=100000)):
        assert attend(**kw) == ALIGN
    n = b.fp8_kv_attention_workspace_size(2, 4, 2, 64, 1, 100000)
    assert n > 0
    assert attend(max_kv=100000, ws=None) == b.FP8_ERR_WORKSPACE
    assert attend(max_kv=100000, ws_bytes=n - 1) == b.FP8_ERR_WORKSPACE
    for bad in ((0, 4, 2, 64, 1, 10), (1, 4, 3, 64, 1, 10), (1, 4, 2, 96, 1, 10), (1, 4, 2, 64, 0, 10), (1, 4, 2, 64, 1, -1)):
        assert b.fp8_kv_attention_workspace_size(*bad) == 0


def test_kv_binding_type_checks():
    cache = b.KVCache.empty(4, 2, 16, 64, device="cpu")
    table, lens = torch.zeros((2, 3), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    x = torch.empty((2, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        b.KVCache(cache.k[:, :, :, :32], cache.v, cache.k_scale, cache.v_scale)
    with pytest.raises(TypeError):
        b.KVCache(cache.k, cache.v, cache.k_scale.double(), cache.v_scale)
    for k, v, t, n in ((x.float(), x, table, lens), (x[:1], x, table, lens), (x, x.transpose(0, 1), table.long(), lens),
                       (x, x, table, lens[:1]), (x[:, :1], x, table, lens), (x.transpose(0, 1).contiguous().transpose(0, 1), x,
                                                                              table, lens)):
        with pytest.raises(TypeError):
            b.fp8_kv_append(k, v, cache, t, n)
    with pytest.raises(TypeError):
        b.fp8_kv_append(x, x, cache, table, lens, cu_q=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        b.fp8_kv_attention(x, cache, table, lens, x[:1], max_kv_len=16)


def test_tensors_off_the_current_device_are_refused():
    """Well-formed calls with host tensors: refused in the binding, before the library sees a pointer."""
    cache = b.KVCache.empty(4, 2, 16, 64, device="cpu")
    table, lens = torch.zeros((2, 3), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    kv = torch.empty((2, 2, 64), dtype=torch.bfloat16)
    x, q, s = torch.empty((4, 64), dtype=torch.bfloat16), torch.empty((4, 64), dtype=torch.uint8), torch.empty(4)
    w, y = torch.empty((8, 64), dtype=torch.uint8), torch.empty((4, 8), dtype=torch.bfloat16)
    for call in (lambda: b.fp8_kv_append(kv, kv, cache, table, lens),
                 lambda: b.fp8_kv_attention(kv, cache, table, lens, kv.clone(), max_kv_len=16),
                 lambda: b.fp8_rmsnorm_quantize(x, None, 1e-5, 0, 1, q, s),
                 lambda: b.fp8_scaled_gemm_act(q, s, 1, 0, w, s, 1, 0, y),
                 lambda: b.fp8_linear_forward_act(x, 0, 1, w, s, 1, 0, y, q)):
        with pytest.raises(ValueError):
            call()
