"""The activations far outside the range of ordinary values: through the bias, over accumulators that are 0.

Tolerance: the last rounding, 2^-8; the activation itself, 2^-14 (see test_gpu_gemm_act); and the
magnitudes below the normal range, 2^-126."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import fp8_dynamic_scaled_b200.binding as fp8  # noqa: E402
from test_gpu_gemm_act import GELU, MX, NONE, PAIRS, RELU, SILU, TANH, act64  # noqa: E402

INF, BIG = math.inf, float(torch.finfo(torch.bfloat16).max)
VALUES = [INF, BIG, 1e30, 2e19, 1e10, 1e3, 17.0, 16.0, 15.9375, 0.0, -8.0, -12.5, -15.9375, -16.0, -17.0, -1e3, -1e10,
          -2e19, -1e30, -BIG]


def call(M, N, am, bm, bias, act, **kw):
    K = 128
    a, b = (torch.zeros((n, K), dtype=torch.uint8, device="cuda") for n in (M, N))
    sa, sb = (torch.full(fp8.scale_shape(m, n, K), 127 if m == MX else 1.0, device="cuda",
                         dtype=torch.uint8 if m == MX else torch.float32) for n, m in ((M, am), (N, bm)))
    y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    fp8.fp8_scaled_gemm_act(a, sa, am, 0, b, sb, bm, 0, y, bias=bias, activation=act, **kw)
    return y


@pytest.mark.parametrize("am,bm", PAIRS)
@pytest.mark.parametrize("M", [3, 100, 300])        # the decode, the tiled, the CTA-pair kernel
@pytest.mark.parametrize("act", [NONE, RELU, GELU, TANH, SILU])
def test_largest_values_and_infinity(M, act, am, bm):
    bias = torch.tensor(VALUES * 3, dtype=torch.bfloat16, device="cuda")
    N = bias.numel()
    amax, yq = torch.zeros(1, device="cuda"), torch.zeros((M, N), dtype=torch.uint8, device="cuda")
    y = call(M, N, am, bm, bias, act, amax=amax, yq=yq, yq_scale=torch.ones(1, device="cuda"))
    ref = act64(bias.double(), act)
    if act == TANH:                                 # v^3 of the largest leaves no trace in v (1 or 0 of it)
        ref = torch.where(bias.abs() > 1e4, bias.double().clamp(min=0), ref)
    ref = ref[None, :].expand(M, N)
    assert bool(((y == INF) == (ref == INF)).all())
    d = (y.double() - ref).abs()
    assert bool(((d <= (2.0 ** -8 + 2.0 ** -14) * ref.abs() + 2.0 ** -126) | (ref == INF)).all())
    assert amax.item() == INF
    assert torch.equal(yq, y.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("M", [3, 100, 300])
@pytest.mark.parametrize("act", [RELU, GELU, TANH, SILU])
def test_nan_stays_and_minus_infinity_has_its_limit(M, act):
    bias = torch.tensor([math.nan, -INF, 1.0] * 8, dtype=torch.bfloat16, device="cuda")
    y = call(M, 24, 1, 1, bias, act)
    assert bool(torch.isnan(y[:, 0::3]).all()) and bool(torch.isfinite(y[:, 2::3]).all())
    if act in (RELU, GELU):
        assert bool((y[:, 1::3] == 0).all())
