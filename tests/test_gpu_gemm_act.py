"""GPU parity of fp8_scaled_gemm_act / fp8_linear_forward_act: y = act(acc + bias) + residual.

References in 64 bits.  The GEMM's own error is the acceptance rule of the other GEMM tests,
1e-3 of the sum of the terms' magnitudes; an activation stretches it by its steepest slope
(at most 1.13, GELU's) and adds a few fp32 steps; the last rounding is half a bf16 step, 2^-8.
Where operands are small integers with power-of-two scales the accumulator is exact, and the
activation is held to the last rounding alone, in its tails too."""
import math

import numpy as np
import pytest
import torch

import oracle
from fp8_dynamic_scaled_b200 import inputs
from gpu_util import to_dev_bf16

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import fp8_dynamic_scaled_b200.binding as fp8  # noqa: E402

E4, E5 = fp8.FP8_E4M3, fp8.FP8_E5M2
T, R, B1, B128, MX = (fp8.FP8_SCALE_TENSOR, fp8.FP8_SCALE_ROW, fp8.FP8_SCALE_BLOCK_1x128,
                      fp8.FP8_SCALE_BLOCK_128x128, fp8.FP8_SCALE_MX32)
NONE, RELU, GELU, TANH, SILU = range(5)
PAIRS = [(R, R), (T, R), (B1, B128), (MX, MX)]


def act64(v, act):
    if act == RELU:
        return v.clamp(min=0)
    if act == GELU:
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2.0))
    if act == TANH:
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if act == SILU:
        return v * torch.sigmoid(v)
    return v


def bf16(shape, seed, std=1.0):
    return to_dev_bf16(inputs.bf16_bits((np.random.default_rng(seed).standard_normal(shape) * std).astype(np.float32)))


def operands(M, N, K, am, bm, seed):
    g = np.random.default_rng(seed)
    x = inputs.bf16_bits(g.standard_normal((M, K)).astype(np.float32))
    w = inputs.bf16_bits((g.standard_normal((N, K)) * 0.1).astype(np.float32))
    qa, sa, _ = oracle.quantize(x, E4, am, dequant=False)
    qb, sb, _ = oracle.quantize(w, E4, bm, dequant=False)
    ref, bound = oracle.gemm_ref_full(qa, sa, am, E4, qb, sb, bm, E4)
    dev = [torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in (qa, sa, qb, sb, ref, bound)]
    return dev[:4], dev[4], dev[5], x


def expect(ref, bound, bias, act, res):
    v = ref + (0 if bias is None else bias.double())
    y = act64(v, act) + (0 if res is None else res.double())
    lim = 1.13 * (1e-3 * bound + 2.0 ** -22 * v.abs()) + 2.0 ** -8 * y.abs() + 2.0 ** -20 * (0 if res is None else res.double().abs())
    return y, lim


def near(y, ref, lim, what=""):
    d = (y.double() - ref).abs()
    bad = ~(d <= lim)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("am,bm", PAIRS)
@pytest.mark.parametrize("act", [NONE, RELU, GELU, TANH, SILU])
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (5, 130, 96), (16, 512, 256), (64, 200, 1056), (65, 300, 160),
                                   (130, 257, 288), (256, 512, 512), (300, 264, 128), (515, 1000, 64)])
def test_against_64_bits(M, N, K, act, am, bm):
    (a, sa, b, sb), ref, bound, _ = operands(M, N, K, am, bm, M * 7 + N + K)
    bias, res = bf16(N, 1), bf16((M, N), 2, 4.0)
    for use_bias, use_res in ((True, True), (False, True), (False, False)):
        y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        bb, rr = bias if use_bias else None, res if use_res else None
        fp8.fp8_scaled_gemm_act(a, sa, am, E4, b, sb, bm, E4, y, bias=bb, activation=act, residual=rr, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        near(y, *expect(ref, bound, bb, act, rr), what=f"bias {use_bias} residual {use_res}")


@pytest.mark.parametrize("M", [3, 100, 300])        # the decode, the tiled, the CTA-pair kernel
@pytest.mark.parametrize("act", [RELU, GELU, TANH, SILU])
def test_activation_alone_over_its_range(M, act):
    """acc = n / 16 over [-24, 24), exactly: K = 32, one code of each row times one of each column."""
    N = 768
    a = torch.zeros((M, 32), dtype=torch.uint8, device="cuda")
    a[:, 0] = a[:, 1] = 0x38                        # 1.0
    v = (torch.arange(N, device="cuda") - N // 2) / 16.0
    whole = torch.round(v)                          # |whole| <= 24: 16 + the rest, both exact in E4M3
    b = torch.zeros((N, 32), device="cuda")
    b[:, 0], b[:, 1] = whole.clamp(-16, 16), (whole - whole.clamp(-16, 16)) + 0
    a2 = a.clone()
    a2[:, 2] = 0x38
    b[:, 2] = v - whole                             # multiples of 1/16, at most 1/2
    bq = b.to(torch.float8_e4m3fn)
    assert torch.equal(bq.float(), b)
    one_a, one_b = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    fp8.fp8_scaled_gemm_act(a2, one_a, R, E4, bq.view(torch.uint8), one_b, R, E4, y, activation=act)
    ref = act64(v.double(), act)[None, :].expand(M, N)
    # exp's and erfc's relative error grows with the argument: 2^-16 covers |v| <= 24 for SILU and GELU; the
    # tanh form's exponent reaches 2 * 0.798 * (24 + 0.0447 * 24^3) > 1000, where the result is below bf16's range
    near(y, ref, (2.0 ** -8 + 2.0 ** -14) * ref.abs() + 2.0 ** -126)


@pytest.mark.parametrize("am,bm", PAIRS)
@pytest.mark.parametrize("M,N", [(7, 520), (129, 256), (300, 1024), (300, 130)])
def test_residual_in_place_equals_out_of_place(M, N, am, bm):
    K = 256
    (a, sa, b, sb), ref, bound, _ = operands(M, N, K, am, bm, 3)
    res = bf16((M, N), 4, 4.0)
    y = torch.empty_like(res)
    fp8.fp8_scaled_gemm_act(a, sa, am, E4, b, sb, bm, E4, y, activation=SILU, residual=res)
    z = res.clone()
    fp8.fp8_scaled_gemm_act(a, sa, am, E4, b, sb, bm, E4, z, activation=SILU, residual=z)
    assert torch.equal(y.view(torch.int16), z.view(torch.int16))
    near(z, *expect(ref, bound, None, SILU, res))


@pytest.mark.parametrize("M", [8, 100, 300])
def test_strided_and_unaligned_residual(M):
    N, K = 136, 128
    (a, sa, b, sb), ref, bound, _ = operands(M, N, K, R, R, 5)
    for off, ld in ((0, 200), (8, 144), (1, 201), (3, 139)):
        buf = bf16((M, ld), off + ld)
        res = buf[:, off:off + N]
        out = torch.full((M, ld), 7.0, dtype=torch.bfloat16, device="cuda")
        y = out[:, off:off + N]
        fp8.fp8_scaled_gemm_act(a, sa, R, E4, b, sb, R, E4, y, residual=res)
        near(y, *expect(ref, bound, None, NONE, res))
        out[:, off:off + N] = 7.0                   # nothing outside was written
        assert bool((out == 7.0).all())


@pytest.mark.parametrize("am,bm", PAIRS)
@pytest.mark.parametrize("M,N", [(2, 1), (7, 5), (100, 39), (147, 372), (300, 3), (290, 250), (586, 1157)])
def test_columns_beside_y_are_left(M, N, am, bm):
    """Rows that start on 16 bytes while the last columns end inside 16 bytes: the neighbours of a
    column view keep their bits, for the plain GEMM, the older options and these."""
    K = 256
    (a, sa, b, sb), ref, bound, _ = operands(M, N, K, am, bm, 11)
    ld = (N + 7) // 8 * 8 + 8
    res = bf16((M, N), 4, 4.0)
    for call in range(4):
        out = torch.full((M, ld), 7.0, dtype=torch.bfloat16, device="cuda")
        y = out[:, :N]
        if call == 0:
            fp8.fp8_scaled_gemm(a, sa, am, E4, b, sb, bm, E4, y)
        elif call == 1:
            fp8.fp8_scaled_gemm_ex(a, sa, am, E4, b, sb, bm, E4, y, bias=bf16(N, 1))
        elif call == 2:
            fp8.fp8_scaled_gemm_act(a, sa, am, E4, b, sb, bm, E4, y, activation=SILU, residual=res)
        else:
            y.copy_(res)
            fp8.fp8_scaled_gemm_act(a, sa, am, E4, b, sb, bm, E4, y, residual=y)
        near(y, *expect(ref, bound, bf16(N, 1) if call == 1 else None, SILU if call == 2 else NONE,
                        res if call > 1 else None), what=f"call {call}")
        assert bool((out[:, N:] == 7.0).all()), f"call {call}"


@pytest.mark.parametrize("am,bm", PAIRS)
@pytest.mark.parametrize("M", [9, 70, 290])
def test_amax_and_fp8_output_follow_y(M, am, bm):
    N, K = 272, 128
    (a, sa, b, sb), ref, bound, _ = operands(M, N, K, am, bm, 6)
    bias, res = bf16(N, 7), bf16((M, N), 8)
    for fmt, dt, top in ((E4, torch.float8_e4m3fn, 448.0), (E5, torch.float8_e5m2, 57344.0)):
        y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        amax = torch.zeros(1, device="cuda")
        yq = torch.empty((M, N), dtype=torch.uint8, device="cuda")
        only = torch.empty_like(yq)
        s = torch.tensor([0.01], device="cuda")
        fp8.fp8_scaled_gemm_act(a, sa, am, E4, b, sb, bm, E4, y, bias=bias, activation=TANH, residual=res, amax=amax,
                                yq=yq, yq_scale=s, yq_fmt=fmt)
        fp8.fp8_scaled_gemm_act(a, sa, am, E4, b, sb, bm, E4, None, bias=bias, activation=TANH, residual=res, yq=only,
                                yq_scale=s, yq_fmt=fmt)
        near(y, *expect(ref, bound, bias, TANH, res))
        assert amax.item() == y.float().abs().max().item()
        want = (y.float() / s).clamp(-top, top).to(dt).view(torch.uint8)
        assert torch.equal(yq, want) and torch.equal(only, want)


def test_nothing_set_is_the_plain_gemm_and_zero_k():
    (a, sa, b, sb), _, _, _ = operands(300, 256, 256, R, R, 9)
    y, z = (torch.empty((300, 256), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fp8.fp8_scaled_gemm(a, sa, R, E4, b, sb, R, E4, y)
    fp8.fp8_scaled_gemm_act(a, sa, R, E4, b, sb, R, E4, z)
    assert torch.equal(y.view(torch.int16), z.view(torch.int16))
    for M, N in ((1, 24), (130, 50)):
        a, b = (torch.empty((n, 0), dtype=torch.uint8, device="cuda") for n in (M, N))
        one = torch.ones(max(M, N), device="cuda")
        bias, res = bf16(N, 10), bf16((M, N), 11)
        y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        fp8.fp8_scaled_gemm_act(a, one[:M], R, E4, b, one[:N], R, E4, y, bias=bias, activation=GELU, residual=res)
        near(y, *expect(torch.zeros((M, N), dtype=torch.float64, device="cuda"), 0.0, bias, GELU, res))
        fp8.fp8_scaled_gemm_act(a, one[:M], R, E4, b, one[:N], R, E4, y, residual=res)
        assert torch.equal(y, res)


@pytest.mark.parametrize("am,bm", PAIRS)
@pytest.mark.parametrize("M", [4, 320])
def test_linear_forward_act(M, am, bm):
    N, K = 256, 512
    (a, sa, b, sb), ref, bound, x = operands(M, N, K, am, bm, 12)
    bias, res = bf16(N, 13), bf16((M, N), 14)
    y = res.clone()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp8.fp8_linear_forward_act(to_dev_bf16(x), E4, am, b, sb, bm, E4, y, fp8.workspace_for(2, M, N, K, am), bias=bias,
                               activation=SILU, residual=y, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    near(y, *expect(ref, bound, bias, SILU, res))


def test_side_stream_and_graph():
    M, N, K = 40, 384, 256
    (a, sa, b, sb), ref, bound, _ = operands(M, N, K, R, R, 15)
    res = bf16((M, N), 16)
    y = torch.empty_like(res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call():
        fp8.fp8_scaled_gemm_act(a, sa, R, E4, b, sb, R, E4, y, activation=GELU, residual=res, stream=side)
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side, capture_error_mode="thread_local"):
        call()
    for seed in (17, 18):
        res.copy_(bf16((M, N), seed))
        g.replay()
        torch.cuda.synchronize()
        near(y, *expect(ref, bound, None, GELU, res))


@pytest.mark.parametrize("am,bm", PAIRS)
@pytest.mark.parametrize("M,N,ldq", [(9, 131, 131), (70, 270, 275), (290, 33, 40), (290, 515, 515), (257, 1, 3)])
def test_codes_of_unaligned_rows(M, N, ldq, am, bm):
    """FP8 output whose rows start at any byte, with and without Y; nothing outside is written."""
    K = 128
    (a, sa, b, sb), ref, bound, _ = operands(M, N, K, am, bm, 17)
    res, s = bf16((M, N), 18), torch.tensor([0.02], device="cuda")
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    for with_y in (True, False):
        buf = torch.full((M, ldq), 0x55, dtype=torch.uint8, device="cuda")
        yq = buf[:, ldq - N:]
        amax = torch.zeros(1, device="cuda")
        fp8.fp8_scaled_gemm_act(a, sa, am, E4, b, sb, bm, E4, y if with_y else None, activation=SILU, residual=res,
                                amax=amax, yq=yq, yq_scale=s)
        near(y, *expect(ref, bound, None, SILU, res))
        assert amax.item() == y.float().abs().max().item()
        assert torch.equal(yq, (y.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        assert bool((buf[:, :ldq - N] == 0x55).all())
