"""GPU parity of fp8_rmsnorm_quantize with a plain 64-bit form.

Tolerances, from the arithmetic: u = 2^-24 is fp32's half step.  h is one fp32 addition, so
its bf16 rounding is compared bit for bit with torch's.  The mean of squares sums at most
32 squares in each thread, then 10 levels of a tree: all terms are positive, so its relative
error is at most (32 + 10 + 2) u; the root halves it, and the reciprocal root, the three
products and the scale's division add a few u: y and the scales are within EPS = 2^-18 =
64 u of the 64-bit values, relative.  A code is then one of those that values within 2 EPS
of y / scale round to (the quantiser is monotone); y in bf16 is off by half a step (2^-8) more."""
import numpy as np
import pytest
import torch

from fp8_dynamic_scaled_b200 import inputs
from gpu_util import to_dev_bf16

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import fp8_dynamic_scaled_b200.binding as fp8  # noqa: E402

E4, E5 = fp8.FP8_E4M3, fp8.FP8_E5M2
T, R, B1, MX = fp8.FP8_SCALE_TENSOR, fp8.FP8_SCALE_ROW, fp8.FP8_SCALE_BLOCK_1x128, fp8.FP8_SCALE_MX32
F = {E4: 448.0, E5: 57344.0}
DT = {E4: torch.float8_e4m3fn, E5: torch.float8_e5m2}
EPS = 2.0 ** -18
eps_of = 1e-5


def rand(shape, seed, std=1.0, spread=1.0):
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape) * std * np.exp(spread * g.standard_normal((shape[0], 1)))
    return to_dev_bf16(inputs.bf16_bits(x.astype(np.float32)))


def run(x, w, fmt, mode, residual=None, sum_out=None, want_y=False, amax=None, stream=None, eps=eps_of):
    rows, cols = x.shape
    q = torch.full((rows, cols), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.empty(fp8.scale_shape(mode, rows, cols), dtype=torch.uint8 if mode == MX else torch.float32, device="cuda")
    y = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda") if want_y else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp8.fp8_rmsnorm_quantize(x, w, eps, fmt, mode, q, s, residual=residual, sum_out=sum_out, y=y, amax=amax, dev_status=st,
                             stream=stream)
    torch.cuda.synchronize()
    return q, s, y, int(st.item())


def encode(t, fmt):
    return t.clamp(-F[fmt], F[fmt]).float().to(DT[fmt]).float()


def check(x, w, fmt, mode, q, s, residual=None, y=None, amax=None, eps=eps_of):
    d = torch.float64
    h = x.to(d) + (0 if residual is None else residual.to(d))
    ref = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * (1 if w is None else w.to(d))
    rows, cols = ref.shape
    size = {R: cols, B1: 128, MX: 32}.get(mode, cols)
    n = -(-cols // size)
    a = torch.nn.functional.pad(ref.abs(), (0, n * size - cols)).view(rows, n, size).amax(2)
    if mode == MX:
        e = torch.floor(torch.log2(a.clamp(min=2.0 ** -140))).clamp(min=-119) - 8
        near = (torch.log2(a.clamp(min=2.0 ** -140)) - torch.round(torch.log2(a.clamp(min=2.0 ** -140)))).abs() < 2 * EPS
        got = s.to(d) - 127
        assert bool(((got == e) | (near & ((got - e).abs() <= 1)))[a > 0].all())
        assert bool((got[a == 0] == -127).all())
        scale = torch.pow(2.0, got)
    elif mode == T:
        want = np.float32(max(np.float32(amax.item()), np.float32(1e-12))) / np.float32(F[fmt])
        assert s.item() == float(want)
        scale = s.to(d).view(1, 1)
    else:
        want = a.clamp(min=float(np.float32(1e-12))) / F[fmt]
        scale = s.to(d).view(rows, n)
        assert bool(((scale - want).abs() <= EPS * want).all()), float(((scale - want) / want).abs().max())
    per = scale if mode == T else scale.repeat_interleave(size, 1)[:, :cols]
    t = ref / per
    lo, hi = encode(torch.minimum(t * (1 - 2 * EPS), t * (1 + 2 * EPS)), fmt), encode(torch.maximum(t * (1 - 2 * EPS), t * (1 + 2 * EPS)), fmt)
    got = q.view(DT[fmt]).float()
    bad = ~((got >= lo) & (got <= hi))
    assert not bool(bad.any()), f"{int(bad.sum())} codes off, first at {bad.nonzero()[0].tolist()}"
    if y is not None:
        assert bool(((y.to(d) - ref).abs() <= (2.0 ** -8 + EPS) * ref.abs() + 2.0 ** -133).all())


@pytest.mark.parametrize("mode,fmt", [(R, E4), (R, E5), (B1, E4), (B1, E5), (MX, E4), (T, E4), (T, E5)])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (9, 256), (5, 544), (17, 1024), (2, 1056), (300, 4096),
                                       (7, 5152), (1, 8192), (2, 32768)])
def test_against_64_bits(rows, cols, mode, fmt):
    x, r = rand((rows, cols), rows + cols), rand((rows, cols), rows * cols + 1, std=4.0)
    w = rand((1, cols), 5, spread=0.0).view(-1)
    amax = torch.tensor([3.0], device="cuda") if mode == T else None
    q, s, y, st = run(x, w, fmt, mode, want_y=True, amax=amax)
    assert st == 0
    check(x, w, fmt, mode, q, s, y=y, amax=amax)
    h = torch.empty_like(x)
    q, s, y, st = run(x, w, fmt, mode, residual=r, sum_out=h, want_y=True, amax=amax)
    assert st == 0
    check(x, w, fmt, mode, q, s, residual=r, y=y, amax=amax)
    assert torch.equal(h, (x.float() + r.float()).bfloat16())


def test_16_columns_and_no_weight():
    x = rand((33, 16), 2)
    for mode in (R, B1):
        q, s, _, st = run(x, None, E4, mode)
        assert st == 0
        check(x, None, E4, mode, q, s)


@pytest.mark.parametrize("into", ["x", "residual"])
def test_sum_in_place_and_strided(into):
    rows, cols = 37, 640
    xb, rb = rand((rows, 1024), 3), rand((rows, 800), 4)
    x, r = xb[:, 128:128 + cols], rb[:, 8:8 + cols]
    x0, r0, xb0, rb0 = x.clone(), r.clone(), xb.clone(), rb.clone()
    w = rand((1, cols), 5).view(-1)
    q, s, _, st = run(x, w, E4, R, residual=r, sum_out=x if into == "x" else r)
    assert st == 0
    check(x0, w, E4, R, q, s, residual=r0)
    h = (x0.float() + r0.float()).bfloat16()
    assert torch.equal(x if into == "x" else r, h)
    xb0[:, 128:128 + cols], rb0[:, 8:8 + cols] = x, r          # nothing else was written
    assert torch.equal(xb, xb0) and torch.equal(rb, rb0)


def test_zero_rows_and_extreme_rows():
    """Rows of zeros; of 2^63 and of bf16's largest values, whose squares leave fp32; of subnormals."""
    cols = 512
    w = rand((1, cols), 6, spread=0.0).view(-1)
    x = torch.zeros((7, cols), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for i, size in ((1, 2.0 ** 63), (2, 2.0 ** 100), (3, 2.0 ** -130), (4, 2.0 ** 66), (5, 2.0 ** -64)):
        x[i] = (torch.rand(cols, generator=g, device="cuda") * 2 - 1) * size
    x[6] = torch.finfo(torch.bfloat16).max
    x[6, ::2] *= -1
    for mode in (R, B1, MX):
        q, s, y, st = run(x, w, E4, mode, want_y=True)
        assert st == 0
        check(x, w, E4, mode, q, s, y=y)
        assert int((q[0] & 0x7F).max()) == 0


def test_wide_spread_of_eps():
    x, w = rand((4, 256), 8, std=1e-6), rand((1, 256), 9).view(-1)
    for eps in (1e-20, 1e-12, 1.0, 1e6):
        q, s, y, st = run(x, w, E4, R, want_y=True, eps=eps)
        assert st == 0
        check(x, w, E4, R, q, s, y=y, eps=float(np.float32(eps)))


def test_nonfinite_rows_are_reported_and_stay_in_their_rows():
    x, w = rand((6, 384), 11), rand((1, 384), 12).view(-1)
    q0, s0, _, _ = run(x, w, E4, R)
    for bad in (float("nan"), float("inf"), -float("inf")):
        xb = x.clone()
        xb[2, 100] = bad
        q, s, _, st = run(xb, w, E4, R)
        assert st == fp8.FP8_ERR_NONFINITE
        keep = [0, 1, 3, 4, 5]
        assert torch.equal(q[keep], q0[keep]) and torch.equal(s[keep], s0[keep])
    big = torch.full_like(x, torch.finfo(torch.bfloat16).max)
    assert run(big, w, E4, R, residual=big, sum_out=torch.empty_like(big))[3] == fp8.FP8_ERR_NONFINITE  # h overflows
    am = torch.tensor([float("nan")], device="cuda")
    assert run(x, w, E4, T, amax=am)[3] == fp8.FP8_ERR_NONFINITE


def test_given_amax_below_the_values_saturates():
    x, w = rand((8, 256), 13, spread=0.0), rand((1, 256), 14, spread=0.0).view(-1)
    for a in (1e-30, 1e-3, 0.0):
        am = torch.tensor([a], device="cuda")
        q, s, _, st = run(x, w, E4, T, amax=am)
        assert st == 0
        check(x, w, E4, T, q, s, amax=am)


def test_empty():
    for rows, cols in ((0, 128), (5, 0)):
        x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
        for mode in (R, B1, MX):
            _, s, _, st = run(x, None, E4, mode)
            assert st == 0
            if mode == R and rows:
                assert bool((s == float(np.float32(1e-12) / np.float32(448))).all())
        _, s, _, st = run(x, None, E4, T, amax=torch.tensor([2.0], device="cuda"))
        assert st == 0 and s.item() == float(np.float32(2.0) / np.float32(448))


def test_more_than_2_31_elements():
    rows, cols = 262400, 8192                       # 2.15e9 elements
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[0], x[-1] = rand((1, cols), 15)[0], rand((1, cols), 16)[0]
    q, s, _, st = run(x, None, E4, R)
    assert st == 0
    check(x[[0, rows - 1]], None, E4, R, q[[0, rows - 1]], s[[0, rows - 1]])


def test_side_stream_and_graph():
    x, r = rand((65, 2048), 17), rand((65, 2048), 18)
    w = rand((1, 2048), 19).view(-1)
    q = torch.empty((65, 2048), dtype=torch.uint8, device="cuda")
    s = torch.empty(65, device="cuda")
    h = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call():
        fp8.fp8_rmsnorm_quantize(x, w, eps_of, E4, R, q, s, residual=r, sum_out=h, stream=side)
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    check(x, w, E4, R, q, s, residual=r)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side, capture_error_mode="thread_local"):
        call()
    for seed in (20, 21):
        x.copy_(rand((65, 2048), seed))
        q.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(x, w, E4, R, q, s, residual=r)
        assert torch.equal(h, (x.float() + r.float()).bfloat16())
