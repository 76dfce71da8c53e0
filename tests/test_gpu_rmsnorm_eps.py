"""fp8_rmsnorm_quantize with an eps near either end of the fp32 range, and rows whose mean square is as far off.

The tolerance is test_gpu_rmsnorm's, EPS relative, and one term more: y = RN(RN(h rstd) w) can be subnormal here
(1e-30 under an eps of 1e20), and a product that is subnormal is rounded by up to 2^-150 whatever its size.
The first product's error passes through w, so that y is off by 2^-150 (|w| + 1) at most, and y / scale by that
over the scale.  (The scales need no such term: one below 1e-12 / F_max, or the least of E8M0, is clamped.)"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
from test_gpu_rmsnorm import B1, DT, E4, EPS, F, MX, R, encode, rand, run  # noqa: E402

EPS_VALUES = [3.4e38, 1e38, 1e34, 1e20, 1e-30, 1e-37, 1e-40, 1e-44, 1.5e-45]
SIZES = [0.0, 2.0 ** -133, 1e-30, 3e-23, 1e-22, 3e-20, 1e-10, 1.0, 1e10, 1.8e19, 2.0 ** 66, 3e38]


def check(x, w, mode, q, s, y, eps):
    d = torch.float64
    h = x.to(d)
    ref = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w.to(d)
    rows, cols = ref.shape
    size = {R: cols, B1: 128, MX: 32}[mode]
    n = -(-cols // size)
    a = torch.nn.functional.pad(ref.abs(), (0, n * size - cols)).view(rows, n, size).amax(2)
    got = s.to(d).view(rows, n)
    if mode == MX:
        low, high = (torch.floor(torch.log2((a * f).clamp(min=2.0 ** -119))) - 8 for f in (1 - 2 * EPS, 1 + 2 * EPS))
        assert bool(((got - 127 >= low) & (got - 127 <= high)).all())
        scale = torch.exp2(got - 127)
    else:
        want = a.clamp(min=float(np.float32(1e-12))) / F[E4]
        assert bool(((got - want).abs() <= EPS * want).all())
        scale = got
    per = scale.repeat_interleave(size, 1)[:, :cols]
    t, step = ref / per, 2.0 ** -150 * (w.to(d).abs() + 1) / per
    slack = 2 * EPS * t.abs() + step
    lo, hi = encode(t - slack, E4), encode(t + slack, E4)
    c = q.view(DT[E4]).float()
    bad = ~((c >= lo) & (c <= hi))
    assert not bool(bad.any()), f"{int(bad.sum())} codes off, first at {bad.nonzero()[0].tolist()}"
    assert bool(((y.to(d) - ref).abs() <= (2.0 ** -8 + EPS) * ref.abs() + 2.0 ** -133).all())


@pytest.mark.parametrize("eps", EPS_VALUES)
@pytest.mark.parametrize("cols", [256, 1056, 2080, 8192])
def test_eps_near_the_ends_of_the_range(cols, eps):
    g = torch.Generator(device="cuda").manual_seed(cols)
    u = (torch.rand((len(SIZES), cols), generator=g, device="cuda") * 2 - 1).double()
    x = (u * torch.tensor(SIZES, device="cuda", dtype=torch.float64)[:, None]).bfloat16()
    w = rand((1, cols), 9, spread=0.0).view(-1)
    r = torch.zeros_like(x)
    for mode in (R, B1, MX):
        for res in (None, r):
            q, s, y, st = run(x, w, E4, mode, residual=res, want_y=True, eps=eps)
            assert st == 0
            check(x, w, mode, q, s, y, float(np.float32(eps)))
