"""The attention kernels' bounded waits: under a limit of 200 ns every call reports FP8_ERR_TIMEOUT and
ends (no hang, no fault, tensor memory freed), and the same call at the default limit is right."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import fp8_dynamic_scaled_b200.binding as fp8  # noqa: E402
from kv_util import Paged  # noqa: E402
from test_gpu_kv_attention import near, queries, run  # noqa: E402


@pytest.fixture
def short_limit():
    fp8.fp8_testing_set_wait_limit_ns(200)
    yield
    fp8.fp8_testing_set_wait_limit_ns(0)


CASES = [([30000, 5000], [1, 1], 8, 128), ([30000, 5000], [1, 1], 8, 64), ([50000], [4], 8, 128),
         ([3000, 2000], [700, 2000], 4, 128), ([3000, 2000], [700, 2000], 4, 64)]


@pytest.mark.parametrize("lens,new,group,dim", CASES)
def test_a_wait_that_runs_out_is_reported(lens, new, group, dim, short_limit):
    p = Paged(lens, 2, 64, dim, 0, seed=1)
    q = queries(p, sum(new), group, 1)
    for _ in range(3):
        assert run(p, q, new)[1] == fp8.FP8_ERR_TIMEOUT
    fp8.fp8_testing_set_wait_limit_ns(0)
    out, st = run(p, q, new)
    assert st == 0
    near(out, p, q, new)
