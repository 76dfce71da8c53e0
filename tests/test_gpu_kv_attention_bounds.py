"""fp8_kv_attention under bounds far above what the call holds, as a captured graph has them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import fp8_dynamic_scaled_b200.binding as fp8  # noqa: E402
from kv_util import Paged  # noqa: E402
from test_gpu_kv_attention import check, near, queries, run  # noqa: E402


@pytest.mark.parametrize("new", [[1, 1, 1], [3, 0, 5], [200, 1, 64]])
@pytest.mark.parametrize("max_q", [1 << 12, (1 << 24) - 1])
def test_loose_bound_of_the_tokens(new, max_q):
    p = Paged([900, 40, 333], 2, 64, 128, 0, seed=21)
    check(p, new, 8, max_q=max_q, max_kv=1 << 20)


def test_loose_bounds_with_the_most_query_heads():
    p = Paged([5], 1, 16, 64, 0, seed=22)
    q = queries(p, 2, 1 << 16, 3)
    out, st = run(p, q, [2], max_q=1 << 23)
    assert st == 0
    sel = [0, 1, 777, (1 << 16) - 1]
    near(out[:, sel], p, q[:, sel].contiguous(), [2])
