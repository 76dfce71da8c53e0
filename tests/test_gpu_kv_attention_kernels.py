"""What fp8_kv_attention promises, for each of its kernels in turn: tiles of 8 rows, of 16 rows, and the prompt kernel's
of 128 (a row is a query token and one of the heads that share a KV head)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import fp8_dynamic_scaled_b200.binding as fp8  # noqa: E402
from kv_util import Paged  # noqa: E402
from test_gpu_kv_attention import check, queries, run  # noqa: E402

GROUP = 8
# Up to 8 rows of a sequence always take tiles of 8.  Above, the library compares 14 + 0.27 us per SM and
# tile of 16 rows x 32 tokens with 7 + 2.1 us per 128 tokens and wave of 256-row CTAs: with at most 1000 tokens 16 rows
# of two sequences (256 tiles: 14.5 us against 23.8) stay, 300 tokens x 8 heads of two (38,400: 84 us against 23.8) do not.
NEW = {"8": [1, 1], "16": [2, 2], "prompt": [300, 280]}


def v_scales(p, b, exponents):
    """Sets the V scales of sequence b's pages."""
    pages = p.table[b, :len(exponents)].long()
    p.scale["v"][pages] = torch.exp2(exponents.float())[:, None]


@pytest.mark.parametrize("fmt,dim", [(0, 128), (1, 64)])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("order", ["alternate", "small first", "large first", "random"])
@pytest.mark.parametrize("small,large", [(-56, 24), (-48, 10)])
@pytest.mark.parametrize("kind", sorted(NEW))
def test_v_scales_at_both_ends_of_their_range(kind, small, large, order, page, fmt, dim):
    """V pages 2^80 apart: the tokens of the small ones (pages of zeros have such scales) add nothing to the output
    but count in the softmax's sum."""
    p = Paged([1000, 700], 2, page, dim, fmt, seed=23)
    for b, n in enumerate(p.lens):
        i = torch.arange(-(-n // page), device="cuda")
        half = len(i) // 2
        big = {"alternate": i % 2 == 1, "small first": i >= half, "large first": i < half,
               "random": torch.rand(len(i), generator=p.g, device="cuda") < 0.5}[order]
        v_scales(p, b, torch.where(big, large, small))
    check(p, NEW[kind], GROUP)


@pytest.mark.parametrize("small_first", [False, True])
def test_v_scales_that_differ_between_the_parts_of_a_split(small_first):
    """A long cache whose parts, in different CTAs, each hold V pages of one size alone."""
    p = Paged([60000], 1, 64, 128, 0, seed=24)
    e = torch.full((-(-60000 // 64),), -56.0, device="cuda")
    e[len(e) // 2:] = 24.0
    v_scales(p, 0, e if small_first else e.flip(0))
    check(p, [1], 8)
    check(p, [2], 8)


@pytest.mark.parametrize("bad", [2.0 ** -57, 2.0 ** 25, 0.0, -1.0, float("inf"), float("nan")])
@pytest.mark.parametrize("kind", sorted(NEW))
def test_v_scales_out_of_range_are_reported(kind, bad):
    p = Paged([1000, 700], 2, 16, 64, 0, seed=25)
    q = queries(p, sum(NEW[kind]), GROUP, 1)
    for scale in (bad, 2.0 ** -56, 2.0 ** 24):
        p.scale["v"][p.table[1, 7].long(), 1] = scale
        assert run(p, q, NEW[kind])[1] == (fp8.FP8_ERR_INVALID_ARG if scale is bad else 0)
