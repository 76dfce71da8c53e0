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
# of two sequences and two KV heads (128 tiles: 14.2 us against 23.8) stay, 300 tokens x 8 heads (19,200: 49 us) do not.
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


@pytest.mark.parametrize("dim,fmt", [(128, 0), (64, 1)])
@pytest.mark.parametrize("kind", sorted(NEW))
def test_one_hot_softmax_picks_its_token(kind, dim, fmt):
    """Scores that are exact (sums of small integers), one token of each head ahead of all others by 64 nats or more: the
    output is that token's V, whose codes bf16 holds, bit for bit (a weight's rounding to fp16, 2^-11, is
    below half a step of bf16, 2^-9 of the value)."""
    p = Paged([1000, 700], 2, 32, dim, fmt, seed=26)
    g = torch.Generator(device="cuda").manual_seed(3)
    signs = torch.randint(0, 2, (2 * GROUP, dim), generator=g, device="cuda") * 2.0 - 1.0
    dt = torch.float8_e4m3fn if fmt == 0 else torch.float8_e5m2
    k = torch.randint(-4, 5, p.codes["k"].shape, generator=g, device="cuda").float()        # |score| <= 4 dim
    want = []
    for b, n in enumerate(p.lens):
        rows = torch.empty((2 * GROUP, dim), dtype=torch.float64, device="cuda")
        at = torch.randperm(400, generator=g, device="cuda")[:2 * GROUP].tolist()           # seen by every query
        for h, t in enumerate(at):
            k[p.table[b, t // 32].long(), h // GROUP, t % 32] = 8 * signs[h]                # score 8 dim
            rows[h] = p.values("v", b, n)[h // GROUP, t]
        want.append(rows)
    p.codes["k"] = torch.where(p.codes["k"] == (0x7F if fmt == 0 else 0x7E), p.codes["k"], k.to(dt).view(torch.uint8))
    p.scale["k"].fill_(0.25)
    new = NEW[kind]
    for std in (1.0, 2.0 ** 60, 2.0 ** -60):
        q = (signs * std).bfloat16().expand(sum(new), 2 * GROUP, dim).contiguous()
        out, st = run(p, q, new, scale=64.0 / dim / std)             # 4 dim of the 8 dim: 64 nats at least
        assert st == 0
        ref = torch.cat([w.expand(n, 2 * GROUP, dim) for w, n in zip(want, new)])
        assert torch.equal(out.double(), ref)


@pytest.mark.parametrize("scale,std", [(-0.1, 1.0), (0.0, 1.0), (1.0, 0.3), (1e-30, 2.0 ** 80), (2.0 ** 90, 2.0 ** -100)])
@pytest.mark.parametrize("kind", sorted(NEW))
def test_softmax_scales_and_query_sizes(kind, scale, std):
    check(Paged([1000, 700], 2, 16, 64, 0, seed=27), NEW[kind], GROUP, std=std, scale=scale)


@pytest.mark.parametrize("fmt,dim", [(0, 128), (1, 64)])
@pytest.mark.parametrize("kind", sorted(NEW))
def test_scales_that_differ_and_are_no_powers_of_two(kind, fmt, dim):
    p = Paged([1000, 700], 2, 32, dim, fmt, seed=28)
    g = torch.Generator(device="cuda").manual_seed(4)
    for n, spread in (("k", 3), ("v", 20)):
        e = (torch.rand(p.scale[n].shape, generator=g, device="cuda") * 2 - 1) * spread
        p.scale[n] *= torch.exp2(e)
    check(p, NEW[kind], GROUP, std=0.2)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 16, 20])
def test_ragged_calls_of_a_few_tokens(group, dim):
    """Tiles of 8 and 16 rows: up to 80 rows a sequence (5 sequences, 2 KV heads, 700 tokens: 16 us against 19.6)."""
    check(Paged([40, 1, 300, 16, 700], 2, 32, dim, 0, seed=group), [3, 1, 2, 0, 4], group, std=2.0)


@pytest.mark.parametrize("group,dim", [(8, 128), (4, 64)])
def test_prompts_and_single_tokens_in_one_call(group, dim):
    """Chunked serving: most sequences add one token, some over a long cache, while one or two bring a chunk."""
    lens = [900, 1, 20000, 640, 33, 3000, 129, 700, 16, 2048]
    new = [1, 1, 1, 640, 1, 1, 129, 1, 0, 300]
    check(Paged(lens, 2, 64, dim, 0, seed=29), new, group)
    check(Paged(lens, 1, 16, dim, 1, seed=30), [min(n, 2) for n in new], group)
