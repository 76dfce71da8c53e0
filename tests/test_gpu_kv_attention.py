"""fp8_kv_attention against attention in 64 bits over the dequantised cache (kv_util states the tolerance)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import fp8_dynamic_scaled_b200.binding as fp8  # noqa: E402
from kv_util import Paged, attention64, starts  # noqa: E402


def queries(paged, T, group, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((T, group * paged.heads, paged.dim), generator=g, device="cuda") * std).bfloat16()


def run(paged, q, new, scale=None, use_cu=True, max_q=None, max_kv=None, out=None, stream=None, lens=None):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, float("nan")) if out is None else out
    cu = torch.tensor(starts(new), dtype=torch.int32, device="cuda") if use_cu else None
    max_q = max(new + [1]) if max_q is None else max_q
    max_kv = max(paged.lens + [1]) if max_kv is None else max_kv
    cache = paged.cache(fp8)
    ws = fp8.kv_attention_workspace(q, cache, len(new), max_q, max_kv)
    if ws is not None:
        ws.fill_(0xFF)                              # needs no initialisation
    fp8.fp8_kv_attention(q, cache, paged.table, paged.kv_lens if lens is None else lens, out, max_kv_len=max_kv, cu_q=cu,
                         max_q_len=max_q, softmax_scale=scale, workspace=ws, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    return out, int(st.item())


def near(out, paged, q, new, scale=None):
    cu = starts(new)
    ref, lim = attention64(paged, q, cu, paged.dim ** -0.5 if scale is None else scale)
    d = (out[:cu[-1]].double() - ref).abs()
    bad = ~(d <= lim)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}, " \
                                f"worst {float((d / lim.clamp(min=1e-30)).nan_to_num(9e9).max()):.3g} of the limit"


def check(paged, new, group, seed=1, std=1.0, scale=None, **kw):
    q = queries(paged, sum(new), group, seed, std)
    out, st = run(paged, q, new, scale, **kw)
    assert st == 0
    near(out, paged, q, new, scale)
    return out


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_single_tokens(page, dim, fmt):
    lens = [1, 2, 15, 16, 17, page, page + 1, 500, 0, 129]
    for heads, group in ((1, 1), (2, 8), (1, 5)):
        check(Paged(lens, heads, page, dim, fmt, seed=page + dim + heads), [1] * len(lens), group, use_cu=False)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 7, 8, 16, 20])
def test_ragged_chunks(group, dim):
    lens = [40, 1, 300, 16, 0, 70, 129]
    new = [3, 1, 17, 16, 0, 0, 64]
    check(Paged(lens, 2, 32, dim, 0, seed=group), new, group, std=2.0)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_prompts(page, dim, fmt):
    """Whole prompts and chunks behind earlier tokens, at sizes around the tiles' edges."""
    lens = [127, 128, 129, 257, 700, 1025]
    new = [127, 128, 129, 255, 130, 1]
    check(Paged(lens, 2, page, dim, fmt, seed=page), new, 4)


def test_long_prompt():
    check(Paged([2500, 1900], 1, 64, 128, 0, seed=3), [2300, 1900], 8)


@pytest.mark.parametrize("lens", [[5000], [100003, 7], [1, 20000, 513, 0]])
@pytest.mark.parametrize("fmt", [0, 1])
def test_long_caches_are_split(lens, fmt):
    for page in (16, 128):
        check(Paged(lens, 2, page, 128, fmt, seed=4), [1] * len(lens), 8)
    check(Paged(lens, 2, 64, 64, fmt, seed=5), [min(n, 4) for n in lens], 4)


def test_max_kv_above_the_lengths_changes_only_the_split():
    p = Paged([900, 30], 2, 64, 128, 0, seed=6)
    for max_kv in (900, 4096, 100000):
        check(p, [1, 1], 8, max_kv=max_kv)


@pytest.mark.parametrize("std", [1e-3, 30.0, 1e4])
def test_flat_and_one_hot_softmax(std):
    check(Paged([700, 333], 2, 32, 128, 0, seed=7), [5, 40], 4, std=std)


def test_scales_of_very_different_pages():
    """V pages 2^40 apart: the weight of a page counts with its scale."""
    p = Paged([640, 200], 2, 16, 128, 0, seed=8)
    g = torch.Generator(device="cuda").manual_seed(1)
    e = torch.randint(-20, 21, p.scale["v"].shape, generator=g, device="cuda")
    p.scale["v"] *= torch.exp2(e.float())
    check(p, [1, 9], 8)
    p.scale["k"] *= torch.exp2(torch.randint(-3, 4, p.scale["k"].shape, generator=g, device="cuda").float())
    check(p, [1, 9], 8, std=0.2)


def test_scales_that_are_no_powers_of_two():
    p = Paged([300, 64], 2, 32, 64, 1, seed=9)
    for n in "kv":
        p.scale[n] *= 1.37
    check(p, [2, 64], 4)


def test_other_softmax_scales_and_query_sizes():
    p = Paged([200], 1, 16, 64, 0, seed=10)
    for scale, std in ((1.0, 0.3), (0.01, 1.0), (-0.1, 1.0), (0.0, 1.0), (1e-30, 2.0 ** 80), (2.0 ** 90, 2.0 ** -100)):
        check(p, [3], 4, std=std, scale=scale)


def test_zero_queries_and_tokens_that_see_nothing():
    p = Paged([40, 2], 2, 16, 64, 0, seed=11)
    q = queries(p, 8, 4, 1)
    q[0] = 0
    out, st = run(p, q, [3, 5])                     # 5 tokens of a sequence that holds 2: three see nothing
    assert st == 0 and bool((out[3:6] == 0).all())
    ref, lim = attention64(p, q[[0, 1, 2, 6, 7]], [0, 3, 5], 0.125)
    assert bool(((out[[0, 1, 2, 6, 7]].double() - ref).abs() <= lim).all())
    assert bool(torch.isfinite(out).all())


def test_empty_caches():
    p = Paged([0, 0], 2, 16, 64, 0, seed=11)
    q = queries(p, 2, 4, 1)
    for max_kv in (0, 64):
        out, st = run(p, q, [1, 1], max_kv=max_kv)
        assert st == 0 and bool((out == 0).all())
    out, st = run(p, q, [0, 0])                     # no tokens in the call: nothing is written
    assert st == 0 and bool(torch.isnan(out).all())


def test_strided_rows_and_rows_behind_the_last_sequence():
    p = Paged([70, 33], 2, 32, 64, 0, seed=12)
    wide = queries(Paged([1], 12, 16, 64, 0), 10, 1, 2)             # 12 heads of 64 per row
    q = wide[:, 2:10]
    buf = torch.full((10, 12, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, 4:12]
    got, st = run(p, q, [3, 4], out=out, max_q=6)
    assert st == 0
    near(out, p, q, [3, 4])
    assert bool((buf[:, :4] == 5.0).all()) and bool((buf[7:] == 5.0).all())


def test_results_do_not_depend_on_the_other_sequences_and_repeat():
    p = Paged([900, 40, 333], 2, 64, 128, 0, seed=13)
    q = queries(p, 3, 8, 3)
    a, _ = run(p, q, [1, 1, 1])
    b, _ = run(p, q, [1, 1, 1])
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    pages = p.table[1, :1].long()
    for n in "kv":
        p.codes[n][pages] = 0x11
    c, _ = run(p, q, [1, 1, 1])
    assert torch.equal(a[[0, 2]].view(torch.int16), c[[0, 2]].view(torch.int16))


@pytest.mark.parametrize("what", ["page", "cu", "max_q", "long", "beyond_max_kv", "negative"])
@pytest.mark.parametrize("rows", [1, 200])
def test_bad_device_arguments_are_reported(what, rows):
    p = Paged([400, 400], 2, 16, 64, 0, seed=14)
    q = queries(p, 2 * rows, 2, 4)
    cu, lens, max_q, max_kv = [0, rows, 2 * rows], [400, 400], rows, 400
    if what == "page":
        p.table[1, 3] = 10 ** 6
    elif what == "cu":
        cu = [0, rows, 2 * rows + 1]
    elif what == "max_q":
        cu = [0, rows - 1, 2 * rows]
    elif what == "long":
        lens = [400, p.table.shape[1] * 16 + 1]
        max_kv = 10 ** 5
    elif what == "beyond_max_kv":
        max_kv = 399
        lens = [399, 400]
    else:
        lens = [400, -5]
    cache = p.cache(fp8)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    ws = fp8.kv_attention_workspace(q, cache, 2, max_q, max_kv)
    fp8.fp8_kv_attention(q, cache, p.table, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, max_kv_len=max_kv,
                         cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_q_len=max_q, workspace=ws,
                         dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == fp8.FP8_ERR_INVALID_ARG
    n, keep = cu[1], lens[0]
    p.lens = [keep, 0]
    ref, lim = attention64(p, q[:n], [0, n, n], 0.125)
    assert bool(((out[:n].double() - ref).abs() <= lim).all())


def test_offsets_past_32_bits():
    """A cache of more than 2^32 code bytes, its last pages in use."""
    pages, heads, page, dim = 70000, 8, 64, 128                      # 4.6e9 bytes of K
    k = torch.zeros((pages, heads, page, dim), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    s = torch.ones((pages, heads), device="cuda")
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    cache = fp8.KVCache(k, v, s, s.clone())
    x = queries(Paged([1], 8, 16, 128, 0), 150, 1, 5)
    fp8.fp8_kv_append(x, x, cache, table, lens, cu_q=torch.tensor([0, 150], dtype=torch.int32, device="cuda"), max_q_len=150)
    p = Paged([150], 8, 64, 128, 0, seed=15)
    p.codes, p.scale, p.table = {"k": k, "v": v}, {"k": s, "v": cache.v_scale}, table
    check(p, [1], 2)
    check(p, [150], 2)


def test_side_stream_and_graph_over_a_growing_sequence():
    """A captured decode step (append, then attention), replayed as the lengths on the device grow."""
    p = Paged([700, 700], 2, 64, 128, 0, seed=16)
    g0 = torch.Generator(device="cuda").manual_seed(2)
    lens = torch.tensor([600, 63], dtype=torch.int32, device="cuda")
    q = queries(p, 2, 8, 6)
    k, v = (torch.randn((2, 2, 128), generator=g0, device="cuda").bfloat16() for _ in range(2))
    out = torch.empty_like(q)
    cache = p.cache(fp8)
    ws = fp8.kv_attention_workspace(q, cache, 2, 1, 700)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        fp8.fp8_kv_append(k, v, cache, p.table, lens, stream=side)
        fp8.fp8_kv_attention(q, cache, p.table, lens, out, max_kv_len=700, workspace=ws, stream=side)
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side, capture_error_mode="thread_local"):
        step()
    for i in range(3):
        lens += 1
        q.copy_(queries(p, 2, 8, 30 + i))
        k.copy_(torch.randn((2, 2, 128), generator=g0, device="cuda"))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        p.lens = lens.tolist()
        near(out, p, q, [1, 1])


def test_two_calls_at_once_with_workspaces_of_their_own():
    p = Paged([9000], 2, 64, 128, 0, seed=17)
    qs = [queries(p, 1, 8, 40 + i) for i in range(2)]
    outs = [torch.empty_like(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    caches = [p.cache(fp8) for _ in range(2)]
    ws = [fp8.kv_attention_workspace(qs[i], caches[i], 1, 1, 9000) for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            fp8.fp8_kv_attention(qs[i], caches[i], p.table, p.kv_lens, outs[i], max_kv_len=9000, workspace=ws[i],
                                 stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        near(outs[i], p, qs[i], [1])


def test_weights_far_below_the_largest_still_count():
    """One token ahead of 100,000 equal ones by 2^16 to one: together they outweigh it, alone each is 2^-16 of it."""
    n = 100000
    p = Paged([n], 1, 128, 64, 0, seed=18, spread=0.0)
    p.codes["k"].zero_()
    p.scale["k"].fill_(1.0)
    page, slot = divmod(777, 128)
    p.codes["k"][p.table[0, page].long(), 0, slot, 0] = 0x38          # 1.0
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 11.0
    out, st = run(p, q, [1], scale=1.0)
    assert st == 0
    assert math.exp(11.0) < n
    near(out, p, q, [1], scale=1.0)


@pytest.mark.parametrize("group", [8, 16])
def test_many_long_sequences(group):
    """More sequences than a warp has lanes, and many tiles and several units per CTA (8 and 16 rows)."""
    lens = [700 + 97 * (i % 13) for i in range(40)]
    lens[3], lens[35] = 9001, 6400
    check(Paged(lens, 4, 64, 128, 0, seed=19), [1] * 40, group)


@pytest.mark.parametrize("group,dim,fmt", [(8, 128, 0), (16, 64, 1), (7, 128, 1)])
def test_a_few_tokens_over_long_caches(group, dim, fmt):
    """Several row tiles of 16 per sequence, each split over CTAs."""
    check(Paged([20000, 3000, 9, 0], 2, 64, dim, fmt, seed=20), [8, 5, 9, 0], group)
