"""fp8_kv_append against its definition in 64 bits: scales and codes bit for bit (a bf16 value over a
power of two is exact, and each code is one rounding of it), everything else left as it was."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import fp8_dynamic_scaled_b200.binding as fp8  # noqa: E402
from kv_util import DT, TOP, Paged, page_scale, starts  # noqa: E402


def encode(x, fmt):
    return x.clamp(-TOP[fmt], TOP[fmt]).float().to(DT[fmt]).view(torch.uint8)


def expected(paged, x, name, new, lens):
    """(codes, scales) after the call, from the definition."""
    codes, scale, P, fmt = paged.codes[name].clone(), paged.scale[name].clone(), paged.page, paged.fmt
    cu = starts(new)
    for b, n in enumerate(lens):
        at, t = n - new[b], cu[b]
        while at < n:
            page, lo = int(paged.table[b, at // P]), at % P
            cnt = min(P - lo, n - at)
            part = x[t:t + cnt].double().transpose(0, 1)
            s = page_scale(part.abs().amax((1, 2)), fmt)
            if lo:
                old = scale[page].double()
                s = torch.maximum(s, old)
                held = codes[page, :, :lo].contiguous().view(DT[fmt]).double() * (old / s)[:, None, None]
                codes[page, :, :lo] = encode(held, fmt)
            scale[page] = s.float()
            codes[page, :, lo:lo + cnt] = encode(part / s[:, None, None], fmt)
            at, t = at + cnt, t + cnt
    return codes, scale


def run(paged, k, v, new, lens, use_cu=True, max_q=None, extra=None):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor(starts(new), dtype=torch.int32, device="cuda") if use_cu else None
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    fp8.fp8_kv_append(k, v, paged.cache(fp8), paged.table, kv, cu_q=cu, max_q_len=max(new + [1]) if max_q is None else max_q,
                      dev_status=st)
    torch.cuda.synchronize()
    return int(st.item())


def new_tokens(paged, T, seed, std=1.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = paged.heads * paged.dim
    rows = (torch.randn((T, 2 * w + pad), generator=g, device="cuda") * std).bfloat16()
    return rows[:, :w].view(T, paged.heads, paged.dim), rows[:, w:2 * w].view(T, paged.heads, paged.dim)


def check(paged, new, lens, seed=1, std=1.0, **kw):
    k, v = new_tokens(paged, sum(new), seed, std, pad=8)
    want = {n: expected(paged, x, n, new, lens) for n, x in (("k", k), ("v", v))}
    assert run(paged, k, v, new, lens, **kw) == 0
    for n in "kv":
        assert torch.equal(paged.scale[n], want[n][1]), n
        assert torch.equal(paged.codes[n], want[n][0]), n


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("heads", [1, 3, 8])
def test_ragged_calls(page, dim, heads, fmt):
    lens = [1, page, page + 1, 5 * page - 3, 7, 2 * page, 300]
    new = [1, page, 2, 3 * page + 5, 0, 1, 300]
    check(Paged(lens, heads, page, dim, fmt, seed=page + dim), new, lens)


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [2, 5, 0, 8], [1, 0, 0, 0]])
def test_decode_steps_and_a_page_that_fills_up(new):
    lens = [20, 33, 64, 8]
    p = Paged([64] * 4, 2, 32, 128, 0, seed=5)
    for step in range(12):
        check(p, new, [min(64, n + step * max(new)) for n in lens], seed=step, std=2.0 ** (step - 4))


def test_no_cu_q_is_one_token_each():
    lens = [5, 16, 17, 100]
    p = Paged(lens, 4, 16, 64, 1, seed=6)
    check(p, [1] * 4, lens, use_cu=False)


def test_scale_grows_and_codes_move_into_subnormals():
    for fmt in (0, 1):
        p = Paged([40], 2, 64, 128, fmt, seed=7, spread=0.0)
        for step, std in enumerate((1.0, 1.0, 300.0, 0.01, 1e4, 1e-5, 1e7)):
            check(p, [2], [28 + 2 * step], seed=step, std=std)


def test_extreme_values():
    """Zeros, subnormals, and bf16's largest."""
    for fmt in (0, 1):
        p = Paged([4, 4, 4, 4], 1, 16, 64, fmt, seed=8)
        k, v = new_tokens(p, 16, 3)
        k[0:4] = 0
        v[0:4] = -0.0
        k[4:8] *= 2.0 ** -130
        k[8:12] = torch.finfo(torch.bfloat16).max
        v[12:16] = torch.tensor(1.75, dtype=torch.bfloat16)
        new, lens = [4] * 4, [4] * 4
        want = {n: expected(p, x, n, new, lens) for n, x in (("k", k), ("v", v))}
        assert run(p, k, v, new, lens) == 0
        for n in "kv":
            assert torch.equal(p.scale[n], want[n][1]) and torch.equal(p.codes[n], want[n][0])


def test_rows_behind_the_last_sequence_are_not_read():
    lens = [9, 30]
    p = Paged(lens, 2, 16, 64, 0, seed=9)
    k, v = new_tokens(p, 20, 4)
    k[8:] = float("nan")
    new = [3, 5]
    want = {n: expected(p, x, n, new, lens) for n, x in (("k", k), ("v", v))}
    assert run(p, k, v, new, lens) == 0
    for n in "kv":
        assert torch.equal(p.scale[n], want[n][1]) and torch.equal(p.codes[n], want[n][0])


def test_nonfinite_is_reported():
    for bad in (float("nan"), float("inf")):
        p = Paged([9], 2, 16, 64, 0, seed=10)
        k, v = new_tokens(p, 3, 5)
        v[1, 1, 5] = bad
        assert run(p, k, v, [3], [9]) == fp8.FP8_ERR_NONFINITE


@pytest.mark.parametrize("what", ["page", "negative_page", "cu", "cu_end", "max_q", "short", "long", "negative"])
def test_bad_device_arguments_touch_nothing(what):
    """What only the device sees: the sequence (or page) is reported and left alone; the other is written."""
    p = Paged([40, 20], 2, 16, 64, 0, seed=11)
    k, v = new_tokens(p, 8, 6)
    cu, lens, max_q = [0, 4, 8], [40, 20], 4
    if what == "page":
        p.table[1, 1] = p.codes["k"].shape[0]
    elif what == "negative_page":
        p.table[1, 1] = -1
    elif what == "cu":
        cu = [0, 4, 3]
    elif what == "cu_end":
        cu = [0, 4, 9]
    elif what == "max_q":
        cu, lens = [0, 2, 8], [40, 20]
    elif what == "short":
        lens = [40, 3]
    elif what == "long":
        lens = [40, p.table.shape[1] * 16 + 1]
    else:
        lens = [40, -1]
    first = cu[1]
    want = {n: expected(p, x[:first], n, [first, 0], [40, 20]) for n, x in (("k", k), ("v", v))}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp8.fp8_kv_append(k, v, p.cache(fp8), p.table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                      cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_q_len=max_q, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == fp8.FP8_ERR_INVALID_ARG
    for n in "kv":
        assert torch.equal(p.scale[n], want[n][1]) and torch.equal(p.codes[n], want[n][0])


def test_nothing_to_do():
    p = Paged([5], 2, 16, 64, 0, seed=12)
    before = {n: p.codes[n].clone() for n in "kv"}
    k, v = new_tokens(p, 1, 7)
    assert run(p, k[:0], v[:0], [0], [5]) == 0
    assert all(torch.equal(p.codes[n], before[n]) for n in "kv")


def test_graph_replay_over_a_growing_sequence():
    """One captured decode step: the lengths live on the device."""
    p = Paged([64, 64], 2, 32, 128, 0, seed=13)
    k, v = new_tokens(p, 2, 8)
    k, v = k.clone(), v.clone()
    lens = torch.tensor([10, 31], dtype=torch.int32, device="cuda")
    cache = p.cache(fp8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp8.fp8_kv_append(k, v, cache, p.table, lens, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side, capture_error_mode="thread_local"):
        fp8.fp8_kv_append(k, v, cache, p.table, lens, stream=side)
    for step in range(4):
        a, c = new_tokens(p, 2, 20 + step, std=2.0 ** step)
        k.copy_(a)
        v.copy_(c)
        lens += 1
        now = lens.tolist()
        want = {n: expected(p, x, n, [1, 1], now) for n, x in (("k", k), ("v", v))}
        g.replay()
        torch.cuda.synchronize()
        for n in "kv":
            assert torch.equal(p.scale[n], want[n][1]) and torch.equal(p.codes[n], want[n][0])
