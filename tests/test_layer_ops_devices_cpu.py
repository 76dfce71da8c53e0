"""The bindings' guard against tensors that are not on the current device, argument by argument: a call
whose other tensors all claim to be there is refused for the one that does not, before the library
sees a pointer.  (The library is a stand-in that counts calls; no kernel can run here.)"""
import pytest
import torch

from fp8_dynamic_scaled_b200 import binding as b

BF, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32


class Claims(torch.Tensor):
    """A host tensor that says it is on device `place` (-1: the host)."""
    place = 0

    def get_device(self):
        return self.place

    @property
    def is_cuda(self):
        return self.place >= 0


def here(*shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(Claims)


@pytest.fixture
def calls(monkeypatch):
    seen = []
    monkeypatch.setattr(b.torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(b.torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    for name in ("fp8_rmsnorm_quantize", "fp8_scaled_gemm_act", "fp8_linear_forward_act", "fp8_kv_append",
                 "fp8_kv_attention"):
        monkeypatch.setattr(b._lib, name, lambda *a, name=name: seen.append(name) or 0)
    return seen


def norm(t):
    b.fp8_rmsnorm_quantize(t["x"], t["weight"], 1e-5, 0, b.FP8_SCALE_TENSOR, t["q"], t["scale"], residual=t["residual"],
                           sum_out=t["sum_out"], y=t["y"], amax=t["amax"], dev_status=t["dev_status"], stream=0)


def gemm(t):
    b.fp8_scaled_gemm_act(t["a"], t["a_scale"], 1, 0, t["b"], t["b_scale"], 1, 0, t["y"], bias=t["bias"], activation=1,
                          residual=t["residual"], amax=t["amax"], yq=t["yq"], yq_scale=t["yq_scale"],
                          dev_status=t["dev_status"], stream=0)


def linear(t):
    b.fp8_linear_forward_act(t["x"], 0, b.FP8_SCALE_DELAYED, t["w"], t["w_scale"], 1, 0, t["y"], t["workspace"],
                             hist=t["hist"], bias=t["bias"], activation=1, residual=t["residual"], amax=t["amax"],
                             yq=t["yq"], yq_scale=t["yq_scale"], dev_status=t["dev_status"], stream=0)


def append(t):
    b.fp8_kv_append(t["k"], t["v"], t["cache"], t["page_table"], t["kv_lens"], cu_q=t["cu_q"], max_q_len=2,
                    dev_status=t["dev_status"], stream=0)


def attend(t):
    b.fp8_kv_attention(t["q"], t["cache"], t["page_table"], t["kv_lens"], t["out"], max_kv_len=16, cu_q=t["cu_q"],
                       max_q_len=2, workspace=t["workspace"], dev_status=t["dev_status"], stream=0)


def epilogue():
    return dict(y=here(4, 8, dtype=BF), bias=here(8, dtype=BF), residual=here(4, 8, dtype=BF), amax=here(1, dtype=F32),
                yq=here(4, 8, dtype=U8), yq_scale=here(1, dtype=F32), dev_status=here(1, dtype=I32))


def paged():
    return dict(page_table=here(2, 3, dtype=I32), kv_lens=here(2, dtype=I32), cu_q=here(3, dtype=I32),
                dev_status=here(1, dtype=I32))


def cache():
    codes = [here(4, 2, 16, 64, dtype=U8) for _ in range(2)]
    return b.KVCache(*codes, *(here(4, 2, dtype=F32) for _ in range(2)))


CALLS = {
    "norm": (norm, lambda: dict(x=here(4, 64, dtype=BF), weight=here(64, dtype=BF), q=here(4, 64, dtype=U8),
                                scale=here(4, dtype=F32), residual=here(4, 64, dtype=BF), sum_out=here(4, 64, dtype=BF),
                                y=here(4, 64, dtype=BF), amax=here(1, dtype=F32), dev_status=here(1, dtype=I32))),
    "gemm": (gemm, lambda: epilogue() | dict(a=here(4, 32, dtype=U8), a_scale=here(4, dtype=F32), b=here(8, 32, dtype=U8),
                                             b_scale=here(8, dtype=F32))),
    "linear": (linear, lambda: epilogue() | dict(x=here(4, 32, dtype=BF), w=here(8, 32, dtype=U8),
                                                 w_scale=here(8, dtype=F32), workspace=here(4096, dtype=U8))),
    "append": (append, lambda: paged() | dict(k=here(3, 2, 64, dtype=BF), v=here(3, 2, 64, dtype=BF))),
    "attend": (attend, lambda: paged() | dict(q=here(3, 4, 64, dtype=BF), out=here(3, 4, 64, dtype=BF),
                                              workspace=here(4096, dtype=U8))),
}


def history(off=None, place=-1):
    h = b.History(4, device="cpu")
    for n in ("ring", "pending", "ticket"):
        t = getattr(h, n).as_subclass(Claims)
        t.place = place if n == off else 0
        setattr(h, n, t)
    return h


@pytest.mark.parametrize("place", [-1, 1])
@pytest.mark.parametrize("op", sorted(CALLS))
def test_each_tensor_is_guarded(op, place, calls):
    call, make = CALLS[op]
    extra = dict(cache=cache(), hist=history())
    call(make() | extra)
    assert len(calls) == 1
    for name in make():
        t = make() | extra
        t[name].place = place
        with pytest.raises(ValueError):
            call(t)
    assert len(calls) == 1
    if op == "linear":
        for name in ("ring", "pending", "ticket"):
            with pytest.raises(ValueError):
                call(make() | extra | dict(hist=history(name, place)))
    if op in ("append", "attend"):
        c = cache()
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            t.place = place
        with pytest.raises(ValueError):
            call(make() | dict(cache=c))
    assert len(calls) == 1


BAD_SHAPES = [dict(y=(4, 7)), dict(y=(3, 8)), dict(y=(8, 4)), dict(yq=(4, 9)), dict(yq=(2, 8)), dict(residual=(4, 7)),
              dict(bias=(7,))]


@pytest.mark.parametrize("op", ["gemm", "linear"])
def test_shapes_of_the_activation_gemm(op, calls):
    """What a kernel would read or write past the end of: outputs that are not [M, N], operands of another K, scale
    buffers that are too short; and views whose elements are not where the call takes them to be."""
    call, make = CALLS[op]
    extra = dict(hist=history())
    wt, ws = ("b", "b_scale") if op == "gemm" else ("w", "w_scale")
    bad = [{n: here(*shape, dtype=make()[n].dtype)} for d in BAD_SHAPES for n, shape in d.items()]
    bad += [{wt: here(8, 48, dtype=U8)}, {wt: here(8, 64, dtype=U8)[:, :32]}, {wt: here(256, dtype=U8)},
            {ws: here(7, dtype=F32)}, {ws: here(8, dtype=U8)}, {ws: here(8, 2, dtype=F32)[:, 0]},
            {"y": here(4, 16, dtype=BF)[:, ::2]}, {"yq": here(8, 4, dtype=U8).t()}, {"bias": here(16, dtype=BF)[::2]},
            {"amax": here(0, dtype=F32)}, {"amax": here(1, dtype=BF)}, {"yq_scale": here(1, dtype=BF)}]
    if op == "gemm":
        bad += [dict(a=here(4, 64, dtype=U8)[:, :32]), dict(a=here(128, dtype=U8)), dict(a_scale=here(3, dtype=F32))]
    else:
        bad += [dict(x=here(4, 64, dtype=BF)[:, ::2]), dict(x=here(128, dtype=BF)), dict(x=here(32, 4, dtype=BF).t())]
    for kw in bad:
        with pytest.raises(TypeError):
            call(make() | extra | kw)
    assert not calls
    good = [dict(y=None), dict(y=here(4, 24, dtype=BF)[:, 8:16]), dict(yq=here(4, 11, dtype=U8)[:, 3:]), dict(yq=None)]
    for kw in good:
        call(make() | extra | kw)
    assert len(calls) == len(good)


def test_scale_buffers_of_every_mode(calls):
    M, N, K = 4, 130, 256
    t = dict(y=here(M, N, dtype=BF), a=here(M, K, dtype=U8), b=here(N, K, dtype=U8))

    def run(am, sa, bm, sb):
        b.fp8_scaled_gemm_act(t["a"], sa, am, 0, t["b"], sb, bm, 0, t["y"], activation=1, stream=0)
    B1, B128, MX = b.FP8_SCALE_BLOCK_1x128, b.FP8_SCALE_BLOCK_128x128, b.FP8_SCALE_MX32
    run(B1, here(4, 2, dtype=F32), B128, here(2, 2, dtype=F32))
    run(MX, here(4, 8, dtype=U8), MX, here(N, 8, dtype=U8).view(torch.float8_e8m0fnu))
    run(0, here(1, dtype=F32), 5, here(1, dtype=F32))
    assert len(calls) == 3
    for args in ((B1, here(4, 2, dtype=F32), B128, here(1, 2, dtype=F32)), (B1, here(4, 1, dtype=F32), B128, here(2, 2, dtype=F32)),
                 (MX, here(4, 8, dtype=U8), MX, here(N, 7, dtype=U8)), (MX, here(4, 8, dtype=F32), MX, here(N, 8, dtype=U8)),
                 (0, here(0, dtype=F32), 1, here(N, dtype=F32))):
        with pytest.raises(TypeError):
            run(*args)
    assert len(calls) == 3


def test_attention_into_its_own_queries_is_refused(calls):
    call, make = CALLS["attend"]
    t = make() | dict(cache=cache())
    with pytest.raises(ValueError):
        call(t | dict(out=t["q"]))
    with pytest.raises(ValueError):
        call(t | dict(out=t["q"].view(3, 4, 64)))
    none = here(0, 4, 64, dtype=BF)
    call(t | dict(q=none, out=none))
    assert len(calls) == 1


def test_a_cache_is_on_one_device():
    for i in range(4):
        t = [here(4, 2, 16, 64, dtype=U8), here(4, 2, 16, 64, dtype=U8), here(4, 2, dtype=F32), here(4, 2, dtype=F32)]
        t[i].place = -1
        with pytest.raises(ValueError):
            b.KVCache(*t)


def test_host_tensors_are_refused_before_cuda_is_up(monkeypatch):
    monkeypatch.setattr(b.torch.cuda, "is_initialized", lambda: False)
    for op, (call, make) in CALLS.items():
        t = make() | dict(cache=cache(), hist=history())
        for x in make():
            t[x].place = -1
        with pytest.raises(ValueError):
            call(t)
