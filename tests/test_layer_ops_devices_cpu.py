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
