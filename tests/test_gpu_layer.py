"""The operators together, as a decoder layer runs them around the FP8 linears:

    norm (residual added) -> QKV projection -> append to the cache -> attention -> output projection + residual
    -> norm -> up projection with GELU, FP8 output -> down projection + residual

for prompt chunks and then decode steps of a ragged batch, the decode step as a captured graph whose
lengths grow on the device.  Every stage is compared with its definition in 64 bits on what the
stage before gave it (each stage's tolerance is stated with its own tests)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)
import fp8_dynamic_scaled_b200.binding as fp8  # noqa: E402
import test_gpu_gemm_act as ga  # noqa: E402
import test_gpu_rmsnorm as rn  # noqa: E402
from kv_util import Paged, starts  # noqa: E402
from test_gpu_kv_append import expected  # noqa: E402
from test_gpu_kv_attention import near  # noqa: E402

E4, R = fp8.FP8_E4M3, fp8.FP8_SCALE_ROW
HID, HEADS, KV, DIM, FF, EPS = 512, 8, 2, 64, 1024, 1e-5


class Layer:
    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.w, self.s = {}, {}
        for name, n, k in (("qkv", (HEADS + 2 * KV) * DIM, HID), ("o", HID, HEADS * DIM), ("up", FF, HID), ("down", HID, FF)):
            w = (torch.randn((n, k), generator=g, device="cuda") * k ** -0.5).bfloat16()
            self.w[name], self.s[name], _ = fp8.empty_quant_outputs(n, k, R)
            fp8.fp8_quantize(w, E4, R, self.w[name], self.s[name])
        self.n1, self.n2 = ((1 + 0.1 * torch.randn(HID, generator=g, device="cuda")).bfloat16() for _ in range(2))
        self.bias = (0.1 * torch.randn(FF, generator=g, device="cuda")).bfloat16()
        self.up_scale = torch.tensor([2.0 ** -6], device="cuda")

    def buffers(self, T):
        def bf(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device="cuda")

        def codes(n):
            return torch.empty((T, n), dtype=torch.uint8, device="cuda")
        return dict(h=bf(T, HID), q1=codes(HID), s1=torch.empty(T, device="cuda"), qkv=bf(T, (HEADS + 2 * KV) * DIM),
                    att=bf(T, HEADS, DIM), h2=bf(T, HID), q2=codes(HID), s2=torch.empty(T, device="cuda"), ff=codes(FF),
                    out=bf(T, HID), st=torch.zeros(1, dtype=torch.int32, device="cuda"))

    def run(self, x, res, b, cache, table, lens, cu, max_q, max_kv, attn_ws, lin_ws, stream=None):
        T = x.shape[0]
        kw = dict(dev_status=b["st"], stream=stream)
        fp8.fp8_rmsnorm_quantize(x, self.n1, EPS, E4, R, b["q1"], b["s1"], residual=res, sum_out=b["h"], **kw)
        fp8.fp8_scaled_gemm(b["q1"], b["s1"], R, E4, self.w["qkv"], self.s["qkv"], R, E4, b["qkv"], **kw)
        q, k, v = (b["qkv"][:, lo * DIM:hi * DIM].view(T, hi - lo, DIM)
                   for lo, hi in ((0, HEADS), (HEADS, HEADS + KV), (HEADS + KV, HEADS + 2 * KV)))
        fp8.fp8_kv_append(k, v, cache, table, lens, cu_q=cu, max_q_len=max_q, **kw)
        fp8.fp8_kv_attention(q, cache, table, lens, b["att"], cu_q=cu, max_q_len=max_q, max_kv_len=max_kv,
                             workspace=attn_ws, **kw)
        fp8.fp8_linear_forward_act(b["att"].view(T, HEADS * DIM), E4, R, self.w["o"], self.s["o"], R, E4, b["h2"], lin_ws,
                                   residual=b["h"], **kw)
        fp8.fp8_rmsnorm_quantize(b["h2"], self.n2, EPS, E4, R, b["q2"], b["s2"], **kw)
        fp8.fp8_scaled_gemm_act(b["q2"], b["s2"], R, E4, self.w["up"], self.s["up"], R, E4, None, bias=self.bias,
                                activation=fp8.FP8_ACT_GELU, yq=b["ff"], yq_scale=self.up_scale, **kw)
        fp8.fp8_scaled_gemm_act(b["ff"], self.up_scale, fp8.FP8_SCALE_TENSOR, E4, self.w["down"], self.s["down"], R, E4,
                                b["out"], residual=b["h2"], **kw)

    def product(self, q, s, name):
        a = q.view(torch.float8_e4m3fn).double() * s.double().view(-1, 1)
        w = self.w[name].view(torch.float8_e4m3fn).double() * self.s[name].double()[:, None]
        return a @ w.T, a.abs() @ w.abs().T

    def check(self, x, res, b, paged, before, new):
        assert int(b["st"].item()) == 0
        T = x.shape[0]
        rn.check(x, self.n1, E4, R, b["q1"], b["s1"], residual=res, eps=EPS)
        assert torch.equal(b["h"], (x.float() + res.float()).bfloat16())
        ref, bound = self.product(b["q1"], b["s1"], "qkv")
        ga.near(b["qkv"], *ga.expect(ref, bound, None, ga.NONE, None), what="qkv")
        for name, lo in (("k", HEADS), ("v", HEADS + KV)):
            part = b["qkv"][:, lo * DIM:(lo + KV) * DIM].view(T, KV, DIM)
            codes, scale = expected(before, part, name, new, paged.lens)
            assert torch.equal(paged.codes[name], codes) and torch.equal(paged.scale[name], scale)
        near(b["att"], paged, b["qkv"][:, :HEADS * DIM].view(T, HEADS, DIM), new)
        aq, s, _ = fp8.empty_quant_outputs(T, HEADS * DIM, R)
        fp8.fp8_quantize(b["att"].view(T, HEADS * DIM), E4, R, aq, s)
        ref, bound = self.product(aq, s, "o")
        ga.near(b["h2"], *ga.expect(ref, bound, None, ga.NONE, b["h"]), what="output projection")
        rn.check(b["h2"], self.n2, E4, R, b["q2"], b["s2"], eps=EPS)
        ref, bound = self.product(b["q2"], b["s2"], "up")
        y, lim = ga.expect(ref, bound, self.bias, ga.GELU, None)
        lo, hi = (rn.encode((y + d) / self.up_scale.double(), E4) for d in (-lim, lim))
        got = b["ff"].view(torch.float8_e4m3fn).float()
        assert bool(((got >= lo) & (got <= hi)).all())
        ref, bound = self.product(b["ff"], self.up_scale.expand(T), "down")
        ga.near(b["out"], *ga.expect(ref, bound, None, ga.NONE, b["h2"]), what="down projection")


def snapshot(paged):
    copy = Paged.__new__(Paged)
    copy.__dict__.update(paged.__dict__)
    copy.codes = {n: paged.codes[n].clone() for n in "kv"}
    copy.scale = {n: paged.scale[n].clone() for n in "kv"}
    return copy


def test_prompt_chunks_then_decode_steps():
    layer = Layer(1)
    new, lens = [40, 1, 130], [40, 70, 130]
    paged = Paged([n + 10 for n in lens], KV, 32, DIM, E4, seed=2)       # pages for ten more tokens each
    paged.lens = list(lens)
    g = torch.Generator(device="cuda").manual_seed(3)

    def tokens(T):
        return (torch.randn((T, HID), generator=g, device="cuda").bfloat16() for _ in range(2))
    # ---- the chunks
    T = sum(new)
    x, res = tokens(T)
    b = layer.buffers(T)
    cache, kv = paged.cache(fp8), torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor(starts(new), dtype=torch.int32, device="cuda")
    before = snapshot(paged)
    ws = fp8.kv_attention_workspace(b["att"], cache, 3, 130, 150)
    layer.run(x, res, b, cache, paged.table, kv, cu, 130, 150, ws, fp8.workspace_for(2, T, HID, HEADS * DIM, R))
    torch.cuda.synchronize()
    layer.check(x, res, b, paged, before, new)
    # ---- decode steps: one graph, the lengths on the device
    x, res = tokens(3)
    b = layer.buffers(3)
    ws, lws = fp8.kv_attention_workspace(b["att"], cache, 3, 1, 150), fp8.workspace_for(2, 3, HID, HEADS * DIM, R)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        layer.run(x, res, b, cache, paged.table, kv, None, 1, 150, ws, lws, stream=side)
    kv += 1
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side, capture_error_mode="thread_local"):
        step()
    for i in range(3):
        for t, fresh in zip((x, res), tokens(3)):
            t.copy_(fresh)
        kv += 1
        paged.lens = kv.tolist()
        before = snapshot(paged)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        layer.check(x, res, b, paged, before, [1, 1, 1])
