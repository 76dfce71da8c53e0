"""A paged FP8 KV cache built in plain torch for the tests, and attention over it in 64 bits."""
import math

import torch

DT = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}
TOP = {0: 448.0, 1: 57344.0}
NAN_CODE = {0: 0x7F, 1: 0x7E}


def page_scale(amax, fmt):
    """Least power of two s with max(amax, 1e-12) <= F_max s."""
    m, e = torch.frexp(amax.double().clamp(min=1e-12) / TOP[fmt])       # exact mantissas: F_max = 1.75 * 2^n
    s = torch.ldexp(torch.ones_like(m), e)
    return torch.where(amax.double().clamp(min=1e-12) <= TOP[fmt] * s / 2, s / 2, s)


class Paged:
    """Pages in random order, every slot and page that holds no token filled with NaN codes, every page-table
    entry past a sequence's length set to a page that does not exist."""

    def __init__(self, kv_lens, heads, page, dim, fmt, seed=0, spread=0.5, spare=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.fmt, self.page, self.dim, self.heads = g, fmt, page, dim, heads
        self.lens = list(kv_lens)
        need = [-(-n // page) for n in self.lens]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        width = max(need + [1]) + 2
        self.table = torch.full((len(self.lens), width), -7, dtype=torch.int32, device="cuda")
        used = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[used:used + n]
            used += n
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.codes, self.scale = {}, {}
        for name in "kv":
            x = torch.randn((pages, heads, page, dim), generator=g, device="cuda")
            x *= torch.exp(spread * torch.randn((pages, heads, 1, 1), generator=g, device="cuda"))
            s = page_scale(x.abs().amax((2, 3)), fmt).float()
            c = (x / s[:, :, None, None]).to(DT[fmt]).view(torch.uint8)
            live = torch.zeros((pages, page), dtype=torch.bool, device="cuda")
            for b, n in enumerate(self.lens):
                for i in range(need[b]):
                    live[int(self.table[b, i]), :min(page, n - i * page)] = True
            c = torch.where(live[:, None, :, None], c, torch.full_like(c, NAN_CODE[fmt]))
            self.codes[name], self.scale[name] = c, s

    def cache(self, fp8):
        return fp8.KVCache(self.codes["k"], self.codes["v"], self.scale["k"], self.scale["v"], self.fmt)

    def values(self, name, b, n):
        """[heads, n, dim] in 64 bits: the first n tokens of sequence b."""
        pages = self.table[b, :-(-n // self.page)].long()
        x = self.codes[name][pages].view(DT[self.fmt]).double() * self.scale[name][pages].double()[:, :, None, None]
        return x.transpose(0, 1).reshape(self.heads, -1, self.dim)[:, :n]


def attention64(paged, q, cu, scale, lens=None):
    """(out, limit of the error) of the tokens of every sequence, in 64 bits.

    The kernel rounds a weight to fp16 (2^-11) and accumulates scores in fp32 over dim
    terms; a score's error d (in units of 1) is at most 2^-23 (dim + 8) of the sum of its
    terms' magnitudes, and a few fp32 steps of the score itself (the exponent's argument); a
    weight is then off by a factor exp(2 d) at most, against the sum as well.  The last
    rounding to bf16 is half a step, 2^-8."""
    outs, lims = [], []
    lens = paged.lens if lens is None else lens
    for b, n in enumerate(lens):
        rows = q[cu[b]:cu[b + 1]].double()
        new, group = rows.shape[0], q.shape[1] // paged.heads
        if new == 0:
            continue
        o, lim = torch.zeros_like(rows), torch.zeros_like(rows)
        if n > 0:
            k, v = paged.values("k", b, n), paged.values("v", b, n)
            see = torch.arange(n, device="cuda")[None, :] <= n - new + torch.arange(new, device="cuda")[:, None]
            for h in range(q.shape[1]):
                z = rows[:, h] @ k[h // group].T * scale
                mag = rows[:, h].abs() @ k[h // group].abs().T * abs(scale)
                z = z.masked_fill(~see, -math.inf)
                d = (2.0 ** -23 * (paged.dim + 8) * mag + 2.0 ** -21 * (z.abs() + 16)).masked_fill(~see, 0.0)
                p = torch.softmax(z, 1).nan_to_num(0.0)
                seen_d = torch.where(p > 2.0 ** -60, d, torch.zeros_like(d)).amax(1, keepdim=True)
                o[:, h] = p @ v[h // group]
                lim[:, h] = 2.0 ** -8 * o[:, h].abs() + (2.0 ** -11 + 2 * seen_d * torch.exp(2 * seen_d)) * (p @ v[h // group].abs()) \
                    + 2.0 ** -30 * v[h // group].abs().amax(0)
        outs.append(o)
        lims.append(lim)
    if not outs:
        e = torch.zeros((0, q.shape[1], q.shape[2]), dtype=torch.float64, device="cuda")
        return e, e
    return torch.cat(outs), torch.cat(lims)


def starts(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cu
