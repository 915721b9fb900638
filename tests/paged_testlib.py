"""Plain 64-bit restatements of the paged cache and of dense attention over it,
and the error bounds the GPU tests hold the kernels to."""
import math

import torch

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
         "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}


def code_values(kind):
    """Non-negative values of an 8-bit format in code order (no infinities, no NaN)."""
    bits, bias, n = (3, 7, 127) if kind == "e4m3" else (2, 15, 124)
    out = []
    for code in range(n):
        e, f = code >> bits, code & ((1 << bits) - 1)
        out.append(math.ldexp(f, 1 - bias - bits) if e == 0
                   else math.ldexp((1 << bits) + f, e - bias - bits))
    return torch.tensor(out, dtype=torch.float64)


def nearest_code(y, kind):
    """Codes (uint8) of float64 values: nearest, ties to the even code, saturating."""
    grid = code_values(kind)
    a = y.abs()
    up = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    down = (up - 1).clamp(min=0)
    over, under = grid[up] - a, a - grid[down]
    code = torch.where((over < under) | ((over == under) & (up % 2 == 0)), up, down)
    code = torch.where(a >= grid[-1], torch.full_like(code, len(grid) - 1), code)
    sign = torch.signbit(y)
    return (code + 128 * sign).to(torch.uint8)


class Cache:
    """A paged cache and packed rows of its sequences' newest tokens, on the CPU."""

    def __init__(self, seed, q_lens, kv_lens, heads, kv_heads, dim, page, dtype="bf16", cache="same",
                 layout="NHD", spare=3, before=0, behind=0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.dtype, self.cache, self.layout, self.page = g, dtype, cache, layout, page
        self.q_lens, self.kv_lens = list(q_lens), list(kv_lens)
        self.Hq, self.H, self.D = heads, kv_heads, dim
        B = len(q_lens)
        self.T = before + sum(q_lens) + behind
        self.cu = torch.zeros(B + 1, dtype=torch.int32)
        self.cu[1:] = torch.tensor(q_lens, dtype=torch.int32).cumsum(0)
        self.cu += before
        t = TORCH[dtype]
        qkv = torch.randn((self.T, heads + 2 * kv_heads, dim), generator=g).to(t)
        self.qkv = qkv
        self.lens = torch.tensor(kv_lens, dtype=torch.int32)
        used = [-(-n // page) for n in kv_lens]
        self.pages = sum(used) + spare
        width = max(max(used), 1) + 1
        self.table = torch.full((B, width), -7, dtype=torch.int32)
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at: at + n]
            at += n
        shape = ((self.pages, page, kv_heads, dim) if layout == "NHD"
                 else (self.pages, kv_heads, page, dim))
        k, v = (torch.randn(shape, generator=g) for _ in range(2))
        self.scale_k = self.scale_v = None
        if cache == "same":
            self.k, self.v = k.to(t), v.to(t)
        else:
            self.scale_k = (0.5 + torch.rand(kv_heads, generator=g)) * 4 / LARGEST[cache]
            self.scale_v = (0.5 + torch.rand(kv_heads, generator=g)) * 4 / LARGEST[cache]
            top = LARGEST[cache]
            by = (1, 1, kv_heads, 1) if layout == "NHD" else (1, kv_heads, 1, 1)
            self.k = (k / self.scale_k.view(by)).clamp(-top, top).to(TORCH[cache])
            self.v = (v / self.scale_v.view(by)).clamp(-top, top).to(TORCH[cache])

    def split(self, qkv):
        return qkv[:, : self.Hq], qkv[:, self.Hq: self.Hq + self.H], qkv[:, self.Hq + self.H:]

    def cells(self, b):
        """(page, place) of every token of sequence b; page -1 where it has none."""
        j = torch.arange(self.kv_lens[b])
        page = self.table[b][j // self.page].long()
        page = torch.where((page >= 0) & (page < self.pages), page, torch.full_like(page, -1))
        return page, j % self.page

    def values(self, pools, scale, b):
        """Float64 (tokens, kv heads, dim) of sequence b, and which tokens are there."""
        page, place = self.cells(b)
        p = pools.transpose(1, 2) if self.layout == "HND" else pools
        if self.cache != "same":
            x = p.float()[page.clamp(min=0), place].double()
            if scale is not None:
                x = x * scale.double().view(1, -1, 1)
        else:
            x = p[page.clamp(min=0), place].double()
        return x, page >= 0

    def poison(self):
        """NaN and infinity in every place that holds no token."""
        free = torch.ones(self.pages, self.page, dtype=torch.bool)
        for b in range(len(self.kv_lens)):
            page, place = self.cells(b)
            free[page[page >= 0], place[page >= 0]] = False
        for x in (self.k, self.v):
            y = x.view(torch.uint8) if self.cache != "same" else x
            y = y.transpose(1, 2) if self.layout == "HND" else y
            if self.cache == "same":
                y[free] = float("nan")
                y[free, 0] = float("inf")
            else:
                y[free] = 0x7F          # NaN in both formats
        return self

    def to(self, dev):
        """Device copies of what the calls take."""
        d = {n: getattr(self, n) for n in ("qkv", "cu", "table", "lens", "k", "v", "scale_k", "scale_v")}
        return {n: None if x is None else x.to(dev) for n, x in d.items()}


def attend(q, k, v, there, causal, scale):
    """One sequence in float64: q (n, Hq, D), k, v (L, H, D), there (L,): which
    keys exist.  Returns out, lse, A = sum_j p_j |v_j|, and S = the largest
    scale * sum_d |q_d k_d| of each row."""
    n, Hq, D = q.shape
    L, H = k.shape[:2]
    G = Hq // H
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    seen = there[None, :].expand(n, L)
    if causal:
        seen = seen & (torch.arange(L)[None, :] <= torch.arange(n)[:, None] + L - n)
    x = torch.einsum("ihd,jhd->hij", q, k) * scale
    x = torch.where(seen[None], x, torch.full_like(x, -math.inf))
    if L == 0:
        z = torch.zeros(n, Hq, D, dtype=torch.float64)
        return z, torch.full((n, Hq), -math.inf, dtype=torch.float64), z, z[..., 0]
    m = x.amax(-1, keepdim=True).clamp(min=-1e300)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1).T
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    # absent values count as zero (they may hold anything)
    v = torch.where(there[:, None, None], v, torch.zeros_like(v))
    out = torch.einsum("hij,jhd->ihd", p, v)
    A = torch.einsum("hij,jhd->ihd", p, v.abs())
    S = torch.einsum("ihd,jhd->hij", q.abs(), torch.where(there[:, None, None], k, torch.zeros_like(k)).abs())
    return out, lse, A, (S * abs(scale)).amax(-1).T


def check(got, lse, ref, dtype, keys, where=""):
    """out and lse of one sequence against attend()'s.

    Half a step h of the output type; the weights p are rounded to 16 bits
    before the second product (at most h of each: h A in all); scores are fp32
    sums of D products and a few fp32 operations (an error of at most
    (D + 8) 2^-24 S of the exponent, which moves p and the sum of p), the sums
    over the keys add at most keys * 2^-24, exp2 2^-21."""
    out, l, A, S = ref
    D = out.shape[-1]
    h = torch.finfo(TORCH[dtype]).eps / 2
    c = (2 * (D + 8) * S[..., None] + 2 * keys) * 2.0 ** -24 + 2.0 ** -20
    tol = h * out.abs() + (h + c) * (1 + h) * A + 1e-30
    if dtype == "f16":
        tol = tol + 2.0 ** -25           # half a step of fp16's smallest numbers
    err = (got.double() - out).abs()
    assert torch.isfinite(got.double()).all(), f"{where}: not finite"
    worst = (err / tol).max() if err.numel() else torch.tensor(0.0)
    assert worst <= 1.0, f"{where}: {float(worst):.3g} times the bound"
    none = torch.isneginf(l)
    assert torch.all(got[none] == 0) and not torch.signbit(got[none].float()).any(), where
    if lse is not None:
        assert torch.equal(torch.isneginf(lse), none), f"{where}: rows without a key"
        lt = (c[..., 0] + 2.0 ** -21 + l.abs() * 2.0 ** -22)[~none]
        assert torch.all((lse.double() - l)[~none].abs() <= lt), f"{where}: lse"
