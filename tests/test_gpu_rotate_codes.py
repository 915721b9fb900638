"""8-bit codes of rotated keys on the GPU: the nearest to the exact quotient, on inputs made
to lie next to borders between two codes."""
import math

import pytest
import torch

import sparse_attention_serving_sfa_gb300 as sfa
from tests import paged_testlib as P
from tests import parts_testlib as X
from tests.test_gpu_paged import raw

pytestmark = pytest.mark.gpu

H, D = 16, 64


@pytest.fixture(scope="module", autouse=True)
def built():
    sfa.build()
    sfa.load()


def frequencies(r):
    return (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float()


def turn(x, y, cos, sin):
    return x * cos - y * sin, x * sin + y * cos


def angles(pos, freq):
    """cos and sin, float64 (tokens, 1, pairs): the product is exact (29 + 24 bits)."""
    assert max(pos) < 1 << 29
    a = [[int(p) * float(f) for f in freq] for p in pos]
    return tuple(torch.tensor([[f(v) for v in row] for row in a], dtype=torch.float64)[:, None] for f in (math.cos, math.sin))


def made(dtype, kind, pos, freq, mag, seed):
    """Pairs (x, y), float64 (tokens, heads, pairs) that `dtype` holds, and a scale for each
    head.  One element of each pair lies next to a border between two codes, the nearest of
    16,384 pairs; and of one pair of each head next to a border that its scale was made for,
    at 2^-26 to 2^-37 of it.  `mag`: log2 of the pairs' magnitude."""
    g = torch.Generator().manual_seed(seed)
    cos, sin = (v[:, 0] for v in angles(pos, freq))
    T, R = cos.shape
    grid = P.code_values(kind)
    borders = (grid[1:] + grid[:-1]) / 2

    def rand(*shape):
        return torch.rand(shape, generator=g, dtype=torch.float64)

    def sign(*shape):
        return (torch.randint(0, 2, shape, generator=g) * 2 - 1).double()

    def any_of(values, *shape):
        return values[torch.randint(0, len(values), shape, generator=g)]

    def held(v):
        return v.to(P.TORCH[dtype]).double()

    def least(off, fine):
        return torch.where(fine, off, torch.full_like(off, math.inf)).argmin(-1, keepdim=True)
    x, y = torch.zeros(2, T, H, R, dtype=torch.float64)
    scale = torch.zeros(H, dtype=torch.float64)
    for h in range(H):
        # the scale, for one pair of the first token
        i, K = int(torch.randint(0, R, (1,), generator=g)), 8192
        a0, b0 = (held(sign(K) * torch.exp2(mag + 2 * rand(K) - 1)) for _ in "xy")
        u, at = turn(a0, b0, cos[0, i], sin[0, i])[h % 2].abs(), any_of(borders, K)
        s = (u / at).float().double()
        fine = torch.isfinite(s) & (s > 0) & torch.isfinite(a0 + b0)
        off = (u / torch.where(fine, s, torch.ones_like(s)) / at - 1).abs()
        best = int(least((off.log2() + (26, 30, 34, 37)[h // 2 % 4]).abs(), fine & (off > 0)))
        scale[h] = s[best]
        # the pairs: y from x and a border, rounded to what the type holds
        N = 16384
        low, high = (2.0 ** -8, 2.0 ** 13) if dtype == "f16" else (2.0 ** (mag - 3), 2.0 ** min(mag + 3, 127))
        usable = borders[(borders * s[best] >= low) & (borders * s[best] <= high)]
        for k in range(T):
            c, d = cos[k][:, None], sin[k][:, None]
            first = d.abs() >= c.abs()                       # of the two outputs: in which y counts more
            want = any_of(usable, R, N) * sign(R, N) * s[best]
            a = held(want.abs() * torch.exp2(2 * rand(R, N) - 1) * sign(R, N))
            b = held(torch.where(first, (a * c - want) / d, (want - a * d) / c))
            u, v = turn(a, b, c, d)
            off = (torch.where(first, u, v) - want).abs() / (a.abs() + b.abs())
            near = least(off, torch.isfinite(a + b) & (off > 0))
            x[k, h], y[k, h] = a.gather(1, near)[:, 0], b.gather(1, near)[:, 0]
        x[0, h, i], y[0, h, i] = a0[best], b0[best]
    return x, y, scale


def append(dtype, kind, x, y, scale, pos, freq, interleaved):
    """Codes (tokens, heads, 2, pairs) that the call writes for the pairs' rotation."""
    T, R = x.shape[0], x.shape[-1]
    page = 16 if max(pos) < 1 << 20 else 1 << 14
    pairs = torch.stack((x, y), -1 if interleaved else -2).flatten(-2)
    k = torch.zeros(T, H, D, dtype=P.TORCH[dtype])
    k[..., : 2 * R] = pairs.to(k.dtype)
    assert torch.equal(k[..., : 2 * R].double(), pairs)
    pools = [torch.zeros(T, page, H, D, dtype=P.TORCH[kind], device="cuda") for _ in "kv"]
    table = torch.full((T, max(pos) // page + 1), -1, dtype=torch.int32)
    for t, p in enumerate(pos):
        table[t, p // page] = t
    lens, cu = torch.tensor(pos, dtype=torch.int32) + 1, torch.arange(T + 1, dtype=torch.int32)
    s = scale.float().cuda()
    sfa.paged_append_rotated(k.cuda(), k.cuda(), cu.cuda(), *pools, table.cuda(), lens.cuda(), freq.cuda(),
                             interleaved=interleaved, scale_k=s, scale_v=s)
    got = raw(pools[0])[torch.arange(T), [p % page for p in pos]][..., : 2 * R]
    return got.unflatten(-1, (R, 2)).transpose(-1, -2) if interleaved else got.unflatten(-1, (2, R))


def exact(x, y, scale, pos, freq):
    """Quotients (tokens, heads, 2, pairs) in 64 bits and how far off they, or the pair's
    rotation in 64 bits on the device, may be.

    Relative to |x| + |y|: the angle, 4 units of 2^-64 turns a position (five roundings to
    units; for frequencies up to 1 the rest is below a tenth of one); the series, 2^-45 (the
    terms behind the seventh of the sine and the eighth of the cosine: (pi/4)^15 / 15! =
    2^-45.5); its arithmetic in units of 2^-61; the 64-bit roundings here and there, 2^-50.
    An angle of zero is exact."""
    cos, sin = angles(pos, freq)
    s = scale[:, None]
    q = torch.stack([v / s for v in turn(x, y, cos, sin)], 2)
    p = torch.tensor(pos, dtype=torch.float64)[:, None, None]
    off = torch.where(p * freq.double() != 0, p * 4 * 2.0 ** -64 * 2 * math.pi + 2.0 ** -45 + 2.0 ** -50, torch.tensor(0.0).double())
    return q, (off * ((x.abs() + y.abs()) / s))[:, :, None].expand_as(q)


def check(got, q, off, kind):
    low, high = (P.nearest_code(v, kind).view(P.TORCH[kind]).float() for v in (q - off, q + off))
    at = got.contiguous().view(P.TORCH[kind]).float()
    bad = ~((low <= at) & (at <= high))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}: {at[bad][:4].tolist()} for {q[bad][:4].tolist()}"
    # codes are told apart nearly everywhere (of the inputs alone; far out the angle lets some
    # of the nearest pairs be either)
    assert (low != high).sum() <= 0.02 * low.numel()


CASES = [(dtype, kind, pairs) for dtype in ("bf16", "f16") for kind in ("e4m3", "e5m2") for pairs in (False, True)]
# Where a token stands.  (Beyond 2^29 the product with a frequency is not exact in 64 bits.)
PLACES = [[1, 7, 100], [4093, 100003, 131071], [1 << 20, 20000003, (1 << 28) - 1]]


@pytest.mark.parametrize("place", range(len(PLACES)))
@pytest.mark.parametrize("dtype,kind,interleaved", CASES)
def test_next_to_borders(dtype, kind, interleaved, place):
    pos, freq = PLACES[place], frequencies(D if place else 32)
    x, y, scale = made(dtype, kind, pos, freq, 0.0, 7 + place)
    q, off = exact(x, y, scale, pos, freq)
    # what makes this a test: rotation and quotient in 32 bits give other codes
    cos, sin = (v.float() for v in angles(pos, freq))
    plain = torch.stack([v / scale.float()[:, None] for v in turn(x.float(), y.float(), cos, sin)], 2)
    assert (P.nearest_code(plain.double(), kind) != P.nearest_code(q, kind)).sum() >= 10
    check(append(dtype, kind, x, y, scale, pos, freq, interleaved), q, off, kind)


@pytest.mark.parametrize("mag", [126, 115, 98, -98, -115, -131])
@pytest.mark.parametrize("kind,interleaved", [("e4m3", False), ("e4m3", True), ("e5m2", False), ("e5m2", True)])
def test_scales_and_keys_at_the_ends_of_the_range(kind, interleaved, mag):
    """bf16 keys up to the largest and down into the subnormal numbers, with scales (any
    positive finite one) that bring them to codes of every size."""
    pos, freq = [3, 50, 1000], frequencies(D)
    x, y, scale = made("bf16", kind, pos, freq, mag, 50)
    q, off = exact(x, y, scale, pos, freq)
    check(append("bf16", kind, x, y, scale, pos, freq, interleaved), q, off, kind)


@pytest.mark.parametrize("dtype,kind,interleaved", CASES)
def test_ties(dtype, kind, interleaved):
    """Angles of zero (the first position, or a frequency of zero): exact quotients, ties to
    the even code, whatever the scale."""
    g = torch.Generator().manual_seed(4)
    grid = P.code_values(kind)
    borders = (grid[1:] + grid[:-1]) / 2
    borders = borders[borders <= 1024]                       # (times the scale an fp16 number)
    scale = torch.tensor([1.0, 3.0, 5.0, 7.0] * 4).double() * torch.exp2(torch.randint(-3, 3, (H,), generator=g).double())
    pos, freq = [0, 900], frequencies(D)
    freq[1::2] = 0.0
    pick = torch.randint(0, len(borders), (2, 2, H, D // 2), generator=g)
    sign = (torch.randint(0, 2, pick.shape, generator=g) * 2 - 1).double()
    x, y = borders[pick] * sign * scale[:, None]
    q, off = exact(x, y, scale, pos, freq)
    assert (off == 0).sum() == off.numel() * 3 // 4
    on = torch.isin(q.abs(), borders)
    assert on[off == 0].all()
    got = append(dtype, kind, x, y, scale, pos, freq, interleaved)
    want = P.nearest_code(q, kind)
    assert torch.equal(got[off == 0], want[off == 0])
    check(got, q, off, kind)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rotated", [False, True])
def test_subnormal_values_and_scales(kind, rotated):
    """Values as they are: every subnormal bf16 number over subnormal scales whose quotient
    rounded to fp32 is a border that the exact one only nearly is, the difference being below
    the smallest fp32 number."""
    grid = P.code_values(kind)
    borders = (grid[1:] + grid[:-1]) / 2
    m = torch.arange(128, dtype=torch.float64)
    x = m * 2.0 ** -133
    # scales: the multiples of 2^-149 around the exact x / border, where that is subnormal
    at = (x[1:, None] / borders).flatten()
    s = torch.cat([torch.floor(at * 2.0 ** 149), torch.ceil(at * 2.0 ** 149)]).unique()
    s = s[(s >= 1) & (s < 2 ** 23)] * 2.0 ** -149
    q = x / s[:, None]                                       # off by 2^-53 of itself; borders by 2^-33 or more, or met
    rounded = torch.isin(q.float().double(), borders) & ~torch.isin(q, borders)
    s = s[rounded.sum(1).topk(64).indices]
    q, rounded = x / s[:, None], (x / s[:, None]).float().double()
    want = P.nearest_code(q, kind)
    # what makes this a test: the quotient in fp32 gives other codes
    assert (P.nearest_code(rounded, kind) != want).sum() >= 64
    k = x.to(torch.bfloat16).expand(64, 128).contiguous()
    assert torch.equal(k.double(), x.expand(64, 128))
    new = torch.stack((k, -k)).cuda()                        # two tokens of 64 heads
    pools = [torch.zeros(1, 16, 64, 128, dtype=P.TORCH[kind], device="cuda") for _ in "kv"]
    lists = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 2], [[0]], [2])]
    scale = s.float().cuda()
    if rotated:
        sfa.paged_append_rotated(new, new, lists[0], *pools, *lists[1:], frequencies(64).cuda(), scale_k=scale, scale_v=scale)
    else:
        sfa.paged_append(new, new, lists[0], *pools, *lists[1:], scale_k=scale, scale_v=scale)
    for pool, first in ((pools[0], 64 if rotated else 0), (pools[1], 0)):        # (what does not turn)
        got = raw(pool)[0, :2]
        assert torch.equal(got[0, :, max(first, 1):], want[:, max(first, 1):])
        assert torch.equal(got[1, :, max(first, 1):], want[:, max(first, 1):] + 128)


@pytest.mark.parametrize("interleaved", [False, True])
def test_large_frequencies(interleaved):
    """Angles of frequencies up to 2^20 at positions up to the last a table can have."""
    page, T, R = 1 << 20, 3, 32
    freq = torch.logspace(0, 20, R, base=2.0) * (torch.arange(R) % 3 - 1).sign().add(0.5).sign()
    freq[-1], freq[-2] = 2.0 ** 20, -1e6
    g = torch.Generator().manual_seed(8)
    qk = torch.randn((T, 2, 2 * R), generator=g).half()
    pools = [torch.zeros(1, page, 1, 2 * R, dtype=torch.float16, device="cuda") for _ in "kv"]
    for last in (1023 * page, 700000001):
        table = torch.full((1, 1023), 0, dtype=torch.int32)
        lens, cu = torch.tensor([last], dtype=torch.int32), torch.tensor([0, T], dtype=torch.int32)
        d = qk.cuda()
        out = sfa.paged_append_rotated(d[:, 1:], d[:, 1:], cu.cuda(), *pools, table.cuda(), lens.cuda(), freq.cuda(), q=d[:, :1],
                                       interleaved=interleaved)
        pos = list(range(last - T, last))
        X.check_rotated(out.cpu(), *X.rotated(qk[:, :1], pos, freq, interleaved), "f16")
        got = pools[0].cpu()[0, [p % page for p in pos]]
        X.check_rotated(got, *X.rotated(qk[:, 1:], pos, freq, interleaved), "f16")
