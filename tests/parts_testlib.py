"""Plain 64-bit restatements of attention over parts of the keys and of the position
rotation, beside those of paged_testlib."""
import math

import torch

from tests import paged_testlib as P


def attend_seen(q, k, v, seen, scale):
    """One sequence in float64: q (n, Hq, D), k, v (L, H, D), seen (n, L): which keys a
    row sees.  What attend() of paged_testlib returns."""
    n, Hq, D = q.shape
    L, H = k.shape[:2]
    some = seen.any(0)
    k, v = (torch.where(some[:, None, None], x, torch.zeros_like(x)).repeat_interleave(Hq // H, 1) for x in (k, v))
    if L == 0:
        z = torch.zeros(n, Hq, D, dtype=torch.float64)
        return z, torch.full((n, Hq), -math.inf, dtype=torch.float64), z, z[..., 0]
    x = torch.einsum("ihd,jhd->hij", q, k) * scale
    x = torch.where(seen[None], x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True).clamp(min=-1e300)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + total.log()).squeeze(-1).T
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    out, A = torch.einsum("hij,jhd->ihd", p, v), torch.einsum("hij,jhd->ihd", p, v.abs())
    S = torch.einsum("ihd,jhd->hij", q.abs(), k.abs()) * seen[None]
    return out, lse, A, (S * abs(scale)).amax(-1).T


def window_mask(n, L, window, sinks):
    """(n, L): which keys the newest n of L tokens see."""
    p = torch.arange(n)[:, None] + L - n
    j = torch.arange(L)[None, :]
    return (j <= p) & ((p - j < window) | (j < sinks))


def poison_unseen(c, seen):
    """NaN in the places of a cache's tokens that no row of any sequence sees (seen: a
    (rows, tokens) mask for each)."""
    bad = torch.zeros(c.pages, c.page, dtype=torch.bool)
    for good in (False, True):
        for b, s in enumerate(seen):
            page, place = c.cells(b)
            pick = (page >= 0) & (s.any(0) == good)
            bad[page[pick], place[pick]] = not good
    for x in (c.k, c.v):
        y = x.view(torch.uint8) if c.cache != "same" else x
        y = y.transpose(1, 2) if c.layout == "HND" else y
        y[bad] = float("nan") if c.cache == "same" else 0x7F
    return c


def rotated(x, pos, inv_freq, interleaved):
    """Float64 rows x (tokens, heads, D) turned by their positions; and for every element
    the sum of the magnitudes it is made of."""
    r = 2 * len(inv_freq)
    # the exact angle, whole turns taken off in integers where the product is long
    angle = torch.tensor([[math.fmod(int(t) * float(f), 2 * math.pi) if abs(int(t) * float(f)) < 2 ** 20
                           else float(_reduced(int(t), float(f))) for f in inv_freq] for t in pos],
                         dtype=torch.float64).view(len(pos), -1)
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    x = x.double()
    y, size = x.clone(), x.abs()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        to = (slice(0, r, 2), slice(1, r, 2))
    else:
        a, b = x[..., : r // 2], x[..., r // 2: r]
        to = (slice(0, r // 2), slice(r // 2, r))
    y[..., to[0]], y[..., to[1]] = a * cos - b * sin, a * sin + b * cos
    for s in to:
        size[..., s] = a.abs() + b.abs()
    return y, size, r


def _reduced(t, f):
    """t * f modulo 2 pi, by exact fractions (2 pi to 100 digits)."""
    from fractions import Fraction
    two_pi = Fraction("6.2831853071795864769252867665590057683943387987502116419498891846156328125724179972560696506842341359")
    x = Fraction(t) * Fraction(f)
    return x - two_pi * (x // two_pi)


# What a rotated element may be off by, relative to the sum of the magnitudes that make
# it, before its rounding: the angle 2^-22, cosine and sine one unit in the last place
# (2^-23), two products and a sum 2^-23.
ROTATION = 2.0 ** -22 + 2.0 ** -23 + 2.0 ** -23


def check_rotated(got, want, size, r, dtype):
    """16-bit results: what turns within its bound, the rest to the bit."""
    got = got.double()
    h = torch.finfo(P.TORCH[dtype]).eps / 2
    tol = h * want.abs() + ROTATION * (1 + h) * size + (2.0 ** -25 if dtype == "f16" else 0)
    err = (got - want).abs()
    assert torch.all((err <= tol)[..., :r]), f"{float((err / tol)[..., :r].nan_to_num().max()):.3g} times the bound"
    assert torch.equal(got[..., r:], want[..., r:])


def check_rotated_codes(got, want, size, r, scale, kind):
    """8-bit codes: those of a quotient within the rotation's bound (mostly that is one
    code), the rest the nearest to the bit."""
    s = scale.double().view(1, -1, 1)
    tol = ROTATION * size
    tol[..., r:] = 0

    def value(y):
        code = P.nearest_code(y / s, kind)
        return code.view(P.TORCH[kind]).float()
    low, high, at = value(want - tol), value(want + tol), got.view(P.TORCH[kind]).float()
    assert torch.all((low <= at) & (at <= high))
    # The check says little where two codes are allowed.  That is so of the inputs alone:
    # codes lie 2^-4 of their value apart at least, the bound is 2^-20.7 of the pair's size,
    # so it takes a quotient within 2^-15 of a border, or one much smaller than its pair
    # (at positions around 2^30 one element of 768 is 0.0013 of a pair of 1.27, its quotient
    # 0.2109 on the border between 0.2031 and 0.2188).
    assert (low != high).sum() <= 1 + 1e-3 * low.numel()
