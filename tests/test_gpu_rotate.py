"""Appending with the position rotation on the GPU: the pages and the rotated queries
against plain 64-bit arithmetic."""
import pytest
import torch

import sparse_attention_serving_sfa_gb300 as sfa
from tests import paged_testlib as P
from tests import parts_testlib as X
from tests.test_gpu_paged import kw, raw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    sfa.build()
    sfa.load()


def frequencies(r, base=10000.0):
    return (base ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float()


def positions(c):
    """Token of every row of the sequences, and those rows."""
    rows, pos = [], []
    for b, n in enumerate(c.q_lens):
        rows += range(int(c.cu[b]), int(c.cu[b + 1]))
        pos += range(c.kv_lens[b] - n, c.kv_lens[b])
    return rows, pos


def check_pages(c, d, rows, pos, freq, interleaved):
    """The pools as they must be: new tokens rotated (K) or as they are (V), every
    other place as it was."""
    _, k, v = c.split(c.qkv)
    for x, pool, scale, got, turned in ((k, c.k, c.scale_k, d["k"], True), (v, c.v, c.scale_v, d["v"], False)):
        got, old = raw(got), raw(pool).clone()
        g, w = (y.transpose(1, 2) if c.layout == "HND" else y for y in (got, old))
        where = {}
        for b, n in enumerate(c.q_lens):
            page, place = c.cells(b)
            for i in range(n):
                at = c.kv_lens[b] - n + i
                if at >= 0 and page[at] >= 0:
                    where[int(c.cu[b]) + i] = (int(page[at]), int(place[at]))
        have = [i for i, t in enumerate(rows) if t in where]
        at = tuple(torch.tensor(y, dtype=torch.long) for y in zip(*[where[rows[i]] for i in have])) if have else None
        if have:
            new, p = x[[rows[i] for i in have]], [pos[i] for i in have]
            if turned:
                want, size, r = X.rotated(new, p, freq, interleaved)
            else:
                want, size, r = new.double(), new.double().abs(), 0
            if c.cache == "same":
                X.check_rotated(g[at].view(P.TORCH[c.dtype]), want, size, r, c.dtype)
            else:
                X.check_rotated_codes(g[at], want, size, r, scale, c.cache)
            w[at] = g[at]
        assert torch.equal(got, old)


CASES = [
    # q_lens, kv_lens, heads, kv_heads, dim, page, dtype, cache, layout, rotary, interleaved
    ([1], [1], 1, 1, 64, 1, "bf16", "same", "NHD", 64, False),
    ([1, 1, 1], [7, 1, 33], 32, 8, 128, 16, "bf16", "e4m3", "NHD", 128, False),
    ([5, 0, 17, 1], [5, 9, 40, 1], 6, 3, 64, 5, "f16", "e5m2", "HND", 32, True),
    ([33, 2, 0, 64], [50, 2, 0, 64], 2, 2, 128, 24, "f16", "e4m3", "HND", 96, True),
    ([130, 7], [131, 3000], 16, 1, 128, 64, "bf16", "e5m2", "NHD", 16, False),
    ([19, 3], [19, 90], 15, 5, 128, 7, "f16", "same", "HND", 48, False),
    ([70, 9], [5000, 9], 5, 5, 64, 20, "bf16", "same", "HND", 64, True),
    ([900, 1300], [900, 1301], 4, 2, 64, 16, "f16", "same", "NHD", 64, False),
]


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim,page,dtype,cache,layout,rotary,interleaved", CASES)
def test_append_rotated(q_lens, kv_lens, heads, kv_heads, dim, page, dtype, cache, layout, rotary, interleaved):
    c = P.Cache(11, q_lens, kv_lens, heads, kv_heads, dim, page, dtype, cache, layout, before=2, behind=3)
    freq = frequencies(rotary)
    rows, pos = positions(c)
    for way in ("new", "in place", "none", "given"):
        d = c.to("cuda")
        q, k, v = c.split(d["qkv"])
        given = {"new": None, "in place": q, "none": None,
                 "given": torch.full((c.T, heads + 1, dim), 9.0, dtype=q.dtype, device="cuda")[:, :heads]}[way]
        out = sfa.paged_append_rotated(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"], freq.cuda(),
                                       q=None if way == "none" else q, q_out=given, interleaved=interleaved, **kw(c, d))
        torch.cuda.synchronize()
        check_pages(c, d, rows, pos, freq, interleaved)
        old = c.split(c.qkv)[0]
        if way == "none":
            assert out is None and torch.equal(d["qkv"].cpu(), c.qkv)
            continue
        want, size, r = X.rotated(old[rows], pos, freq, interleaved)
        X.check_rotated(out.cpu()[rows], want, size, r, dtype)
        others = [t for t in range(c.T) if t not in set(rows)]
        if way == "in place":
            assert out.data_ptr() == q.data_ptr() and torch.equal(out.cpu()[others], old[others])
            assert torch.equal(d["qkv"].cpu()[:, heads:], c.qkv[:, heads:])
        elif way == "given":
            assert (out.cpu()[others] == 9).all() and (given._base.cpu()[:, heads] == 9).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "e4m3")])
def test_far_positions(dtype, cache, interleaved):
    """Positions up to the last a table can have, frequencies from 0 to beyond a turn a
    token, some negative (angles below 2^28)."""
    page, dim = 1 << 20, 64
    c = P.Cache(12, [9, 3], [9, 3], 2, 1, dim, 16, dtype, cache)
    freq = frequencies(32, 500000.0)
    freq[3:9] = torch.tensor([0.0, -1.0, 3.25, 7.0, -12.0, 1e-9])
    shape = (2, page, 1, dim)
    for last in (1000003, 20000000, 1023 * page):
        if last > 1 << 25:
            freq = freq * 0.02
        c.kv_lens = [last, last - 5]
        width = -(-last // page)
        table = torch.full((2, width), -1, dtype=torch.int32)
        table[0, (last - 9) // page:] = 0
        table[1, (last - 8) // page:] = 1
        pools = [torch.zeros(shape, dtype=P.TORCH[cache if cache != "same" else dtype], device="cuda") for _ in "kv"]
        d = c.to("cuda")
        q, k, v = c.split(d["qkv"])
        lens = torch.tensor(c.kv_lens, dtype=torch.int32, device="cuda")
        out = sfa.paged_append_rotated(k, v, d["cu"], *pools, table.cuda(), lens, freq.cuda(), q=q,
                                       interleaved=interleaved, **kw(c, d))
        rows, pos = positions(c)
        cq, ck, _ = c.split(c.qkv)
        want, size, r = X.rotated(cq[rows], pos, freq, interleaved)
        X.check_rotated(out.cpu(), want, size, r, dtype)
        got = raw(pools[0]).flatten(0, 1)[[(0 if i < 9 else page) + p % page for i, p in enumerate(pos)]]
        want, size, r = X.rotated(ck[rows], pos, freq, interleaved)
        if cache == "same":
            X.check_rotated(got.view(P.TORCH[dtype]), want, size, r, dtype)
        else:
            X.check_rotated_codes(got, want, size, r, c.scale_k, cache)


def test_rows_without_a_place():
    """Pages out of range and tokens before the first: no key is written, the query is
    rotated by its position all the same."""
    c = P.Cache(5, [20, 6, 4], [20, 4, 30], 4, 2, 64, 4, "bf16", "e4m3")
    c.table[0, 1] = c.pages
    c.table[2, 6] = -1
    d = c.to("cuda")
    q, k, v = c.split(d["qkv"])
    freq = frequencies(64)
    out = sfa.paged_append_rotated(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"], freq.cuda(), q=q, **kw(c, d))
    rows, pos = positions(c)
    assert min(pos) == -2
    check_pages(c, d, rows, pos, freq, False)
    X.check_rotated(out.cpu(), *X.rotated(c.split(c.qkv)[0], pos, freq, False), "bf16")


@pytest.mark.parametrize("B", [33, 1100])
def test_finds_sequences_among_many(B):
    q_lens = [(b * 7) % 3 for b in range(B)]
    kv_lens = [n + b % 4 for b, n in enumerate(q_lens)]
    c = P.Cache(6, q_lens, kv_lens, 1, 1, 64, 2, "f16", "same")
    d = c.to("cuda")
    q, k, v = c.split(d["qkv"])
    freq = frequencies(64)
    out = sfa.paged_append_rotated(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"], freq.cuda(), q=q)
    rows, pos = positions(c)
    X.check_rotated(out.cpu(), *X.rotated(c.split(c.qkv)[0], pos, freq, False), "f16")
    check_pages(c, d, rows, pos, freq, False)


def test_infinities_and_nan_stay_in_their_pairs():
    c = P.Cache(7, [4], [10], 2, 2, 64, 16, "bf16", "same")
    q, k, v = c.split(c.qkv)
    q[1, 0, 3] = float("nan")
    k[2, 1, 40] = float("inf")
    k[3, 0, 63] = float("nan")                  # beyond what turns
    v[0, 0, 0] = float("inf")
    d = c.to("cuda")
    q2, k2, v2 = c.split(d["qkv"])
    freq = frequencies(32)
    out = sfa.paged_append_rotated(k2, v2, d["cu"], d["k"], d["v"], d["table"], d["lens"], freq.cuda(), q=q2).cpu()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[1, 0, [3, 19]] = True
    assert torch.equal(~torch.isfinite(out.float()), bad)
    page, place = (x[6:] for x in c.cells(0))
    keys = d["k"].cpu()[page, place].float()
    assert torch.isinf(keys[2, 1, 40]) and torch.isnan(keys[3, 0, 63]) and (~torch.isfinite(keys)).sum() == 2
    assert torch.equal(d["v"].cpu()[page, place], v)


def test_nothing_to_do():
    c = P.Cache(8, [0, 0], [5, 9], 4, 2, 64, 16, "f16")
    d = c.to("cuda")
    q, k, v = c.split(d["qkv"])
    out = sfa.paged_append_rotated(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"], frequencies(64).cuda(), q=q)
    assert out.shape == (0, 4, 64)
    assert torch.equal(raw(d["k"]), raw(c.k))
