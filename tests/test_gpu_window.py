"""Attention through a sliding window with sinks on the GPU, over pages and over packed
rows, against plain 64-bit arithmetic."""
import math

import pytest
import torch

import sparse_attention_serving_sfa_gb300 as sfa
from tests import paged_testlib as P
from tests import parts_testlib as X
from tests.test_gpu_paged import SHAPES, kw, run_paged, widen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    sfa.build()
    sfa.load()


def masks(c, window, sinks):
    return [X.window_mask(n, L, window, sinks) for n, L in zip(c.q_lens, c.kv_lens)]


def check_window(c, out, lse, window, sinks, scale=0.0):
    scale = scale or 1 / math.sqrt(c.D)
    q, _, _ = c.split(c.qkv)
    for b, seen in enumerate(masks(c, window, sinks)):
        s = slice(int(c.cu[b]), int(c.cu[b + 1]))
        k, there = c.values(c.k, c.scale_k, b)
        v, _ = c.values(c.v, c.scale_v, b)
        ref = X.attend_seen(q[s].double(), k, v, seen & there, scale)
        P.check(out[s], lse[s], ref, c.dtype, max(1, int(seen.sum(1).max()) if seen.numel() else 1), f"sequence {b}")
    for x in (out, lse):
        assert torch.all(x[: c.cu[0]] == 9) and torch.all(x[c.cu[-1]:] == 9)


WINDOWS = [(1, 0), (1, 1), (7, 3), (64, 0), (100, 130), (128, 128), (333, 4), (1000, 1), ((1 << 31) - 1, 0), (5, (1 << 31) - 1)]


@pytest.mark.parametrize("cache,layout,dtype", [("same", "NHD", "bf16"), ("same", "HND", "f16"),
                                                ("e4m3", "HND", "bf16"), ("e5m2", "NHD", "f16")])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_window_over_pages(shape, cache, layout, dtype):
    q_lens, kv_lens, heads, kv_heads, dim, page = SHAPES[shape]
    for window, sinks in WINDOWS:
        c = P.Cache(100 + shape, q_lens, kv_lens, heads, kv_heads, dim, page, dtype, cache, layout,
                    before=1, behind=2).poison()
        X.poison_unseen(c, masks(c, window, sinks))
        # both kernels, whatever the lengths
        for hint in (1, 0):
            out, lse = run_paged(c, True, hint, window=window, sinks=sinks)
            check_window(c, out, lse, window, sinks)


@pytest.mark.parametrize("cache,layout,dtype", [("same", "NHD", "bf16"), ("e4m3", "HND", "f16"),
                                                ("e5m2", "NHD", "bf16")])
@pytest.mark.parametrize("shape", [1, 2, 3, 4, 6, 9, 10])
def test_table_much_wider_than_the_sequences(shape, cache, layout, dtype):
    q_lens, kv_lens, heads, kv_heads, dim, page = SHAPES[shape]
    for window, sinks in ((1, 0), (200, 5), (2000, 0), (1 << 20, 1)):
        c = P.Cache(200 + shape, q_lens, kv_lens, heads, kv_heads, dim, page, dtype, cache, layout,
                    before=1, behind=2).poison()
        X.poison_unseen(c, masks(c, window, sinks))
        widen(c)
        out, lse = run_paged(c, True, 0, window=window, sinks=sinks)
        check_window(c, out, lse, window, sinks)


@pytest.mark.parametrize("cache,dtype,layout", [("same", "bf16", "HND"), ("same", "f16", "NHD"), ("e4m3", "bf16", "NHD"),
                                                ("e5m2", "f16", "HND")])
@pytest.mark.parametrize("page", [1, 8, 16, 20, 24, 64, 128, 160])
def test_pages_behind_the_window_are_gone(page, cache, dtype, layout):
    """A serving program gives pages back as the window leaves them: their entries name
    no page, or another sequence's."""
    window, sinks = 300, 5
    c = P.Cache(31, [40, 1, 170], [900, 1500, 1100], 8, 2, 128, page, dtype, cache, layout, behind=1).poison()
    for n, (q_len, L) in enumerate(zip(c.q_lens, c.kv_lens)):
        first = L - q_len - window + 1                       # the lowest key of the first row
        for x in range(-(-sinks // page), first // page):
            c.table[n, x] = (-1, c.pages, int(c.table[(n + 1) % 3, 0]))[x % 3]
    full = [X.window_mask(n, L, window, sinks) for n, L in zip(c.q_lens, c.kv_lens)]
    for hint in (170, 0, 1):
        out, lse = run_paged(c, True, hint, window=window, sinks=sinks)
        check_window(c, out, lse, window, sinks)
    assert all(m.any() for m in full)


@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("hint,wide", [(1, False), (0, False), (0, True)])
def test_missing_pages_inside_the_window(cache, hint, wide):
    c = P.Cache(21, [1, 70, 3], [90, 200, 64], 8, 2, 128, 16, "bf16", cache).poison()
    c.table[0, 2] = c.pages
    c.table[0, 5] = -1                       # all a short window shows
    c.table[1, 0] = -1
    c.table[1, 9] = 1 << 30
    c.table[2] = -5
    if wide:
        widen(c)
    for window, sinks in ((10, 0), (50, 3)):
        out, lse = run_paged(c, True, hint, window=window, sinks=sinks)
        check_window(c, out, lse, window, sinks)
    assert torch.isneginf(lse[-3:]).all()


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3"), ("bf16", "e5m2")])
@pytest.mark.parametrize("hint,wide", [(1, False), (0, False), (0, True)])
def test_large_scores_and_scales(dtype, cache, hint, wide):
    c = P.Cache(22, [6, 1, 40], [700, 333, 600], 8, 2, 128, 16, dtype, cache)
    q, _, _ = c.split(c.qkv)
    q *= torch.logspace(-6, 1.2, c.T).to(q.dtype)[:, None, None]
    for b in range(3):
        page, place = c.cells(b)
        if cache == "same":
            c.k[page, place] *= torch.linspace(0.01, 3, len(page)).to(c.k.dtype)[:, None, None]
    if wide:
        widen(c)
    for scale in (0.0, 1.0):
        out, lse = run_paged(c, True, hint, scale, window=200, sinks=2)
        check_window(c, out, lse, 200, 2, scale)


@pytest.mark.parametrize("dtype,cache", [("f16", "same"), ("bf16", "e4m3")])
@pytest.mark.parametrize("q_lens,kv_lens,window,sinks", [
    ([1] * 7, [30000, 1, 17, 2500, 64, 9000, 128], 8000, 4), ([1] * 3, [60000, 59999, 3], 50000, 70),
    ([700, 3], [20000, 9000], 6000, 1), ([2500], [2500], 300, 40), ([3000, 1, 900], [3000, 700, 901], 1000, 0)])
def test_long_windows_split_over_many_ranges(q_lens, kv_lens, window, sinks, dtype, cache):
    c = P.Cache(23, q_lens, kv_lens, 8, 2, 64, 16, dtype, cache).poison()
    X.poison_unseen(c, masks(c, window, sinks))
    for hint in (max(q_lens), 0):
        out, lse = run_paged(c, True, hint, window=window, sinks=sinks)
        check_window(c, out, lse, window, sinks)
        again, lse2 = run_paged(c, True, hint, window=window, sinks=sinks)
        assert torch.equal(out, again) and torch.equal(lse, lse2)      # nothing depends on timing


@pytest.mark.parametrize("hint", [1, 0])
def test_offsets_beyond_32_bits(hint):
    """Pools of more than 2^31 elements, the pages used at their far end."""
    H, D, page = 8, 128, 64
    pages = (1 << 31) // (H * D * page) + 40
    c = P.Cache(24, [2, 33], [100, 400], 16, H, D, page, "bf16")
    d = c.to("cuda")
    shift = pages - c.pages
    for n in "kv":
        x = torch.empty((pages, page, H, D), dtype=torch.bfloat16, device="cuda")
        x[shift:] = d[n]
        d[n] = x
    d["table"] = torch.where(d["table"] >= 0, d["table"] + shift, d["table"])
    out, lse = run_paged(c, True, hint, d=d, window=90, sinks=3)
    check_window(c, out, lse, 90, 3)


@pytest.mark.parametrize("group", [65, 128, 129])
def test_large_groups(group):
    c = P.Cache(44, [9, 30], [200, 131], group, 1, 128, 16, "bf16").poison()
    for hint in (0, 1):
        out, lse = run_paged(c, True, hint, window=33, sinks=2)
        check_window(c, out, lse, 33, 2)


def test_lists_are_read_as_clamped():
    c = P.Cache(25, [4, 4], [40, 40], 4, 2, 64, 16, "f16")
    d = c.to("cuda")
    d["cu"] = torch.tensor([-3, 5, 1 << 30], dtype=torch.int32, device="cuda")
    d["lens"] = torch.tensor([1 << 30, -4], dtype=torch.int32, device="cuda")
    for hint in (1, 0):
        for window, sinks in ((1, 0), ((1 << 31) - 1, (1 << 31) - 1)):
            run_paged(c, True, hint, d=d, window=window, sinks=sinks)


# ---------------------------------------------------------------- packed rows

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim", [
    ([1], [1], 1, 1, 64), ([5, 0, 300], [9, 4, 300], 8, 2, 128), ([700, 33], [700, 40], 6, 2, 64),
    ([1, 1, 1], [500, 3, 1200], 32, 8, 128), ([257], [2000], 3, 1, 128), ([4, 9], [0, 3], 4, 4, 64)])
def test_window_over_packed_rows(q_lens, kv_lens, heads, kv_heads, dim, dtype):
    g = torch.Generator().manual_seed(5)
    t = P.TORCH[dtype]

    def cumulative(lens, before):
        cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(lens).cumsum(0)
        return cu + before
    cq, ck = cumulative(q_lens, 2), cumulative(kv_lens, 1)
    T, N = sum(q_lens) + 5, sum(kv_lens) + 3
    q = torch.randn((T, heads + 1, dim), generator=g).to(t)[:, :heads]
    kv = torch.randn((N, 2 * kv_heads, dim), generator=g).to(t)
    for window, sinks in WINDOWS:
        kv2 = kv.clone()
        seen = [X.window_mask(n, L, window, sinks) for n, L in zip(q_lens, kv_lens)]
        free = torch.ones(N, dtype=torch.bool)
        for b, s in enumerate(seen):
            free[int(ck[b]): int(ck[b + 1])] = ~s.any(0)
        kv2[free] = float("nan")
        k, v = kv2[:, :kv_heads], kv2[:, kv_heads:]
        kd = kv2.cuda()
        for hint in (1, 0):
            out = torch.full((T, heads, dim), 9.0, dtype=t, device="cuda")
            lse = torch.full((T, heads), 9.0, device="cuda")
            qd = torch.zeros((T, heads + 1, dim), dtype=t, device="cuda")
            qd[:, :heads] = q
            sfa.varlen_attention(qd[:, :heads], kd[:, :kv_heads], kd[:, kv_heads:], cq.cuda(), ck.cuda(), out=out, lse=lse,
                                 max_q_len=hint, window=window, sinks=sinks)
            out, lse = out.cpu(), lse.cpu()
            assert sfa.sfa_get_last_error() == sfa.SFA_OK
            for b, s in enumerate(seen):
                rows, keys = slice(int(cq[b]), int(cq[b + 1])), slice(int(ck[b]), int(ck[b + 1]))
                ref = X.attend_seen(q[rows].double(), k[keys].double(), v[keys].double(), s, 1 / math.sqrt(dim))
                P.check(out[rows], lse[rows], ref, dtype, max(1, kv_lens[b]), f"sequence {b}")
            for x in (out, lse):
                assert torch.all(x[: cq[0]] == 9) and torch.all(x[cq[-1]:] == 9)


def test_a_long_prompt():
    """8,192 tokens through windows that end inside tiles; rows picked from everywhere."""
    n, H, D = 8192, 2, 128
    g = torch.Generator().manual_seed(9)
    q = torch.randn((n, 4 * H, D), generator=g).bfloat16()
    k, v = (torch.randn((n, H, D), generator=g).bfloat16() for _ in range(2))
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    rows = torch.tensor([0, 1, 126, 127, 128, 700, 1499, 1500, 1501, 1627, 4095, 4096, 8000, 8191])
    for window, sinks in ((1500, 0), (1500, 7), (129, 1), (4096, 128)):
        out, lse = sfa.varlen_attention(q.cuda(), k.cuda(), v.cuda(), cu, cu, return_lse=True, window=window, sinks=sinks)
        seen = X.window_mask(n, n, window, sinks)[rows]
        ref = X.attend_seen(q[rows].double(), k.double(), v.double(), seen, 1 / math.sqrt(D))
        P.check(out.cpu()[rows], lse.cpu()[rows], ref, "bf16", window + sinks)
