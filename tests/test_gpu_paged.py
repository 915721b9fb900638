"""The paged KV cache on the GPU: appending (quantising), reading back, and
attention of new tokens over the pages, against plain 64-bit arithmetic."""
import math

import pytest
import torch

import sparse_attention_serving_sfa_gb300 as sfa
from tests import paged_testlib as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    sfa.build()
    sfa.load()


def kw(c, d):
    return dict(kv_layout=c.layout, scale_k=d["scale_k"], scale_v=d["scale_v"])


def raw(x):
    return x.view(torch.uint8).cpu() if x.element_size() == 1 else x.view(torch.int16).cpu()


# ---------------------------------------------------------------- append

CACHES = [
    # q_lens, kv_lens, heads, dim, page, dtype, cache, layout
    ([1], [1], 1, 64, 1, "bf16", "same", "NHD"),
    ([1, 1, 1], [7, 1, 33], 8, 128, 16, "bf16", "e4m3", "NHD"),
    ([5, 0, 17, 1], [5, 9, 40, 1], 3, 64, 5, "f16", "e5m2", "HND"),
    ([33, 2, 0, 64], [50, 2, 0, 64], 2, 128, 24, "f16", "e4m3", "HND"),
    ([130, 7], [131, 300], 8, 128, 64, "bf16", "e5m2", "NHD"),
    ([19, 3], [19, 90], 5, 128, 7, "f16", "same", "HND"),
]


@pytest.mark.parametrize("q_lens,kv_lens,heads,dim,page,dtype,cache,layout", CACHES)
def test_append(q_lens, kv_lens, heads, dim, page, dtype, cache, layout):
    c = P.Cache(11, q_lens, kv_lens, heads, heads, dim, page, dtype, cache, layout, before=2, behind=3)
    d = c.to("cuda")
    _, k, v = c.split(d["qkv"])
    assert not k.is_contiguous() or k.shape[0] == 1
    sfa.paged_append(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"], **kw(c, d))
    torch.cuda.synchronize()
    for x, pool, scale, got in ((c.split(c.qkv)[1], c.k, c.scale_k, d["k"]),
                                (c.split(c.qkv)[2], c.v, c.scale_v, d["v"])):
        want = raw(pool).clone()
        w = want.transpose(1, 2) if layout == "HND" else want
        for b, n in enumerate(c.q_lens):
            new = x[c.cu[b]: c.cu[b] + n]
            page_, place = (y[c.kv_lens[b] - n:] for y in c.cells(b))
            if cache == "same":
                w[page_, place] = new.contiguous().view(torch.int16)
            else:
                w[page_, place] = P.nearest_code(new.double() / scale.double().view(1, -1, 1), cache)
        assert torch.equal(raw(got), want)          # every other place as it was


@pytest.mark.parametrize("extreme", [False, True])
@pytest.mark.parametrize("cache", ["e4m3", "e5m2"])
def test_append_rounds_the_exact_quotient(cache, extreme):
    """Every fp16 value, over scales that put many of them on borders between
    two codes, and over one where the quotient rounded to fp32 sits on a border
    that the exact one does not."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(torch.float16)
    # the fp32 neighbours of x / tie: x / s is just off the tie
    near = torch.tensor(1.0) / torch.tensor(1.0625)
    scales = torch.tensor([1.0, 0.25, 3.0, 1 / 3, float(near),
                           float(torch.nextafter(near, torch.tensor(2.0))),
                           float(torch.nextafter(near, torch.tensor(0.0))), 0.7])
    if extreme:
        scales = torch.tensor([1e-38, 3e-39, 1e-30, 2.0 ** -120, 1e30, 1.5e38, 3e38, 2.0 ** 127])
    x = every.view(-1, 1, 128).expand(-1, 8, -1).contiguous()      # 512 tokens, 8 heads
    T, H, D = x.shape
    pool = torch.zeros(T // 16, 16, H, D, dtype=P.TORCH[cache], device="cuda")
    pool2 = torch.zeros_like(pool)
    table = torch.arange(T // 16, dtype=torch.int32, device="cuda").view(1, -1)
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    sfa.paged_append(x.cuda(), x.cuda(), cu, pool, pool2, table, lens, scale_k=scales.cuda(),
                     scale_v=scales.flip(0).cuda())
    for got, s in ((pool, scales), (pool2, scales.flip(0))):
        got = raw(got).view(T, H, D)
        want = P.nearest_code(torch.nan_to_num(x.double(), nan=0.0, posinf=math.inf, neginf=-math.inf) /
                              s.double().view(1, -1, 1), cache)
        nan = torch.isnan(x)
        assert torch.equal(got[~nan], want[~nan])
        assert torch.isnan(got[nan].view(P.TORCH[cache]).float()).all()


def test_append_leaves_places_without_a_page_alone():
    c = P.Cache(5, [20, 6, 4], [20, 4, 30], 2, 2, 64, 4, "bf16", "e4m3")
    c.table[0, 1] = c.pages                 # out of range
    c.table[2, 6] = -1
    # sequence 1 claims more new tokens than it has: the first two have no position
    d = c.to("cuda")
    _, k, v = c.split(d["qkv"])
    sfa.paged_append(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"], **kw(c, d))
    want = raw(c.k).clone()
    new = c.split(c.qkv)[1]
    for b, n in enumerate(c.q_lens):
        page, place = c.cells(b)
        m = min(n, c.kv_lens[b])
        x = P.nearest_code(new[c.cu[b + 1] - m: c.cu[b + 1]].double() / c.scale_k.double().view(1, -1, 1), "e4m3")
        page, place = page[-m:], place[-m:]
        want[page[page >= 0], place[page >= 0]] = x[page >= 0]
    assert torch.equal(raw(d["k"]), want)


@pytest.mark.parametrize("B", [33, 1100])
def test_append_finds_sequences_among_many(B):
    q_lens = [(b * 7) % 3 for b in range(B)]
    kv_lens = [n + b % 4 for b, n in enumerate(q_lens)]
    c = P.Cache(6, q_lens, kv_lens, 1, 1, 64, 2, "f16", "same")
    d = c.to("cuda")
    _, k, v = c.split(d["qkv"])
    sfa.paged_append(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"])
    ko, vo = sfa.paged_read(d["k"], d["v"], d["table"], d["lens"], d["cu"], c.T)
    assert torch.equal(ko, k) and torch.equal(vo, v)


# ---------------------------------------------------------------- read

@pytest.mark.parametrize("q_lens,kv_lens,heads,dim,page,dtype,cache,layout", CACHES)
def test_read(q_lens, kv_lens, heads, dim, page, dtype, cache, layout):
    c = P.Cache(12, q_lens, kv_lens, heads, heads, dim, page, dtype, cache, layout, before=1, behind=2)
    c.poison()
    d = c.to("cuda")
    out = tuple(torch.full((c.T, heads, dim), 9.0, dtype=P.TORCH[dtype], device="cuda") for _ in range(2))
    sfa.paged_read(d["k"], d["v"], d["table"], d["lens"], d["cu"], c.T, out=out, **kw(c, d))
    for got, pool, scale in ((out[0], c.k, c.scale_k), (out[1], c.v, c.scale_v)):
        got = got.cpu()
        for b, n in enumerate(c.q_lens):
            want = c.values(pool, scale, b)[0][c.kv_lens[b] - n:]
            x = got[c.cu[b]: c.cu[b + 1]].double()
            if cache == "same":
                assert torch.equal(x, want)
            else:
                # one rounding to fp32, one to 16 bits
                h = torch.finfo(P.TORCH[dtype]).eps / 2
                assert torch.all((x - want).abs() <= (h + 2.0 ** -24) * (1 + h) * want.abs() + 2.0 ** -25)
        assert torch.all(got[: c.cu[0]] == 9) and torch.all(got[c.cu[-1]:] == 9)


def test_read_gives_zeros_where_there_is_no_token():
    c = P.Cache(13, [9, 6], [9, 4], 2, 2, 128, 4, "f16", "same")
    c.table[0, 1] = 1 << 30
    d = c.to("cuda")
    k, v = (x.cpu() for x in sfa.paged_read(d["k"], d["v"], d["table"], d["lens"], d["cu"], c.T))
    assert torch.all(k[4:8] == 0) and torch.all(v[9:11] == 0)
    assert torch.equal(k[11:], c.values(c.k, None, 1)[0].half())


# ---------------------------------------------------------------- attention

def run_paged(c, causal, max_q_len, scale=0.0, d=None, **more):
    d = d or c.to("cuda")
    q, _, _ = c.split(d["qkv"])
    out = torch.full((c.T, c.Hq, c.D), 9.0, dtype=P.TORCH[c.dtype], device="cuda")
    lse = torch.full((c.T, c.Hq), 9.0, device="cuda")
    sfa.paged_attention(q, d["k"], d["v"], d["table"], d["lens"], d["cu"], scale, causal,
                        max_q_len=max_q_len, out=out, lse=lse, **kw(c, d), **more)
    torch.cuda.synchronize()
    assert sfa.sfa_get_last_error() == sfa.SFA_OK
    return out.cpu(), lse.cpu()


def check_paged(c, out, lse, causal, scale=0.0):
    scale = scale or 1 / math.sqrt(c.D)
    q, _, _ = c.split(c.qkv)
    for b in range(len(c.q_lens)):
        s = slice(int(c.cu[b]), int(c.cu[b + 1]))
        k, there = c.values(c.k, c.scale_k, b)
        v, _ = c.values(c.v, c.scale_v, b)
        ref = P.attend(q[s].double(), k, v, there, causal, scale)
        P.check(out[s], lse[s], ref, c.dtype, max(1, c.kv_lens[b]), f"sequence {b}")
    for x in (out, lse):
        assert torch.all(x[: c.cu[0]] == 9) and torch.all(x[c.cu[-1]:] == 9)


# q_lens, kv_lens, heads, kv_heads, dim, page
SHAPES = [
    ([1], [1], 1, 1, 64, 16),
    ([1, 1, 1, 1], [129, 64, 1, 4000], 32, 8, 128, 16),           # decode, grouped heads
    ([1, 0, 1, 1], [77, 5, 0, 300], 16, 1, 128, 5),               # an empty one, one without keys
    ([1, 1], [1000, 3], 40, 8, 64, 24),                           # groups of 5
    ([4, 1, 3], [500, 1, 3], 8, 2, 128, 64),                      # a few tokens each
    ([2, 9], [1, 4], 4, 4, 64, 3),                                # more new tokens than keys: empty rows
    ([17, 130, 1], [300, 130, 700], 12, 4, 128, 32),              # a chunk
    ([257, 64], [700, 2049], 6, 2, 64, 16),                       # groups of 3
    ([300, 5], [301, 9], 3, 3, 128, 128),
    ([40, 90], [333, 1111], 32, 1, 128, 64),                      # 32 heads share a kv head
    ([100], [515], 10, 2, 128, 20),
    ([3, 5], [40, 200], 160, 1, 64, 8),                           # a group of 160
]


@pytest.mark.parametrize("cache,layout,dtype", [("same", "NHD", "bf16"), ("same", "HND", "f16"),
                                                ("e4m3", "HND", "bf16"), ("e5m2", "NHD", "f16")])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_paged_attention(shape, cache, layout, dtype):
    q_lens, kv_lens, heads, kv_heads, dim, page = SHAPES[shape]
    c = P.Cache(100 + shape, q_lens, kv_lens, heads, kv_heads, dim, page, dtype, cache, layout,
                before=1, behind=2).poison()
    for causal in (True, False):
        # both kernels, whatever the lengths
        for hint in (1, 0):
            out, lse = run_paged(c, causal, hint)
            check_paged(c, out, lse, causal)


def widen(c):
    """A page table with room for a million tokens: the large tiles take what has more than 32 rows."""
    c.table = torch.cat([c.table, torch.full((len(c.q_lens), (1 << 20) // c.page), -1, dtype=torch.int32)], 1)


@pytest.mark.parametrize("cache,layout,dtype", [("same", "NHD", "bf16"), ("e4m3", "HND", "f16"),
                                                ("e5m2", "NHD", "bf16")])
@pytest.mark.parametrize("shape", [1, 2, 3, 4, 6, 9, 10])
def test_table_much_wider_than_the_sequences(shape, cache, layout, dtype):
    q_lens, kv_lens, heads, kv_heads, dim, page = SHAPES[shape]
    c = P.Cache(200 + shape, q_lens, kv_lens, heads, kv_heads, dim, page, dtype, cache, layout,
                before=1, behind=2).poison()
    widen(c)
    out, lse = run_paged(c, True, 0)
    check_paged(c, out, lse, True)


@pytest.mark.parametrize("cache,layout,dtype", [("same", "NHD", "f16"), ("same", "HND", "bf16"),
                                                ("e4m3", "HND", "f16"), ("e5m2", "NHD", "bf16")])
@pytest.mark.parametrize("page,dim", [(1, 64), (8, 128), (8, 64), (12, 128), (20, 64), (24, 128), (40, 64), (56, 128)])
def test_chunks_over_pages_of_any_size(page, dim, cache, layout, dtype):
    c = P.Cache(300 + page, [150, 300], [700, 1111], 8, 2, dim, page, dtype, cache, layout, behind=1).poison()
    c.table[1, 100 // page] = c.pages               # a page that is not there
    for hint in (300, 0):
        out, lse = run_paged(c, True, hint)
        check_paged(c, out, lse, True)


@pytest.mark.parametrize("cache,dtype,dim", [("same", "f16", 128), ("same", "bf16", 64), ("e5m2", "f16", 128)])
@pytest.mark.parametrize("page,steps", [(20, (1,)), (24, (1, 3)), (20, (1, 3, 5)), (12, (1, 2, 3, 4))])
def test_many_short_items_over_gathered_pages(page, steps, cache, dtype, dim):
    """Pages fetched row by row, items of odd numbers of 128-key steps one after
    the other in every block: the same bits at every call."""
    B = 96
    kv_lens = [128 * steps[b % len(steps)] - (b * 29) % 100 for b in range(B)]
    q_lens = [min(20 + (b * 17) % 41, n) for b, n in enumerate(kv_lens)]
    c = P.Cache(60, q_lens, kv_lens, 32, 8, dim, page, dtype, cache).poison()
    d = c.to("cuda")
    out, lse = run_paged(c, True, max(q_lens), d=d)
    check_paged(c, out, lse, True)
    for _ in range(20):
        again, lse2 = run_paged(c, True, max(q_lens), d=d)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("cache,dtype", [("same", "bf16"), ("same", "f16"), ("e4m3", "bf16"), ("e5m2", "f16")])
@pytest.mark.parametrize("q_lens,kv_lens,heads,kv_heads,dim,page", [
    ([12], [6000], 8, 2, 128, 16),                  # three tiles a head, cut into many parts
    ([20, 5], [3000, 900], 4, 1, 64, 24),
    ([2, 2], [5000, 40], 16, 2, 128, 64),           # sixteen rows
    ([64], [2500], 1, 1, 128, 32),
    ([3], [20000], 5, 1, 64, 16),
])
def test_few_rows_cut_into_parts(q_lens, kv_lens, heads, kv_heads, dim, page, cache, dtype):
    c = P.Cache(41, q_lens, kv_lens, heads, kv_heads, dim, page, dtype, cache, before=2, behind=1).poison()
    # what is said about the lengths changes the kernel and its joins, not the result
    for hint in (max(q_lens), 1, 0):
        out, lse = run_paged(c, True, hint)
        check_paged(c, out, lse, True)


@pytest.mark.parametrize("cache,dtype", [("same", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("decode", [True, False])
def test_many_sequences_sharing_pages(decode, cache, dtype):
    """More sequences than a warp has lanes, some without rows or keys; every
    other one reads its neighbour's pages (a shared prefix)."""
    B = 70
    q_lens = [1 if decode else (0 if b % 7 == 3 else 1 + (b * 37) % 120) for b in range(B)]
    kv_lens = [0 if b % 11 == 5 else 1 + (b * 53) % 400 for b in range(B)]
    c = P.Cache(43, q_lens, kv_lens, 8, 2, 64, 16, dtype, cache, behind=3).poison()
    for b in range(0, B - 1, 2):
        n = -(-min(kv_lens[b], kv_lens[b + 1]) // 16)
        c.table[b + 1, :n] = c.table[b, :n]
    # a place poisoned for one sequence and read by the other is cleared
    for x in (c.k, c.v):
        y = x.view(torch.uint8) if cache != "same" else x
        bad = (y == 0x7F) if cache != "same" else ~torch.isfinite(y)
        for b in range(1, B, 2):
            page, place = c.cells(b)
            z = y[page, place]
            z[bad[page, place]] = 0
            y[page, place] = z
    for hint in (max(q_lens), 0):
        out, lse = run_paged(c, True, hint)
        check_paged(c, out, lse, True)


@pytest.mark.parametrize("cache,dtype", [("same", "f16"), ("e4m3", "bf16"), ("e5m2", "f16")])
@pytest.mark.parametrize("group", [65, 127, 128, 129])
def test_large_groups(group, cache, dtype):
    c = P.Cache(44, [9, 30], [200, 131], group, 1, 128, 16, dtype, cache).poison()
    for hint in (0, 1):
        out, lse = run_paged(c, True, hint)
        check_paged(c, out, lse, True)


@pytest.mark.parametrize("hint,q_lens", [(1, [1, 1]), (0, [40, 70])])
def test_out_at_any_16_bytes(hint, q_lens):
    """An out that begins 16 bytes behind a 32-byte border."""
    c = P.Cache(42, q_lens, [900, 333], 8, 2, 128, 16, "bf16")
    d = c.to("cuda")
    q, _, _ = c.split(d["qkv"])
    room = torch.full((c.T * c.Hq * c.D + 16,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = room[8:-8].view(c.T, c.Hq, c.D)
    assert out.data_ptr() % 32 == 16
    _, lse = sfa.paged_attention(q, d["k"], d["v"], d["table"], d["lens"], d["cu"], max_q_len=hint, out=out,
                                 return_lse=True)
    check_paged(c, out.cpu(), lse.cpu(), True)
    assert (room[:8] == 9).all() and (room[-8:] == 9).all()


@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("hint,wide", [(1, False), (0, False), (0, True)])
def test_pages_out_of_range_are_absent(cache, hint, wide):
    c = P.Cache(21, [1, 70, 3], [90, 200, 64], 8, 2, 128, 16, "bf16", cache).poison()
    c.table[0, 2] = c.pages
    c.table[1, 0] = -1
    c.table[1, 5] = 1 << 30
    c.table[2] = -5                          # nothing left: +0 and -inf
    if wide:
        widen(c)
    out, lse = run_paged(c, True, hint)
    check_paged(c, out, lse, True)
    assert torch.isneginf(lse[-5:-2] if c.cu[-1] < c.T else lse[c.cu[2]:]).all()


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3"), ("bf16", "e5m2")])
@pytest.mark.parametrize("hint,wide", [(1, False), (0, False), (0, True)])
def test_large_scores_and_scales(dtype, cache, hint, wide):
    """Scores in the hundreds, growing along the keys (the running maximum
    moves at every step), rows of q of very different size."""
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
        out, lse = run_paged(c, True, hint, scale)
        check_paged(c, out, lse, True, scale)


def test_long_mixed_lengths_split_over_many_ranges():
    """Lengths from 1 to 30,000: tiles cut into many ranges next to whole ones."""
    c = P.Cache(23, [1] * 7, [30000, 1, 17, 2500, 64, 9000, 128], 8, 2, 64, 16, "f16").poison()
    out, lse = run_paged(c, True, 1)
    check_paged(c, out, lse, True)
    again, lse2 = run_paged(c, True, 1)
    assert torch.equal(out, again) and torch.equal(lse, lse2)      # nothing depends on timing


@pytest.mark.parametrize("hint", [1, 0])
def test_offsets_beyond_32_bits(hint):
    """Pools of more than 2^31 elements, the pages used at their far end."""
    H, D, page = 8, 128, 64
    pages = (1 << 31) // (H * D * page) + 40
    c = P.Cache(24, [2, 33], [100, 400], 16, H, D, page, "bf16")
    d = c.to("cuda")
    big = [torch.empty((pages, page, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    shift = pages - c.pages
    for x, n in zip(big, "kv"):
        x[shift:] = d[n]
        d[n] = x
    table = d["table"]
    d["table"] = torch.where(table >= 0, table + shift, table)
    out, lse = run_paged(c, True, hint, d=d)
    check_paged(c, out, lse, True)
    # the new tokens out of the far pages
    _, k, v = c.split(d["qkv"])
    sfa.paged_append(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"])
    ko, vo = sfa.paged_read(d["k"], d["v"], d["table"], d["lens"], d["cu"], c.T)
    assert torch.equal(ko, k) and torch.equal(vo, v)


def test_device_lists_that_lie_are_clamped():
    """Row lists and lengths beyond what the call was given touch nothing else."""
    c = P.Cache(25, [4, 4], [40, 40], 4, 2, 64, 16, "f16")
    d = c.to("cuda")
    d["cu"] = torch.tensor([-3, 5, 1 << 30], dtype=torch.int32, device="cuda")
    d["lens"] = torch.tensor([1 << 30, -4], dtype=torch.int32, device="cuda")
    q, k, v = c.split(d["qkv"])
    for hint in (1, 0):
        out = sfa.paged_attention(q, d["k"], d["v"], d["table"], d["lens"], d["cu"], max_q_len=hint)
        assert out.shape == q.shape
    sfa.paged_append(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"])
    sfa.paged_read(d["k"], d["v"], d["table"], d["lens"], d["cu"], c.T)
    torch.cuda.synchronize()
    assert sfa.sfa_get_last_error() == sfa.SFA_OK


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("cache,dtype,layout,page", [("same", "bf16", "NHD", 16), ("e4m3", "bf16", "HND", 32),
                                                     ("e5m2", "f16", "NHD", 24)])
def test_serving_run(cache, dtype, layout, page):
    """Prompts appended and attended to in chunks, then single tokens, over one
    cache; the result equals attention over the cache read back."""
    lens = [150, 37, 290]
    total = [n + 3 for n in lens]
    c = P.Cache(31, total, total, 8, 2, 128, page, dtype, cache, layout)
    d = c.to("cuda")
    q, k, v = c.split(d["qkv"])
    first = [int(x) for x in c.cu[:-1]]
    outs = torch.empty((c.T, 8, 128), dtype=P.TORCH[dtype], device="cuda")
    done = [0, 0, 0]
    while done != total:
        # chunks of up to 100 tokens of the prompt, then one token at a time
        n = [min(100, lens[b] - done[b]) if done[b] < lens[b] else min(1, total[b] - done[b]) for b in range(3)]
        at = torch.cat([torch.arange(first[b] + done[b], first[b] + done[b] + n[b]) for b in range(3)]).cuda()
        done = [x + y for x, y in zip(done, n)]
        cu = torch.tensor([0, n[0], n[0] + n[1], sum(n)], dtype=torch.int32, device="cuda")
        kv_lens = torch.tensor(done, dtype=torch.int32, device="cuda")
        sfa.paged_append(k[at], v[at], cu, d["k"], d["v"], d["table"], kv_lens, **kw(c, d))
        outs[at] = sfa.paged_attention(q[at], d["k"], d["v"], d["table"], kv_lens, cu, max_q_len=max(n), **kw(c, d))
    c.k, c.v = d["k"].cpu(), d["v"].cpu()
    for b in range(3):
        s = slice(first[b], first[b] + total[b])
        kk, there = c.values(c.k, c.scale_k, b)
        vv, _ = c.values(c.v, c.scale_v, b)
        ref = P.attend(c.split(c.qkv)[0][s].double(), kk, vv, there, True, 1 / math.sqrt(128))
        P.check(outs[s].cpu(), None, ref, dtype, total[b], f"sequence {b}")
    # the whole cache back, and prompt attention over it
    ko, vo = sfa.paged_read(d["k"], d["v"], d["table"], d["lens"], d["cu"], c.T, dtype=dtype, **kw(c, d))
    whole, lse = sfa.varlen_attention(q, ko, vo, d["cu"], d["cu"], return_lse=True)
    for b in range(3):
        s = slice(first[b], first[b] + total[b])
        ref = P.attend(c.split(c.qkv)[0][s].double(), ko[s].cpu().double(), vo[s].cpu().double(),
                       torch.ones(total[b], dtype=torch.bool), True, 1 / math.sqrt(128))
        P.check(whole[s].cpu(), lse[s].cpu(), ref, dtype, total[b], f"sequence {b}")


# ---------------------------------------------------------------- streams and graphs

def test_captured_step_follows_the_lengths():
    """One captured append + attention, replayed as the lengths on the device grow."""
    c = P.Cache(41, [1, 1, 1], [60, 200, 130], 8, 2, 128, 16, "bf16", "e4m3")
    d = c.to("cuda")
    q, k, v = c.split(d["qkv"])
    lens = d["lens"]
    final = lens.clone()
    lens -= 5
    out = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda")

    def step():
        lens.add_(1)
        sfa.paged_append(k, v, d["cu"], d["k"], d["v"], d["table"], lens, **kw(c, d))
        sfa.paged_attention(q, d["k"], d["v"], d["table"], lens, d["cu"], max_q_len=1, out=out, **kw(c, d))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        d["qkv"].mul_(0.9)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(lens, final)
    c.qkv, c.k, c.v = d["qkv"].cpu(), d["k"].cpu(), d["v"].cpu()
    check_paged(c, out.cpu(), torch.stack([P.attend(c.split(c.qkv)[0][b: b + 1].double(),
                *(c.values(p, s, b)[0] for p, s in ((c.k, c.scale_k), (c.v, c.scale_v))),
                torch.ones(c.kv_lens[b], dtype=torch.bool), True, 1 / math.sqrt(128))[1][0] for b in range(3)]).float(),
                True)


@pytest.mark.parametrize("q_lens,hint", [([1] * 6, 1), ([70, 31, 5], 0)])
def test_streams_and_graphs_do_not_share_a_workspace(q_lens, hint):
    kv_lens = [n + 700 * (b + 1) for b, n in enumerate(q_lens)]
    cases = [P.Cache(50 + i, q_lens, kv_lens, 16, 4, 128, 16, "f16") for i in range(2)]
    dev = [c.to("cuda") for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.empty((c.T, c.Hq, c.D), dtype=torch.float16, device="cuda") for c in cases]

    def call(i):
        c, d = cases[i], dev[i]
        sfa.paged_attention(c.split(d["qkv"])[0], d["k"], d["v"], d["table"], d["lens"], d["cu"],
                            max_q_len=hint, out=outs[i])
    graphs = []
    for i in range(2):
        call(i)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    want = [o.clone() for o in outs]
    for way in ("eager", "graph"):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    call(i) if way == "eager" else graphs[i].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), way
    for c, o in zip(cases, outs):
        for b in range(len(q_lens)):
            s = slice(int(c.cu[b]), int(c.cu[b + 1]))
            ref = P.attend(c.split(c.qkv)[0][s].double(), c.values(c.k, None, b)[0], c.values(c.v, None, b)[0],
                           torch.ones(kv_lens[b], dtype=torch.bool), True, 1 / math.sqrt(128))
            P.check(o[s].cpu(), None, ref, "f16", kv_lens[b], f"sequence {b}")
