"""Attention of batches that share their first tokens, on the GPU, against plain 64-bit
arithmetic and against attention over each sequence's own pages; and runs of rotated
appends, windowed and shared attention as a serving program makes them."""
import ctypes
import math
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import sparse_attention_serving_sfa_gb300 as sfa
from tests import paged_testlib as P
from tests import parts_testlib as X
from tests.test_gpu_paged import kw, run_paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    sfa.build()
    sfa.load()


class Shared(P.Cache):
    """A cache whose sequences share first tokens in groups (groups: (sequences,
    shared tokens) in turn, from sequence `skip` on): the leader's pages, and for the
    others the same as far as they are whole; the rest of a shared page that goes on
    with own tokens is left to chance in all but the leader's."""

    def __init__(self, seed, q_lens, own, heads, kv_heads, dim, page, dtype="bf16", cache="same", layout="NHD",
                 groups=(), skip=0, **more):
        self.leader, self.shared = list(range(len(own))), [0] * len(own)
        self.cu_shared, self.shared_lens = [skip], []
        for n, length in groups:
            first = self.cu_shared[-1]
            for b in range(first, first + n):
                self.leader[b], self.shared[b] = first, length
            self.cu_shared.append(first + n)
            self.shared_lens.append(length)
        total = [a + b for a, b in zip(self.shared, own)]
        super().__init__(seed, q_lens, total, heads, kv_heads, dim, page, dtype, cache, layout, **more)
        for b, a in enumerate(self.leader):
            whole = self.shared[b] // page
            if a != b:
                self.table[b, :whole] = -9           # never looked at

    def cells(self, b):
        page, place = super().cells(b)
        a, n = self.leader[b], self.shared[b]
        if a != b and n:
            head = super().cells(a)
            page[:n], place[:n] = head[0][:n], head[1][:n]
        return page, place

    def lists(self, dev="cuda"):
        return tuple(torch.tensor(x, dtype=torch.int32, device=dev) for x in (self.cu_shared, self.shared_lens))


def run_shared(c, causal, hint, scale=0.0, d=None, **more):
    d = d or c.to("cuda")
    q, _, _ = c.split(d["qkv"])
    out = torch.full((c.T, c.Hq, c.D), 9.0, dtype=P.TORCH[c.dtype], device="cuda")
    lse = torch.full((c.T, c.Hq), 9.0, device="cuda")
    sfa.shared_prefix_attention(q, d["k"], d["v"], d["table"], d["lens"], d["cu"], *c.lists(), scale, causal,
                                max_q_len=hint, out=out, lse=lse, **kw(c, d), **more)
    torch.cuda.synchronize()
    assert sfa.sfa_get_last_error() == sfa.SFA_OK
    return out.cpu(), lse.cpu()


def check_shared(c, out, lse, causal, scale=0.0):
    scale = scale or 1 / math.sqrt(c.D)
    q, _, _ = c.split(c.qkv)
    for b, (n, L) in enumerate(zip(c.q_lens, c.kv_lens)):
        s = slice(int(c.cu[b]), int(c.cu[b + 1]))
        k, there = c.values(c.k, c.scale_k, b)
        v, _ = c.values(c.v, c.scale_v, b)
        j = torch.arange(L)[None, :]
        seen = there[None, :].expand(n, L)
        if causal:
            seen = seen & ((j <= torch.arange(n)[:, None] + L - n) | (j < c.shared[b]))
        ref = X.attend_seen(q[s].double(), k, v, seen, scale)
        P.check(out[s], lse[s], ref, c.dtype, max(1, L), f"sequence {b}")
    for x in (out, lse):
        assert torch.all(x[: c.cu[0]] == 9) and torch.all(x[c.cu[-1]:] == 9)


# q_lens, own tokens, heads, kv_heads, dim, page, groups, skip
SHAPES = [
    ([1], [1], 1, 1, 64, 16, [(1, 1)], 0),
    ([1] * 5, [1, 9, 200, 33, 1], 32, 8, 128, 16, [(5, 300)], 0),
    ([1] * 6, [5, 70, 3, 1, 12, 40], 16, 2, 64, 20, [(2, 999), (3, 50)], 1),           # one before, ends inside pages
    ([1] * 40, [1 + 7 * b % 90 for b in range(40)], 8, 1, 128, 64, [(37, 2000)], 2),   # rows of many tiles
    ([3, 0, 130, 1], [30, 5, 200, 1], 12, 4, 128, 32, [(4, 700)], 0),
    ([90, 257, 40], [90, 300, 400], 6, 2, 64, 24, [(2, 1111), (1, 64)], 0),            # groups of 3 heads
    ([2, 9, 4], [2, 9, 4], 5, 5, 128, 5, [(1, 77), (2, 13)], 0),
    ([40] * 7, [40] * 7, 32, 4, 64, 128, [(7, 4000)], 0),
    ([1] * 9, [1] * 9, 40, 8, 64, 16, [(0, 50), (4, 0), (3, 128), (0, 7)], 1),         # empty groups, nothing shared
    ([30, 2], [10, 1], 4, 2, 64, 16, [(2, 100)], 0),                                   # rows inside the shared part
]


@pytest.mark.parametrize("cache,layout,dtype", [("same", "NHD", "bf16"), ("same", "HND", "f16"),
                                                ("e4m3", "HND", "bf16"), ("e5m2", "NHD", "f16")])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shared_prefix(shape, cache, layout, dtype):
    q_lens, own, heads, kv_heads, dim, page, groups, skip = SHAPES[shape]
    c = Shared(300 + shape, q_lens, own, heads, kv_heads, dim, page, dtype, cache, layout, groups=groups, skip=skip,
               before=1, behind=2).poison()
    for causal in (True, False):
        for hint in (1, 0):
            out, lse = run_shared(c, causal, hint)
            check_shared(c, out, lse, causal)


@pytest.mark.parametrize("cache,dtype,page", [("same", "bf16", 16), ("same", "f16", 20), ("e4m3", "f16", 64), ("e5m2", "bf16", 12)])
@pytest.mark.parametrize("shape", [0, 1, 2, 4, 5, 6, 7, 8, 9])
def test_table_much_wider_than_the_sequences(shape, page, cache, dtype):
    """By what the table could hold there is much to share: a pass over the prefixes and
    one over the own tokens, on either kernel, the large tiles wherever there are more
    than a few rows."""
    q_lens, own, heads, kv_heads, dim, _, groups, skip = SHAPES[shape]
    c = Shared(400 + shape, q_lens, own, heads, kv_heads, dim, page, dtype, cache, groups=groups, skip=skip, behind=1).poison()
    c.table = torch.cat([c.table, torch.full((len(q_lens), (1 << 20) // page), -1, dtype=torch.int32)], 1)
    for hint in (max(q_lens), 1, 0):
        out, lse = run_shared(c, True, hint)
        check_shared(c, out, lse, True)
        again, lse2 = run_shared(c, True, hint)
        assert torch.equal(out, again) and torch.equal(lse, lse2)      # nothing depends on timing


@pytest.mark.parametrize("cache,dtype,dim", [("same", "bf16", 128), ("same", "f16", 64), ("e4m3", "bf16", 64), ("e5m2", "f16", 128)])
@pytest.mark.parametrize("q_lens,own,heads,kv_heads,groups", [
    ([1, 1, 1], [700, 3, 40], 8, 2, [(3, 6000)]),                   # few rows, either pass cut into many parts
    ([2, 1, 3], [2, 2500, 9], 5, 5, [(2, 9000), (1, 70)]),
    ([170] * 8, [170 + 9 * b for b in range(8)], 32, 8, [(8, 1500)]),  # more items than ranges
    ([900, 450], [900, 1450], 16, 4, [(2, 700)]),
    ([3, 9], [40, 30], 160, 1, [(2, 300)]),                         # a group of 160 heads
    ([1] * 70, [1 + 5 * b % 37 for b in range(70)], 4, 1, [(1, 40 + b) for b in range(66)]),  # many groups of one
])
def test_passes_of_any_size(q_lens, own, heads, kv_heads, groups, cache, dtype, dim):
    c = Shared(500, q_lens, own, heads, kv_heads, dim, 16, dtype, cache, groups=groups, before=1, behind=1).poison()
    narrow = c.table
    for wide in (False, True):
        if wide:
            c.table = torch.cat([narrow, torch.full((len(q_lens), 1 << 16), -1, dtype=torch.int32)], 1)
        for hint in (max(q_lens), 0):
            out, lse = run_shared(c, True, hint)
            check_shared(c, out, lse, True)


@pytest.mark.parametrize("cache,dtype", [("same", "bf16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("q_len,hint", [(1, 1), (21, 0)])
def test_equals_attention_over_own_pages(q_len, hint, cache, dtype):
    """With the shared tokens in every sequence's own list, both calls compute the same."""
    c = Shared(7, [q_len] * 12, [q_len + 5 * b for b in range(12)], 16, 4, 128, 16, dtype, cache, groups=[(7, 640), (5, 1600)])
    for b, a in enumerate(c.leader):
        whole = c.shared[b] // 16
        c.table[b, :whole] = c.table[a, :whole]
    d = c.to("cuda")
    out, lse = run_shared(c, True, hint, d=d)
    check_shared(c, out, lse, True)
    other, lse2 = run_paged(c, True, hint, d=d)
    # two roundings to 16 bits of P and one of the output on either side
    h = torch.finfo(P.TORCH[dtype]).eps / 2
    assert (out.double() - other.double()).abs().max() <= 4 * h * max(1.0, out.double().abs().max())
    assert (lse - lse2).abs().max() < 1e-4


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "e4m3"), ("bf16", "e5m2")])
@pytest.mark.parametrize("q_len,hint", [(1, 1), (40, 0)])
def test_one_side_outweighs_the_other(q_len, hint, dtype, cache):
    """Scores in the hundreds, in the shared part for some rows and in the own for
    others."""
    c = Shared(8, [q_len] * 6, [q_len + 40] * 6, 8, 2, 128, 16, dtype, cache, groups=[(6, 500)])
    q, _, _ = c.split(c.qkv)
    q *= torch.logspace(-6, 1.2, c.T).to(q.dtype)[:, None, None]
    if cache == "same":
        for b in range(6):
            page, place = c.cells(b)
            if b % 2:
                c.k[page[500:], place[500:]] *= 3
        c.k[c.cells(0)] *= 0.5
    for scale in (0.0, 1.0):
        out, lse = run_shared(c, True, hint, scale)
        check_shared(c, out, lse, True, scale)


@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("hint", [1, 0])
def test_pages_out_of_range_are_absent(cache, hint):
    c = Shared(9, [1, 30, 3, 2], [20, 90, 64, 2], 8, 2, 128, 16, "bf16", cache, groups=[(2, 100), (2, 40)]).poison()
    c.table[0, 2] = c.pages                 # of the first prefix
    c.table[1, 8] = -1                      # of the second sequence's own
    c.table[2] = -5                         # a prefix and own tokens, all gone
    c.table[3] = 1 << 30
    out, lse = run_shared(c, True, hint)
    check_shared(c, out, lse, True)
    assert torch.isneginf(lse[31:]).all()


def test_lists_that_lie_touch_nothing_else():
    c = Shared(10, [4, 4, 4], [40, 40, 40], 4, 2, 64, 16, "f16", groups=[(3, 20)])
    d = c.to("cuda")
    for cu, lens in (([-5, 1 << 30], [1 << 30]), ([2, 1], [7]), ([0, 3, 1, 99], [5, -5, 1 << 29]), ([9, 9], [9])):
        c.cu_shared, c.shared_lens = cu, lens
        for hint in (1, 0):
            run_shared(c, True, hint, d=d)


@pytest.mark.parametrize("hint", [1, 0])
def test_offsets_beyond_32_bits(hint):
    H, D, page = 8, 128, 64
    pages = (1 << 31) // (H * D * page) + 40
    c = Shared(24, [2, 33], [100, 400], 16, H, D, page, "bf16", groups=[(2, 600)])
    d = c.to("cuda")
    shift = pages - c.pages
    for n in "kv":
        x = torch.empty((pages, page, H, D), dtype=torch.bfloat16, device="cuda")
        x[shift:] = d[n]
        d[n] = x
    d["table"] = torch.where(d["table"] >= 0, d["table"] + shift, d["table"])
    out, lse = run_shared(c, True, hint, d=d)
    check_shared(c, out, lse, True)


def test_nothing_to_do():
    c = Shared(11, [0, 0], [5, 9], 4, 2, 64, 16, "f16", groups=[(2, 30)])
    out, lse = run_shared(c, True, 0)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_a_given_workspace():
    c = Shared(12, [1, 1, 5], [10, 20, 30], 8, 2, 64, 16, "f16", groups=[(3, 200)])
    n = sfa.paged_shared_workspace_size(3, c.T, 8, 2, 64)
    assert n > sfa.paged_workspace_size(3, c.T, 8, 2, 64)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")      # nothing in it needs clearing
    out, lse = run_shared(c, True, 0, workspace=ws)
    check_shared(c, out, lse, True)
    with pytest.raises(sfa.SfaError):
        run_shared(c, True, 0, workspace=ws[: n - 16])


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("cache,dtype,layout,page,interleaved", [("same", "bf16", "NHD", 16, False),
                                                                 ("e4m3", "bf16", "HND", 32, True),
                                                                 ("e5m2", "f16", "NHD", 24, False)])
def test_serving_run(cache, dtype, layout, page, interleaved):
    """A document appended once, then questions of different lengths behind it, then
    single tokens: keys rotated on the way in, one layer's queries over everything, the
    other's through a window; every step against plain arithmetic over the cache."""
    doc, asks, steps = 333, [40, 7, 90], 3
    c = Shared(31, [n + steps for n in asks], [n + steps for n in asks], 8, 2, 128, page, dtype, cache, layout,
               groups=[(3, doc)])
    for b in range(1, 3):
        whole = doc // page
        c.table[b, :whole] = c.table[0, :whole]
    d = c.to("cuda")
    freq = (10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)).float().cuda()
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn((doc, 12, 128), generator=g).to(P.TORCH[dtype]).cuda()
    one = torch.tensor([0, doc], dtype=torch.int32, device="cuda")
    for b in range(3):       # (each into its own copy of a page that goes on)
        sfa.paged_append_rotated(qkv[:, 8:10], qkv[:, 10:], one, d["k"], d["v"], d["table"][b: b + 1].contiguous(),
                                 one[1:], freq, interleaved=interleaved, **kw(c, d))
    q, k, v = c.split(d["qkv"])
    first = [int(x) for x in c.cu[:-1]]
    done = [0, 0, 0]
    for step in range(1 + steps):
        n = asks if step == 0 else [1, 1, 1]
        at = torch.cat([torch.arange(first[b] + done[b], first[b] + done[b] + n[b]) for b in range(3)]).cuda()
        done = [x + y for x, y in zip(done, n)]
        cu = torch.tensor([0, n[0], n[0] + n[1], sum(n)], dtype=torch.int32, device="cuda")
        lens = torch.tensor([doc + x for x in done], dtype=torch.int32, device="cuda")
        turned = sfa.paged_append_rotated(k[at], v[at], cu, d["k"], d["v"], d["table"], lens, freq, q=q[at],
                                          interleaved=interleaved, **kw(c, d))
        pos = [doc + done[b] - n[b] + i for b in range(3) for i in range(n[b])]
        X.check_rotated(turned.cpu(), *X.rotated(q[at].cpu(), pos, freq.cpu(), interleaved), dtype)
        whole = sfa.shared_prefix_attention(turned, d["k"], d["v"], d["table"], lens, cu, *c.lists(), max_q_len=max(n), **kw(c, d))
        near = sfa.paged_attention(turned, d["k"], d["v"], d["table"], lens, cu, max_q_len=max(n), window=100, sinks=4, **kw(c, d))
        c.k, c.v = d["k"].cpu(), d["v"].cpu()
        kv_lens, c.kv_lens = c.kv_lens, [doc + x for x in done]
        for b in range(3):
            s = slice(int(cu[b]), int(cu[b + 1]))
            L = doc + done[b]
            kk, vv = c.values(c.k, c.scale_k, b)[0], c.values(c.v, c.scale_v, b)[0]
            for got, seen in ((whole, X.window_mask(n[b], L, L, 0)), (near, X.window_mask(n[b], L, 100, 4))):
                ref = X.attend_seen(turned[s].cpu().double(), kk, vv, seen, 1 / math.sqrt(128))
                P.check(got[s].cpu(), None, ref, dtype, L, f"sequence {b}")
        c.kv_lens = kv_lens


# ---------------------------------------------------------------- streams, graphs, threads

def calls(c, d, freq, out):
    """What a decode step does: append, one layer through a window, one behind the prefix."""
    q, k, v = c.split(d["qkv"])
    sfa.paged_append_rotated(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"], freq, q=q, q_out=out[0], **kw(c, d))
    sfa.paged_attention(out[0], d["k"], d["v"], d["table"], d["lens"], d["cu"], max_q_len=max(c.q_lens), out=out[1],
                        window=50, sinks=3, **kw(c, d))
    sfa.shared_prefix_attention(out[0], d["k"], d["v"], d["table"], d["lens"], d["cu"], *d["lists"],
                                max_q_len=max(c.q_lens), out=out[2], **kw(c, d))


def test_the_interpreter_lock_is_let_go():
    """While the library runs, other Python threads can: its entry points, stood in for
    by the function that tells whether the calling thread holds the lock."""
    lib, native = sfa.load(), sfa._native()

    def address(f):
        return ctypes.cast(f, ctypes.c_void_p).value
    held = address(ctypes.pythonapi.PyGILState_Check)
    c, d, freq, out = setup(3)
    q, k, v = c.split(d["qkv"])
    native.bind_more(held, held, held, held, address(lib.paged_shared_workspace_size))
    try:                                    # status 1 (held) would raise
        calls(c, d, freq, out)
        sfa.varlen_attention(q, k, v, d["cu"], d["cu"], window=5)
    finally:
        native.bind_more(*[address(f) for f in (lib.paged_append_rotated, lib.paged_run_window, lib.varlen_run_window,
                                                lib.paged_run_shared, lib.paged_shared_workspace_size)])


def setup(i, q_len=1, cache="same", dtype="f16"):
    n = 9
    c = Shared(50 + i, [q_len + (b % 3 if q_len > 1 else 0) for b in range(n)], [q_len + 9 * b + 2 for b in range(n)], 16, 4, 128, 16,
               dtype, cache, groups=[(5, 700), (3, 90)], skip=1)
    for b, a in enumerate(c.leader):
        whole = c.shared[b] // 16
        c.table[b, :whole] = c.table[a, :whole]
    d = c.to("cuda")
    d["lists"] = c.lists()
    freq = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda()
    out = [torch.zeros((c.T, 16, 128), dtype=P.TORCH[dtype], device="cuda") for _ in range(3)]
    return c, d, freq, out


@pytest.mark.parametrize("q_len,cache", [(1, "same"), (1, "e4m3"), (33, "same"), (33, "e5m2")])
def test_streams_graphs_and_threads(q_len, cache):
    """Side by side on streams, as graphs replayed side by side, and from threads:
    every call gets what it gets alone."""
    sets = [setup(i, q_len, cache) for i in range(3)]
    streams = [torch.cuda.Stream() for _ in sets]
    graphs = []
    for s in sets:
        calls(*s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls(*s)
        graphs.append(graph)
    want = []
    for s in sets:
        calls(*s)
        torch.cuda.synchronize()
        want.append([x.clone() for x in s[3]])

    def thread(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(10):
                calls(*sets[i])
        streams[i].synchronize()
    for way in ("streams", "graphs", "threads", "given streams"):
        for s in sets:
            for x in s[3]:
                x.zero_()
        torch.cuda.synchronize()
        if way == "threads":
            with ThreadPoolExecutor(3) as pool:
                list(pool.map(thread, range(3)))
        else:
            for _ in range(10):
                for i, stream in enumerate(streams):
                    if way == "given streams":
                        c, d, freq, out = sets[i]
                        q, k, v = c.split(d["qkv"])
                        sfa.paged_append_rotated(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"], freq, q=q,
                                                 q_out=out[0], stream=stream, **kw(c, d))
                        sfa.paged_attention(out[0], d["k"], d["v"], d["table"], d["lens"], d["cu"], max_q_len=max(c.q_lens),
                                            out=out[1], window=50, sinks=3, stream=stream, **kw(c, d))
                        sfa.shared_prefix_attention(out[0], d["k"], d["v"], d["table"], d["lens"], d["cu"], *d["lists"],
                                                    max_q_len=max(c.q_lens), out=out[2], stream=stream, **kw(c, d))
                        continue
                    with torch.cuda.stream(stream):
                        calls(*sets[i]) if way == "streams" else graphs[i].replay()
        torch.cuda.synchronize()
        for s, w in zip(sets, want):
            for x, y in zip(s[3], w):
                assert torch.equal(x, y), way
    assert sfa.sfa_get_last_error() == sfa.SFA_OK


@pytest.mark.parametrize("wide", [False, True])
def test_captured_step_follows_the_lists(wide):
    """One captured step, replayed as lengths, groups and shared lengths change on the
    device; with a wide table the shared tokens have a pass of their own."""
    c, d, freq, out = setup(9, 1, "same", "bf16")
    if wide:
        room = torch.full((9, 1 << 15), -1, dtype=torch.int32)
        c.table = torch.cat([c.table, room], 1)
        d["table"] = c.table.cuda()
    final = d["lens"].clone()
    d["lens"] -= 4

    def step():
        d["lens"].add_(1)
        calls(c, d, freq, out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        d["qkv"].mul_(0.9)
        graph.replay()
    # the first group ends earlier and one sequence less is in the second
    d["lists"][0].copy_(torch.tensor([1, 6, 8], dtype=torch.int32))
    d["lists"][1].copy_(torch.tensor([333, 64], dtype=torch.int32))
    d["lens"].sub_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(d["lens"], final)
    c.k, c.v = d["k"].cpu(), d["v"].cpu()
    lens = [0] + [333] * 5 + [64] * 2 + [0]
    for b in range(9):
        L = c.kv_lens[b]
        own = P.Cache.cells(c, b)
        at = tuple(x.clone() for x in own)
        a = 1 if b < 6 else 6
        if lens[b]:
            lead = P.Cache.cells(c, a)
            for x, y in zip(at, lead):
                x[: lens[b]] = y[: lens[b]]
        kk, vv = c.k[at].double(), c.v[at].double()
        for got, keys, seen in ((out[2], (kk, vv), X.window_mask(1, L, L, 0)),
                                (out[1], (c.k[own].double(), c.v[own].double()), X.window_mask(1, L, 50, 3))):
            ref = X.attend_seen(out[0][b: b + 1].cpu().double(), *keys, seen, 1 / math.sqrt(128))
            P.check(got[b: b + 1].cpu(), None, ref, "bf16", L, f"sequence {b}")
