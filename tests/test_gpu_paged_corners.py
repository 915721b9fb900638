"""Corners of the paged cache and of the attention over it on the GPU, against
plain 64-bit arithmetic."""
import ctypes
import math
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import sparse_attention_serving_sfa_gb300 as sfa
from tests import paged_testlib as P
from tests.test_gpu_paged import check_paged, kw, raw, run_paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    sfa.build()
    sfa.load()


@pytest.mark.parametrize("cache,dtype,dim", [("same", "f16", 128), ("same", "f16", 64), ("same", "bf16", 128),
                                             ("e4m3", "bf16", 128), ("e5m2", "f16", 64)])
@pytest.mark.parametrize("q_lens,kv_lens,hint", [([1], [1100], 1), ([1, 5, 2], [300, 5000, 2], 1),
                                                 ([70, 33], [500, 1300], 0), ([150, 90], [500, 1300], 0)])
def test_many_small_weights_next_to_large_ones(q_lens, kv_lens, hint, cache, dtype, dim):
    """Every 16th key weighs 2^25 times each of the others and has the value 0: the
    output is made of the small weights alone (2^-25 is half fp16's smallest step)."""
    c = P.Cache(61, q_lens, kv_lens, 8, 2, dim, 16, dtype, cache)
    c.scale_k = c.scale_v = None                       # codes as they are
    q, _, _ = c.split(c.qkv)
    q.zero_()
    q[:, :, 0] = 5
    k, v = torch.zeros(c.k.shape), torch.full(c.v.shape, 256.0)
    for b in range(len(q_lens)):
        page, place = (x[::16] for x in c.cells(b))
        k[page, place, :, 0] = 5                       # q.k = 25
        v[page, place] = 0
    c.k, c.v = k.to(c.k.dtype), v.to(c.v.dtype)
    out, lse = run_paged(c, True, hint, math.log(2))
    check_paged(c, out, lse, True, math.log(2))


@pytest.mark.parametrize("cache,dtype,dim", [("e4m3", "bf16", 128), ("e4m3", "f16", 64), ("e5m2", "bf16", 64),
                                             ("e5m2", "f16", 128)])
@pytest.mark.parametrize("hint", [1, 0])
def test_scales_whose_product_underflows(hint, cache, dtype, dim):
    """scale * scale_k is 0 in fp32: visible keys weigh the same, masked ones and
    those of a missing page nothing."""
    c = P.Cache(62, [3, 150, 40], [200, 333, 40], 8, 2, dim, 16, dtype, cache)
    c.scale_k *= 1e-30
    c.table[1, 3] = c.pages
    for causal in (True, False):
        out, lse = run_paged(c, causal, hint, 1e-20)
        check_paged(c, out, lse, causal, 1e-20)


@pytest.mark.parametrize("cache,dtype,layout", [("same", "bf16", "NHD"), ("e4m3", "f16", "HND")])
@pytest.mark.parametrize("T,behind", [(12, 0), (15, 3)])
def test_lists_are_read_as_clamped(T, behind, cache, dtype, layout):
    """Rows said to lie behind the last, lengths behind the table or negative: append,
    read and attention take the lists as clamped, and so mean the same tokens."""
    # what the lists come to
    c = P.Cache(63, [4, 2, 6], [40, 0, 96], 8, 2, 64, 16, dtype, cache, layout, behind=behind)
    c.table = c.table[:, :6].contiguous()               # 96 tokens and no more
    d = c.to("cuda")
    # (the rows behind the last sequence are no rows of it, unless the list says so)
    d["cu"] = torch.tensor([-2, 4, 6, 12 if behind else 19], dtype=torch.int32, device="cuda")
    d["lens"] = torch.tensor([40, -7, 99], dtype=torch.int32, device="cuda")
    assert c.T == T
    _, k, v = c.split(d["qkv"])
    sfa.paged_append(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"], **kw(c, d))
    for x, n, scale in ((1, "k", c.scale_k), (2, "v", c.scale_v)):
        pool = getattr(c, n)
        w = raw(pool).clone()
        w = w.transpose(1, 2) if layout == "HND" else w
        for b in (0, 2):
            new = c.split(c.qkv)[x][c.cu[b]: c.cu[b + 1]]
            page, place = (y[-c.q_lens[b]:] for y in c.cells(b))
            w[page, place] = (new.contiguous().view(torch.int16) if cache == "same" else
                              P.nearest_code(new.double() / scale.double().view(1, -1, 1), cache))
        w = w.transpose(1, 2) if layout == "HND" else w
        assert torch.equal(raw(d[n]), w)
        setattr(c, n, d[n].cpu())
    got = sfa.paged_read(d["k"], d["v"], d["table"], d["lens"], d["cu"], c.T, dtype=dtype, **kw(c, d))
    h = torch.finfo(P.TORCH[dtype]).eps / 2
    for x, pool, scale in ((got[0].cpu(), c.k, c.scale_k), (got[1].cpu(), c.v, c.scale_v)):
        assert torch.all(x[4:6] == 0)
        for b in (0, 2):
            want = c.values(pool, scale, b)[0][c.kv_lens[b] - c.q_lens[b]:]
            err = (x[c.cu[b]: c.cu[b + 1]].double() - want).abs()
            assert torch.all(err <= (h + 2.0 ** -24) * (1 + h) * want.abs() + 2.0 ** -25)
    for hint in (1, 0):
        out, lse = run_paged(c, True, hint, d=d)
        check_paged(c, out, lse, True)


@pytest.mark.parametrize("cache,dim", [("e4m3", 128), ("e5m2", 64)])
@pytest.mark.parametrize("hint", [1, 0])
def test_small_elements_of_a_row_beside_a_large_one(hint, cache, dim):
    """bf16 rows over an 8-bit cache whose scores come from elements 2^-24 of the
    largest, which meets zeros."""
    c = P.Cache(64, [2, 90, 60], [300, 333, 500], 8, 2, dim, 16, "bf16", cache)
    q, _, _ = c.split(c.qkv)
    q *= 2.0 ** -24
    q[:, :, 0] = 1
    c.k.view(torch.uint8)[..., 0] = 0
    out, lse = run_paged(c, True, hint, 2.0 ** 23)
    check_paged(c, out, lse, True, 2.0 ** 23)


def test_the_interpreter_lock_is_let_go():
    """While the library runs, other Python threads can: its entry points, stood in
    for by the function that tells whether the calling thread holds the lock."""
    lib, native = sfa.load(), sfa._native()
    held = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    size = ctypes.cast(lib.paged_workspace_size, ctypes.c_void_p).value
    c = P.Cache(65, [3, 4], [20, 30], 4, 2, 64, 16, "f16")
    d = c.to("cuda")
    q, k, v = c.split(d["qkv"])
    pools = d["k"], d["v"], d["table"], d["lens"]
    native.bind(held, held, held, size, held)
    try:                                    # status 1 (held) would raise
        sfa.paged_append(k, v, d["cu"], *pools)
        sfa.paged_read(*pools, d["cu"], c.T)
        sfa.paged_attention(q, *pools, d["cu"])
        sfa.varlen_attention(q, k, v, d["cu"], d["cu"])
    finally:
        native.bind(*[ctypes.cast(f, ctypes.c_void_p).value for f in
                      (lib.paged_append, lib.paged_read, lib.paged_run, lib.paged_workspace_size, lib.varlen_run)])


@pytest.mark.parametrize("hint", [1, 0])
def test_calls_from_several_threads(hint):
    """Threads with a stream each: every one gets what it gets alone."""
    cases = [P.Cache(70 + i, [1 + 40 * i, 70, 9], [900, 400 + i, 33], 8, 2, 128, 16, "f16", "e4m3") for i in range(4)]
    dev = [c.to("cuda") for c in cases]
    for c, d in zip(cases, dev):
        sfa.paged_append(*c.split(d["qkv"])[1:], d["cu"], d["k"], d["v"], d["table"], d["lens"], **kw(c, d))
        c.k, c.v = d["k"].cpu(), d["v"].cpu()
    torch.cuda.synchronize()

    def work(i):
        c, d = cases[i], dev[i]
        q, k, v = c.split(d["qkv"])
        stream = torch.cuda.Stream()
        got = []
        with torch.cuda.stream(stream):
            for _ in range(30):
                sfa.paged_append(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"], **kw(c, d))
                got.append(sfa.paged_attention(q, d["k"], d["v"], d["table"], d["lens"], d["cu"], max_q_len=hint,
                                               return_lse=True, **kw(c, d)))
        stream.synchronize()
        return got
    with ThreadPoolExecutor(len(cases)) as pool:
        results = list(pool.map(work, range(len(cases))))
    for c, got in zip(cases, results):
        check_paged(c, got[0][0].cpu(), got[0][1].cpu(), True)
        for out, lse in got[1:]:
            assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("cache,dtype,layout,page", [("e4m3", "bf16", "NHD", 16), ("e5m2", "f16", "HND", 20)])
@pytest.mark.parametrize("have", ["", "k", "v"])
def test_eight_bits_without_scales(have, cache, dtype, layout, page):
    """No scale, or one of the two: the codes of the other are the values."""
    c = P.Cache(66, [5, 180, 90], [70, 300, 400], 8, 2, 128, page, dtype, cache, layout)
    for n in "kv":
        if n not in have:
            setattr(c, f"scale_{n}", None)
            pool = getattr(c, n)
            setattr(c, n, (pool.float() / 64).to(pool.dtype))       # values of ordinary size
    d = c.to("cuda")
    _, k, v = c.split(d["qkv"])
    sfa.paged_append(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"], **kw(c, d))
    for x, n, scale in ((1, "k", c.scale_k), (2, "v", c.scale_v)):
        w = raw(getattr(c, n)).clone()
        w = w.transpose(1, 2) if layout == "HND" else w
        for b, m in enumerate(c.q_lens):
            new = c.split(c.qkv)[x][c.cu[b]: c.cu[b + 1]].double()
            page_, place = (y[-m:] for y in c.cells(b))
            w[page_, place] = P.nearest_code(new if scale is None else new / scale.double().view(1, -1, 1), cache)
        assert torch.equal(raw(d[n]), w.transpose(1, 2) if layout == "HND" else w)
        setattr(c, n, d[n].cpu())
    got = sfa.paged_read(d["k"], d["v"], d["table"], d["lens"], d["cu"], c.T, dtype=dtype, **kw(c, d))
    h = torch.finfo(P.TORCH[dtype]).eps / 2
    for x, pool, scale in ((got[0].cpu(), c.k, c.scale_k), (got[1].cpu(), c.v, c.scale_v)):
        for b, m in enumerate(c.q_lens):
            want = c.values(pool, scale, b)[0][c.kv_lens[b] - m:]
            err = (x[c.cu[b]: c.cu[b + 1]].double() - want).abs()
            assert torch.all(err <= (h + 2.0 ** -24) * (1 + h) * want.abs() + 2.0 ** -25)
    for hint in (1, 0):
        out, lse = run_paged(c, True, hint, d=d)
        check_paged(c, out, lse, True)


@pytest.mark.parametrize("hint,page", [(1, 64), (0, 64), (0, 20)])
def test_eight_bit_pools_beyond_32_bits(hint, page):
    """Pools of more than 2^32 codes, the pages used at their far end."""
    H, D = 8, 128
    c = P.Cache(67, [2, 70], [100, 400], 32, H, D, page, "bf16", "e4m3")
    d = c.to("cuda")
    pages = (1 << 32) // (H * D * page) + c.pages + 1
    shift = pages - c.pages
    for n in "kv":
        big = torch.empty((pages, page, H, D), dtype=torch.uint8, device="cuda")
        big[shift:] = d[n].view(torch.uint8)
        d[n] = big.view(torch.float8_e4m3fn)
    d["table"] = torch.where(d["table"] >= 0, d["table"] + shift, d["table"])
    _, k, v = c.split(d["qkv"])
    sfa.paged_append(k, v, d["cu"], d["k"], d["v"], d["table"], d["lens"], **kw(c, d))
    c.k, c.v = (d[n].view(torch.uint8)[shift:].view(torch.float8_e4m3fn).cpu() for n in "kv")
    ko, vo = sfa.paged_read(d["k"], d["v"], d["table"], d["lens"], d["cu"], c.T, **kw(c, d))
    for x, new, scale in ((ko, k, c.scale_k), (vo, v, c.scale_v)):
        y = P.nearest_code(new.cpu().double() / scale.double().view(1, -1, 1), "e4m3").view(torch.float8_e4m3fn)
        want = (y.float() * scale.view(1, -1, 1)).bfloat16()
        assert torch.equal(x.cpu(), want)
    out, lse = run_paged(c, True, hint, d=d)
    check_paged(c, out, lse, True)


@pytest.mark.parametrize("q_lens", [[1, 1], [200, 130]])
def test_a_scale_below_fp32_is_not_the_default(q_lens):
    """Every visible key weighs the same."""
    c = P.Cache(68, q_lens, [300, 150], 8, 2, 64, 16, "bf16")
    out, lse = run_paged(c, True, max(q_lens), 1e-50)
    check_paged(c, out, lse, True, 1e-50)
    d = c.to("cuda")
    q, k, v = c.split(d["qkv"])
    out, lse = (x.cpu() for x in sfa.varlen_attention(q, k, v, d["cu"], d["cu"], 1e-50, return_lse=True))
    q, k, v = (x.double() for x in c.split(c.qkv))
    for b, n in enumerate(q_lens):
        s = slice(int(c.cu[b]), int(c.cu[b + 1]))
        P.check(out[s], lse[s], P.attend(q[s], k[s], v[s], torch.ones(n, dtype=torch.bool), True, 1e-50), "bf16", n)
