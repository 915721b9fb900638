"""Windows, shared prefixes and rotated appends write what they say and nothing beside it,
also with lists that lie."""
import pytest
import torch

import sparse_attention_serving_sfa_gb300 as sfa
from tests import guard_testlib as G
from tests import paged_testlib as P
from tests.test_gpu_paged import kw, widen
from tests.test_gpu_shared import Shared, check_shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    sfa.build()
    sfa.load()


def int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# cu_seqlens_q of three sequences (None: as they are)
ROWS = [None, [-3, 5, 1 << 30, 7], [9, 2, 1, 0], [0, 0, 0, -1], [1 << 30, 0, 1 << 29, 1 << 30]]
LENGTHS = [None, [1 << 30, -4, 17]]
GROUPS = [([0, 3], [20]), ([-5, 1 << 30], [1 << 30]), ([2, 1], [7]), ([0, 3, 1, 99], [5, -5, 1 << 29]), ([9, 9], [9]),
          ([3, 0, 3, 0, 3], [30, 1 << 30, 1, -1]), ([0, 1, 2, 3], [1 << 30, 0, 40]), ([-1, -1, 0, 0, 1 << 30], [3, 4, 5, 6])]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("rows", [4, 150])
@pytest.mark.parametrize("cache,dtype,dim,page", [("same", "f16", 64, 16), ("same", "bf16", 128, 20), ("e4m3", "bf16", 128, 16),
                                                  ("e5m2", "f16", 64, 12)])
def test_lists_that_lie(cache, dtype, dim, page, rows, wide):
    c = Shared(10, [rows] * 3, [rows + 40, rows, rows + 3], 8, 2, dim, page, dtype, cache, groups=[(3, 400)])
    if wide:
        widen(c)
    took = set()
    for cu in ROWS:
        for lens in LENGTHS:
            d = c.to("cuda")
            d["cu"] = d["cu"] if cu is None else int32(cu)
            d["lens"] = d["lens"] if lens is None else int32(lens)
            for hint in (1, 0):
                for groups in GROUPS:
                    took.add(G.attend(c, sfa.shared_prefix_attention, [int32(x) for x in groups], d=d, max_q_len=hint)[2])
                for window, sinks in ((1, 0), (30, 5), (200, 300)):
                    took.add(G.attend(c, sfa.paged_attention, d=d, max_q_len=hint, window=window, sinks=sinks)[2])
    # (few rows over a table as wide as the sequences take the kernel for few rows alone)
    assert took == ({False, True} if rows > 4 or wide else {False}), took


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("cache,dtype", [("same", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("q_lens,own", [([1, 1, 5], [10, 20, 30]), ([200, 3, 170], [200, 90, 500])])
def test_shared_prefix_within_its_buffers(q_lens, own, cache, dtype, wide):
    c = Shared(12, q_lens, own, 8, 2, 64, 16, dtype, cache, groups=[(2, 500)], before=3, behind=2).poison()
    if wide:
        widen(c)
    for hint in (max(q_lens), 0):
        out, lse, _ = G.attend(c, sfa.shared_prefix_attention, c.lists(), max_q_len=hint)
        check_shared(c, out, lse, True)


@pytest.mark.parametrize("cache,dtype", [("same", "bf16"), ("e4m3", "f16"), ("e5m2", "bf16")])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_append_lists_that_lie(cache, dtype, interleaved):
    """Tokens go to places of pages that the table names, or nowhere; rows of no sequence are
    left as they were."""
    c = P.Cache(5, [9, 4, 20], [40, 9, 300], 4, 2, 64, 12, dtype, cache, before=2, behind=3)
    freq = (10000.0 ** (-torch.arange(0, 48, 2) / 48)).float().cuda()
    for table in (None, -1, 1 << 30):
        for cu in ROWS:
            for lens in LENGTHS:
                g, d = G.Guard(), c.to("cuda")
                k, v, out = g.copy(c.k), g.copy(c.v), g.tensor((c.T, 4, 64), P.TORCH[dtype], value=9.0)
                q, new_k, new_v = c.split(d["qkv"])
                pages = d["table"] if table is None else torch.full_like(d["table"], table)
                row_list = d["cu"] if cu is None else int32(cu)
                sfa.paged_append_rotated(new_k, new_v, row_list, k, v, pages, d["lens"] if lens is None else int32(lens), freq, q=q,
                                         q_out=out, interleaved=interleaved, **kw(c, d))
                g.check()
                if table is not None:
                    assert torch.equal(k.view(torch.uint8).cpu(), c.k.view(torch.uint8))
                    assert torch.equal(v.view(torch.uint8).cpu(), c.v.view(torch.uint8))
                first, last = (min(max(int(x), 0), c.T) for x in (row_list[0], row_list[-1]))
                if cu is None:
                    assert (out[:first] == 9).all() and (out[last:] == 9).all()
