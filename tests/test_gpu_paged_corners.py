"""Corners of the paged cache and of the attention over it on the GPU, against
plain 64-bit arithmetic."""
import math

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
