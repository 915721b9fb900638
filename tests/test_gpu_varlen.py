"""Attention over packed prompts on the GPU against plain 64-bit arithmetic."""
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


def cumulative(lens, before=0):
    return torch.tensor([before + sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32)


def problem(seed, q_lens, k_lens, heads, kv_heads, dim, dtype, before=0, behind=0):
    g = torch.Generator().manual_seed(seed)
    t = P.TORCH[dtype]
    cq, ck = cumulative(q_lens, before), cumulative(k_lens, before)
    q = torch.randn((int(cq[-1]) + behind, heads, dim), generator=g).to(t)
    kv = torch.randn((int(ck[-1]) + behind, 2 * kv_heads, dim), generator=g).to(t)
    return q, kv[:, :kv_heads], kv[:, kv_heads:], cq, ck


def run(q, k, v, cq, ck, causal, hint=0, scale=0.0):
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    sfa.varlen_attention(q.cuda(), k.cuda(), v.cuda(), cq.cuda(), ck.cuda(), scale, causal,
                         max_q_len=hint, out=out, lse=lse)
    torch.cuda.synchronize()
    assert sfa.sfa_get_last_error() == sfa.SFA_OK
    return out.cpu(), lse.cpu()


def check(q, k, v, cq, ck, out, lse, causal, dtype, scale=0.0):
    scale = scale or 1 / math.sqrt(q.shape[-1])
    for b in range(len(cq) - 1):
        s, t = slice(int(cq[b]), int(cq[b + 1])), slice(int(ck[b]), int(ck[b + 1]))
        n = t.stop - t.start
        ref = P.attend(q[s].double(), k[t].double(), v[t].double(), torch.ones(n, dtype=torch.bool), causal, scale)
        P.check(out[s], lse[s], ref, dtype, max(1, n), f"sequence {b}")
    for x in (out, lse):
        assert torch.all(x[: cq[0]] == 9) and torch.all(x[cq[-1]:] == 9)


SHAPES = [
    # q_lens, k_lens (None: the same), heads, kv heads, dim
    ([1], None, 1, 1, 64),
    ([1, 2, 0, 64, 65, 127], None, 4, 4, 128),
    ([128, 129, 1, 255, 256, 257], None, 8, 2, 64),
    ([500, 31, 1000], None, 32, 8, 128),
    ([333, 90], None, 10, 2, 128),                       # groups of 5
    ([200, 7], None, 3, 1, 64),
    ([77, 300], None, 64, 1, 128),                       # 64 heads share a kv head
    ([30], None, 200, 1, 64),                            # a group of 200
    ([1, 1, 1], [900, 1, 130], 16, 4, 128),              # single rows
    ([40, 260, 5, 3], [1500, 100, 0, 2], 8, 2, 128),     # other numbers of keys, empty rows, none
    ([2048], None, 2, 1, 128),
    ([40], [4000], 2, 1, 128),                           # few tiles, long keys
    ([9, 33], [2500, 100], 6, 2, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_varlen_attention(shape, dtype):
    q_lens, k_lens, heads, kv_heads, dim = SHAPES[shape]
    p = problem(200 + shape, q_lens, k_lens or q_lens, heads, kv_heads, dim, dtype, before=3, behind=2)
    for causal in (True, False):
        for hint in (0, 1):
            out, lse = run(*p, causal, hint)
            check(*p, out, lse, causal, dtype)


@pytest.mark.parametrize("hint", [0, 1])
def test_neighbours_never_matter(hint):
    """NaN and infinities in the rows of no sequence and in the sequence next
    door stay there."""
    q, k, v, cq, ck = problem(7, [100, 37, 200], [100, 37, 200], 4, 2, 128, "bf16", before=5, behind=9)
    want, wl = run(q, k, v, cq, ck, True, hint)
    for x in (q, k, v):
        x[:5] = float("nan")
        x[100 + 5: 137 + 5] = float("inf")
        x[-9:] = float("nan")
    out, lse = run(q, k, v, cq, ck, True, hint)
    for s in (slice(5, 105), slice(142, 342)):
        assert torch.equal(out[s], want[s]) and torch.equal(lse[s], wl[s])


def test_large_scores():
    p = problem(8, [300, 41], [300, 41], 4, 2, 64, "f16")
    p[1].mul_(torch.linspace(0.01, 6, p[1].shape[0]).half()[:, None, None])
    for scale in (1.0, 1e-6):
        out, lse = run(*p, True, 0, scale)
        check(*p, out, lse, True, "f16", scale)


def test_no_keys_at_all():
    q = torch.randn(5, 4, 64).half()
    k = torch.empty(0, 2, 64).half()
    cq, ck = torch.tensor([0, 5], dtype=torch.int32), torch.tensor([0, 0], dtype=torch.int32)
    for hint in (0, 1):
        out, lse = run(q, k, k, cq, ck, True, hint)
        assert torch.all(out == 0) and torch.isneginf(lse).all()


def test_no_rows():
    q = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    k = torch.randn(6, 2, 64, device="cuda").half()
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert sfa.varlen_attention(q, k, k, cu, cu).shape == (0, 4, 64)


def test_other_stream_and_given_outputs():
    q, k, v, cq, ck = (x.cuda() for x in problem(9, [150, 60], [150, 60], 8, 2, 128, "bf16"))
    want, wl = sfa.varlen_attention(q, k, v, cq, ck, return_lse=True)
    ws = torch.empty(sfa.varlen_workspace_size(2, 210, 8, 2, 128), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(210, 8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sfa.varlen_attention(q, k, v, cq, ck, out=out, lse=lse, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
