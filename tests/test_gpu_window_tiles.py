"""Windows with sinks on the tensor-core kernel: enough rows that it is the one that runs,
whatever the window, against plain 64-bit arithmetic."""
import pytest
import torch

import sparse_attention_serving_sfa_gb300 as sfa
from tests import guard_testlib as G
from tests import paged_testlib as P
from tests import parts_testlib as X
from tests.test_gpu_paged import widen
from tests.test_gpu_window import check_window, masks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    sfa.build()
    sfa.load()


def run(c, window, sinks, scale=0.0, hint=0):
    out, lse, tiles = G.attend(c, sfa.paged_attention, scale=scale, window=window, sinks=sinks, max_q_len=hint)
    assert tiles, "the kernel for few rows ran"
    check_window(c, out, lse, window, sinks, scale)


CACHES = [("same", "NHD", "bf16"), ("same", "HND", "f16"), ("e4m3", "HND", "bf16"), ("e5m2", "NHD", "f16"),
          ("e4m3", "NHD", "f16"), ("e5m2", "HND", "bf16")]
WINDOWS = [(1, 0), (1, 1), (7, 3), (64, 0), (100, 130), (128, 128), (333, 4), (5, 300), (1000, 1)]
# q_lens, kv_lens, heads, kv_heads, dim, page
SHAPES = [
    ([1, 0, 1, 210, 1], [77, 5, 0, 300, 640], 16, 2, 128, 5),           # single tokens beside a chunk
    ([1] * 5 + [150], [1000, 3, 129, 64, 1, 2500], 40, 8, 64, 24),      # groups of 5
    ([4, 1, 3, 200], [500, 1, 3, 200], 8, 2, 128, 64),
    ([2, 9, 300], [1, 4, 299], 4, 4, 64, 3),                            # rows before the first key
    ([17, 130, 1], [300, 130, 700], 12, 4, 128, 32),
    ([40, 90], [333, 1111], 32, 1, 128, 64),
    ([300], [515], 10, 2, 128, 20),
    ([30, 50], [200, 131], 128, 1, 128, 16),                            # a token a tile
    ([30, 40], [400, 90], 65, 1, 64, 8),
    ([600, 1, 77], [600, 1300, 3000], 3, 3, 128, 128),
]


@pytest.mark.parametrize("cache,layout,dtype", CACHES)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_window(shape, cache, layout, dtype):
    q_lens, kv_lens, heads, kv_heads, dim, page = SHAPES[shape]
    for window, sinks in WINDOWS:
        c = P.Cache(600 + shape, q_lens, kv_lens, heads, kv_heads, dim, page, dtype, cache, layout, before=1, behind=2).poison()
        X.poison_unseen(c, masks(c, window, sinks))
        run(c, window, sinks)


@pytest.mark.parametrize("cache,layout,dtype", CACHES)
@pytest.mark.parametrize("page", [8, 16, 20, 24, 64, 160])
def test_missing_pages_inside_the_window(page, cache, layout, dtype):
    """Pages that a row would see but the table does not name, of sinks and windows, whole
    windows of them, and a sequence without any."""
    c = P.Cache(61, [40, 1, 170, 9], [900, 1500, 1100, 64], 8, 2, 128, page, dtype, cache, layout, behind=1).poison()
    for b, L in enumerate(c.kv_lens):
        used = -(-L // page)
        c.table[b, b % 3: used: 5] = (-1, c.pages, 1 << 30, -5)[b]
    c.table[2, 700 // page: 1000 // page] = -1               # more than the narrow windows show
    c.table[3] = -5
    for window, sinks in ((300, 5), (50, 40), (700, 0), (9, 1)):
        run(c, window, sinks)


@pytest.mark.parametrize("cache,layout,dtype", CACHES)
@pytest.mark.parametrize("page", [16, 20])
def test_large_scores_and_scales(page, cache, layout, dtype):
    c = P.Cache(62, [6, 1, 240], [700, 333, 600], 8, 2, 128, page, dtype, cache, layout)
    q, _, _ = c.split(c.qkv)
    q *= torch.logspace(-6, 1.2, c.T).to(q.dtype)[:, None, None]
    if cache == "same":
        pool = c.k.transpose(1, 2) if layout == "HND" else c.k
        for b in range(3):
            at = c.cells(b)
            pool[at] *= torch.linspace(0.01, 3, len(at[0])).to(c.k.dtype)[:, None, None]
    for scale in (0.0, 1.0):
        run(c, 200, 2, scale)
        run(c, 33, 0, scale)


@pytest.mark.parametrize("cache,layout,dtype", CACHES)
def test_table_much_wider_than_the_sequences(cache, layout, dtype):
    c = P.Cache(63, [300, 1, 40], [900, 70, 41], 8, 2, 64, 16, dtype, cache, layout, before=1, behind=2).poison()
    for window, sinks in ((200, 5), (2000, 0), (1 << 19, 1)):
        w = P.Cache(63, [300, 1, 40], [900, 70, 41], 8, 2, 64, 16, dtype, cache, layout, before=1, behind=2).poison()
        X.poison_unseen(w, masks(c, window, sinks))
        widen(w)
        run(w, window, sinks, hint=300)


def test_few_rows_take_the_other_kernel():
    """(So the check of which one ran says something.)"""
    c = P.Cache(64, [1, 2], [900, 70], 8, 2, 128, 16, "bf16", "e4m3")
    out, lse, tiles = G.attend(c, sfa.paged_attention, window=50, sinks=2, max_q_len=2)
    assert not tiles
    check_window(c, out, lse, 50, 2)
