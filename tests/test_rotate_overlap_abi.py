"""Rotated appends without a GPU: queries are not written over rows that are still to be
read, unless in place."""
import numpy as np
import pytest

import sparse_attention_serving_sfa_gb300 as sfa
from tests.test_paged_abi import FAKE, INVALID, cache
from tests.test_paged_parts_abi import rotated

FAR = FAKE + (1 << 40)


@pytest.fixture(scope="module", autouse=True)
def built():
    sfa.build()
    sfa.load()


def touched(at, stride, width, n):
    return {at // 2 + i * stride + j for i in range(n) for j in range(width)}


def calls():
    """q, k, v, q_out as (offset in bytes, stride) of 4 query heads and 2 kv heads of 128."""
    ways = []
    for n in (1, 2, 5):
        # q_out begins elsewhere in q's rows, or among the keys or values
        for q, out in (((0, 512), (16, 512)), ((16, 512), (0, 512)), ((0, 512), (1024, 512)), ((0, 512), (1024 * n - 16, 512)),
                       ((0, 512), (0, 520)), ((0, 520), (0, 512)), ((0, 1024), (512, 1024)), ((0, 1024), (1040, 1024)),
                       ((0, 2048), (1008, 512)), ((0, 2048), (1024, 1536)), ((4096, 512), (0, 2048))):
            ways.append((n, q, (1 << 30, 256), (1 << 31, 256), out))
        for k, v in (((0, 256), (1 << 31, 256)), ((1 << 31, 256), (0, 256)), ((1008, 1024), (1 << 31, 256)),
                     ((1 << 31, 256), (2032, 1024))):
            ways.append((n, (1 << 30, 512), k, v, (0, 1024)))
    g = np.random.default_rng(3)
    for _ in range(400):
        n = int(g.integers(1, 6))
        at = [16 * int(x) for x in g.integers(0, 400, 4)]
        strides = [512 + 8 * int(g.integers(0, 200)), 256 + 8 * int(g.integers(0, 200)), 256 + 8 * int(g.integers(0, 200)),
                   512 + 8 * int(g.integers(0, 200))]
        if g.integers(0, 2):
            strides = [strides[0]] * 4
        ways.append((n, *zip(at, strides)))
    return ways


def test_queries_written_over_rows_to_be_read():
    """Every call that would write an element which another row of q, k_new or v_new is
    read from is refused (those that would not are left out: they would launch)."""
    refused = 0
    for n, q, k, v, out in calls():
        to = touched(*out, 512, n)
        if not (to & (touched(*q, 512, n) | touched(*k, 256, n) | touched(*v, 256, n))):
            continue
        if q[0] == out[0] and (n == 1 or q[1] == out[1]) and not to & (touched(*k, 256, n) | touched(*v, 256, n)):
            continue                                          # in place
        assert rotated(cache(), n=n, q=FAR + q[0], qs=q[1], k=FAR + k[0], ks=k[1], v=FAR + v[0], vs=v[1], out=FAR + out[0],
                       os=out[1]) == INVALID, (n, q, k, v, out)
        refused += 1
    assert refused > 200


def test_in_place_with_another_stride():
    assert rotated(cache(), k=FAR, v=2 * FAR, qs=512, os=520) == INVALID
    assert rotated(cache(), k=FAR, v=2 * FAR, qs=520, os=512) == INVALID
