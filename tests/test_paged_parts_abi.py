"""Rotated appends, windowed attention and attention behind a shared prefix without a
GPU: bad arguments are turned away on the host before any launch."""
import ctypes

import pytest
import torch

import sparse_attention_serving_sfa_gb300 as sfa
from tests.test_paged_abi import (ATTENTION, BAD_CACHES, FAKE, INVALID, UNSUPPORTED, WORKSPACE, cache,
                                  tensors)


@pytest.fixture(scope="module", autouse=True)
def built():
    sfa.build()
    sfa.load()


def rotated(c, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, qs=512, ks=256, vs=256, os=512, cu=FAKE, n=4, heads=4, freq=FAKE,
             rotary=64, pairs=0, dtype=1)
    a.update(over)
    return sfa.load().paged_append_rotated(ctypes.byref(c) if c else None, a["q"], a["k"], a["v"], a["out"], a["qs"],
                                           a["ks"], a["vs"], a["os"], a["cu"], a["n"], a["heads"], a["freq"],
                                           a["rotary"], a["pairs"], a["dtype"], None)


def windowed(c, **over):
    a = dict(q=FAKE, stride=512, cu=FAKE, n=4, heads=4, hint=0, window=9, sinks=2, scale=0.1, dtype=1, out=FAKE,
             lse=None, ws=FAKE, bytes=1 << 40)
    a.update(over)
    return sfa.load().paged_run_window(ctypes.byref(c), a["q"], a["stride"], a["cu"], a["n"], a["heads"], a["hint"],
                                       a["window"], a["sinks"], a["scale"], a["dtype"], a["out"], a["lse"], a["ws"],
                                       a["bytes"], None)


def varlen_windowed(**over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=512, ks=256, vs=256, cq=FAKE, ck=FAKE, B=2, T=4, N=9, heads=4,
             kv=2, D=128, hint=0, window=9, sinks=2, scale=0.1, dtype=1, out=FAKE, lse=None, ws=FAKE, bytes=1 << 40)
    a.update(over)
    return sfa.load().varlen_run_window(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["cq"], a["ck"], a["B"],
                                        a["T"], a["N"], a["heads"], a["kv"], a["D"], a["hint"], a["window"],
                                        a["sinks"], a["scale"], a["dtype"], a["out"], a["lse"], a["ws"], a["bytes"],
                                        None)


def shared(c, **over):
    a = dict(q=FAKE, stride=512, cu=FAKE, n=4, heads=4, hint=0, groups=FAKE, lens=FAKE, num=2, scale=0.1, causal=1,
             dtype=1, out=FAKE, lse=None, ws=FAKE, bytes=1 << 40)
    a.update(over)
    return sfa.load().paged_run_shared(ctypes.byref(c), a["q"], a["stride"], a["cu"], a["n"], a["heads"], a["hint"],
                                       a["groups"], a["lens"], a["num"], a["scale"], a["causal"], a["dtype"],
                                       a["out"], a["lse"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_bad_caches(over, status):
    c = cache(**over)
    assert rotated(c) == status
    assert windowed(c) == status
    assert shared(c) == status


@pytest.mark.parametrize("over,status", [
    (dict(k=None), INVALID), (dict(v=FAKE + 4), INVALID), (dict(cu=None), INVALID), (dict(n=-1), INVALID),
    (dict(ks=128), INVALID), (dict(vs=257), INVALID), (dict(dtype=0), INVALID), (dict(dtype=2), INVALID),
    (dict(q=FAKE + 2), INVALID), (dict(out=None), INVALID), (dict(out=FAKE + 8), INVALID), (dict(qs=511), INVALID),
    (dict(os=256), INVALID), (dict(heads=0), INVALID), (dict(freq=None), INVALID), (dict(freq=FAKE + 2), INVALID),
    (dict(rotary=0), INVALID), (dict(rotary=-16), INVALID), (dict(rotary=31), INVALID), (dict(rotary=144), INVALID),
    (dict(rotary=24), UNSUPPORTED), (dict(rotary=2), UNSUPPORTED),
    (dict(n=1 << 28), UNSUPPORTED), (dict(heads=1 << 20, qs=1 << 27, os=1 << 27), UNSUPPORTED),
    (dict(n=0), sfa.SFA_OK), (dict(n=0, q=None, heads=0, out=None), sfa.SFA_OK)])
def test_bad_rotated_appends(over, status):
    assert rotated(cache(), **over) == status


def test_null_cache():
    assert rotated(None) == INVALID


WINDOWS = [(dict(window=0), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID)]


@pytest.mark.parametrize("over,status", ATTENTION + WINDOWS + [
    (dict(cu=None), INVALID), (dict(n=-1), INVALID), (dict(stride=511), INVALID), (dict(stride=256), INVALID),
    (dict(dtype=0), INVALID), (dict(n=1 << 28), UNSUPPORTED), (dict(n=0), sfa.SFA_OK)])
def test_bad_windowed_runs(over, status):
    assert windowed(cache(), **over) == status


@pytest.mark.parametrize("over,status", ATTENTION + WINDOWS + [
    (dict(cq=None), INVALID), (dict(ck=None), INVALID), (dict(T=-1), INVALID), (dict(N=-1), INVALID),
    (dict(B=0), INVALID), (dict(kv=0), INVALID), (dict(D=32), INVALID), (dict(D=256), UNSUPPORTED),
    (dict(qs=100), INVALID), (dict(ks=0), INVALID), (dict(vs=260), INVALID), (dict(k=None), INVALID),
    (dict(v=FAKE + 2), INVALID), (dict(N=1 << 30), UNSUPPORTED), (dict(T=1 << 29), UNSUPPORTED), (dict(T=0), sfa.SFA_OK)])
def test_bad_packed_windowed_runs(over, status):
    assert varlen_windowed(**over) == status


@pytest.mark.parametrize("over,status", ATTENTION + [
    (dict(cu=None), INVALID), (dict(n=-1), INVALID), (dict(stride=511), INVALID), (dict(dtype=0), INVALID),
    (dict(groups=None), INVALID), (dict(lens=None), INVALID), (dict(groups=FAKE + 2), INVALID),
    (dict(lens=FAKE + 1), INVALID), (dict(num=0), INVALID), (dict(num=-3), INVALID),
    (dict(n=1 << 28), UNSUPPORTED), (dict(n=0), sfa.SFA_OK)])
def test_bad_shared_runs(over, status):
    assert shared(cache(), **over) == status


def test_the_shared_workspace_holds_the_prefixes_results():
    one, all_ = sfa.paged_workspace_size(4, 100, 32, 8, 128), sfa.paged_shared_workspace_size(4, 100, 32, 8, 128)
    assert all_ == one + 100 * 32 * 130 * 4
    c = cache(num_kv_heads=8)
    assert shared(c, n=100, heads=32, stride=4096, bytes=all_ - 1) == WORKSPACE
    for bad in ((0, 4, 32, 8, 128), (4, -1, 32, 8, 128), (4, 4, 30, 8, 128), (4, 4, 32, 8, 100), (4, 1 << 28, 32, 8, 128)):
        with pytest.raises(sfa.SfaError):
            sfa.paged_shared_workspace_size(*bad)


def test_python_checks_of_rotated_appends():
    t = tensors()
    args = [t["new"], t["new"], t["cu"], t["k"], t["v"], t["table"], t["lens"]]
    freq = torch.ones(32)
    with pytest.raises(ValueError, match="CUDA"):
        sfa.paged_append_rotated(*args, freq, q=t["q"])
    for bad in (freq.double(), freq[None], freq.repeat(2)[::2]):
        with pytest.raises(ValueError, match="inv_freq"):
            sfa.paged_append_rotated(*args, bad)
    for q, out in ((t["q"].half(), None), (t["q"][:3], None), (t["q"][..., :32], None), (t["q"].transpose(0, 1), None),
                   (None, t["q"]), (t["q"], t["q"][:2]), (t["q"], t["q"].half()), (t["q"], torch.zeros(4, 4, 128).bfloat16()[..., ::2]),
                   (torch.zeros(4, 6, 64).bfloat16()[:, :4], None)):
        if q is not None and out is None and q.dim() == 3 and q.shape == (4, 4, 64) and q.dtype == torch.bfloat16:
            # the same memory with another stride
            out = q.as_strided((4, 4, 64), (256, 64, 1))
        with pytest.raises(ValueError):
            sfa.paged_append_rotated(*args, freq, q=q, q_out=out)
    with pytest.raises(TypeError):
        sfa.paged_append_rotated(*args, 32)


def test_python_checks_of_windows_and_groups():
    t = tensors()
    args = [t["q"], t["k"], t["v"], t["table"], t["lens"], t["cu"]]
    with pytest.raises(ValueError, match="CUDA"):
        sfa.paged_attention(*args, window=4, sinks=1)
    with pytest.raises(ValueError, match="causal"):
        sfa.paged_attention(*args, causal=False, window=4)
    packed = [t["q"], t["new"], t["new"], t["cu"], t["cu"]]
    with pytest.raises(ValueError, match="CUDA"):
        sfa.varlen_attention(*packed, window=4)
    with pytest.raises(ValueError, match="causal"):
        sfa.varlen_attention(*packed, causal=False, sinks=2)
    for window, sinks in ((1 << 31, 0), (4, 1 << 40)):
        with pytest.raises(ValueError, match="32 bits"):
            sfa.paged_attention(*args, window=window, sinks=sinks)
    groups, lens = torch.tensor([0, 2], dtype=torch.int32), torch.tensor([20], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sfa.shared_prefix_attention(*args, groups, lens)
    for a, b in ((groups.long(), lens), (groups, lens.long()), (groups[:1], lens), (groups, lens.repeat(2))):
        with pytest.raises(ValueError):
            sfa.shared_prefix_attention(*args, a, b)
    with pytest.raises(ValueError):
        sfa.shared_prefix_attention(t["q"].float(), *args[1:], groups, lens)
