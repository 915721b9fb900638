"""The paged cache and packed-row attention without a GPU: bad arguments are
turned away on the host before any launch."""
import ctypes

import pytest
import torch

import sparse_attention_serving_sfa_gb300 as sfa

FAKE = 1 << 20     # aligned non-null address; never dereferenced by rejected calls


@pytest.fixture(scope="module", autouse=True)
def built():
    sfa.build()
    sfa.load()


def cache(**over):
    a = dict(k=FAKE, v=FAKE, page_table=FAKE, kv_lens=FAKE, num_seqs=2, num_pages=8, page_size=16,
             max_pages=4, num_kv_heads=2, head_dim=128, kv_layout=0, dtype=1, scale_k=None,
             scale_v=None)
    a.update(over)
    return sfa.PagedKV(**a)


INVALID, UNSUPPORTED, WORKSPACE = sfa.SFA_ERR_INVALID_ARG, sfa.SFA_ERR_UNSUPPORTED, sfa.SFA_ERR_WORKSPACE

BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(page_table=None), INVALID),
    (dict(kv_lens=None), INVALID), (dict(num_seqs=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(max_pages=0), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(head_dim=0), INVALID), (dict(head_dim=96), INVALID), (dict(head_dim=192), UNSUPPORTED),
    (dict(kv_layout=2), INVALID), (dict(dtype=4), INVALID), (dict(dtype=-1), INVALID),
    (dict(k=FAKE + 8), INVALID), (dict(page_table=FAKE + 2), INVALID),
    (dict(scale_k=FAKE), UNSUPPORTED),                        # scales of a 16-bit cache
    (dict(dtype=2, scale_v=FAKE + 1), INVALID),
    (dict(page_size=1 << 20, max_pages=1 << 11), UNSUPPORTED),  # positions beyond 30 bits
]


def append(c, **over):
    a = dict(k=FAKE, v=FAKE, ks=256, vs=256, cu=FAKE, n=4, dtype=1)
    a.update(over)
    return sfa.load().paged_append(ctypes.byref(c), a["k"], a["v"], a["ks"], a["vs"], a["cu"], a["n"],
                                   a["dtype"], None)


def read(c, **over):
    a = dict(cu=FAKE, n=4, dtype=1, k=FAKE, v=FAKE)
    a.update(over)
    return sfa.load().paged_read(ctypes.byref(c), a["cu"], a["n"], a["dtype"], a["k"], a["v"], None)


def paged(c, **over):
    a = dict(q=FAKE, stride=512, cu=FAKE, n=4, heads=4, hint=0, scale=0.1, causal=1, dtype=1, out=FAKE,
             lse=None, ws=FAKE, bytes=1 << 40)
    a.update(over)
    return sfa.paged_run(c, a["q"], a["stride"], a["cu"], a["n"], a["heads"], a["hint"], a["scale"],
                         a["causal"], a["dtype"], a["out"], a["lse"], a["ws"], a["bytes"], check=False)


def varlen(**over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=512, ks=256, vs=256, cq=FAKE, ck=FAKE, B=2, T=4, N=9, heads=4,
             kv=2, D=128, hint=0, scale=0.1, causal=1, dtype=1, out=FAKE, lse=None, ws=FAKE, bytes=1 << 40)
    a.update(over)
    return sfa.varlen_run(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["cq"], a["ck"], a["B"],
                          a["T"], a["N"], a["heads"], a["kv"], a["D"], a["hint"], a["scale"],
                          a["causal"], a["dtype"], a["out"], a["lse"], a["ws"], a["bytes"], check=False)


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_bad_caches(over, status):
    c = cache(**over)
    assert append(c) == status
    assert read(c) == status
    assert paged(c) == status


def test_null_cache():
    assert sfa.load().paged_append(None, FAKE, FAKE, 256, 256, FAKE, 4, 1, None) == INVALID


@pytest.mark.parametrize("over,status", [
    (dict(k=None), INVALID), (dict(v=FAKE + 4), INVALID), (dict(cu=None), INVALID), (dict(n=-1), INVALID),
    (dict(ks=128), INVALID), (dict(vs=257), INVALID), (dict(dtype=0), INVALID), (dict(dtype=2), INVALID),
    (dict(n=1 << 30), UNSUPPORTED), (dict(n=0), sfa.SFA_OK)])
def test_bad_appends(over, status):
    assert append(cache(), **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(k=None), INVALID), (dict(v=FAKE + 4), INVALID), (dict(cu=FAKE + 1), INVALID), (dict(n=-1), INVALID),
    (dict(dtype=0), INVALID), (dict(dtype=3), INVALID), (dict(n=0), sfa.SFA_OK)])
def test_bad_reads(over, status):
    assert read(cache(), **over) == status


ATTENTION = [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q=FAKE + 2), INVALID), (dict(lse=FAKE + 2), INVALID),
    (dict(heads=3), INVALID), (dict(heads=0), INVALID), (dict(hint=-1), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(dtype=2), INVALID),
    (dict(ws=None), WORKSPACE), (dict(bytes=16), WORKSPACE), (dict(ws=FAKE + 8), INVALID)]


@pytest.mark.parametrize("over,status", ATTENTION + [
    (dict(cu=None), INVALID), (dict(n=-1), INVALID), (dict(stride=511), INVALID), (dict(stride=256), INVALID),
    (dict(dtype=0), INVALID),                                     # not the 16-bit cache's own
    (dict(n=1 << 28), UNSUPPORTED), (dict(n=0), sfa.SFA_OK)])
def test_bad_paged_runs(over, status):
    assert paged(cache(), **over) == status


@pytest.mark.parametrize("over,status", ATTENTION + [
    (dict(cq=None), INVALID), (dict(ck=None), INVALID), (dict(T=-1), INVALID), (dict(N=-1), INVALID),
    (dict(B=0), INVALID), (dict(kv=0), INVALID), (dict(D=32), INVALID), (dict(D=256), UNSUPPORTED),
    (dict(qs=100), INVALID), (dict(ks=0), INVALID), (dict(vs=260), INVALID), (dict(k=None), INVALID),
    (dict(v=FAKE + 2), INVALID), (dict(N=1 << 30), UNSUPPORTED), (dict(T=1 << 29), UNSUPPORTED), (dict(T=0), sfa.SFA_OK)])
def test_bad_varlen_runs(over, status):
    assert varlen(**over) == status


def test_workspace_sizes():
    n = sfa.paged_workspace_size(4, 4, 32, 8, 128)
    assert n > 0 and sfa.varlen_workspace_size(4, 4, 32, 8, 128) == n
    for bad in ((0, 4, 32, 8, 128), (4, -1, 32, 8, 128), (4, 4, 30, 8, 128), (4, 4, 32, 8, 100)):
        with pytest.raises(sfa.SfaError):
            sfa.paged_workspace_size(*bad)


def tensors():
    t = dict(k=torch.zeros(8, 16, 2, 64).bfloat16(), table=torch.zeros(2, 4, dtype=torch.int32),
             lens=torch.zeros(2, dtype=torch.int32), cu=torch.zeros(3, dtype=torch.int32),
             new=torch.zeros(4, 2, 64).bfloat16(), q=torch.zeros(4, 4, 64).bfloat16())
    t["v"] = t["k"].clone()
    return t


@pytest.mark.parametrize("name,bad", [
    ("k", lambda x: x.transpose(1, 2)), ("k", lambda x: x[0]), ("v", lambda x: x.half()), ("k", lambda x: x.float()),
    ("table", lambda x: x.long()), ("table", lambda x: x[0]), ("lens", lambda x: x[:1]), ("cu", lambda x: x[:2]),
    ("new", lambda x: x[:, :1]), ("new", lambda x: x.transpose(1, 2)), ("new", lambda x: x[..., ::2])])
def test_python_checks_of_the_cache(name, bad):
    t = tensors()
    t[name] = bad(t[name])
    with pytest.raises(ValueError):
        sfa.paged_append(t["new"], t["new"], t["cu"], t["k"], t["v"], t["table"], t["lens"])


def test_python_checks_of_attention():
    t = tensors()
    args = [t["q"], t["k"], t["v"], t["table"], t["lens"], t["cu"]]
    with pytest.raises(ValueError, match="CUDA"):                  # tensors on the host
        sfa.paged_attention(*args)
    with pytest.raises(ValueError):
        sfa.paged_attention(t["q"][:, :, :32], *args[1:])
    with pytest.raises(ValueError):
        sfa.paged_attention(*args, scale_k=torch.ones(3))
    k = t["new"]
    with pytest.raises(ValueError, match="CUDA"):
        sfa.varlen_attention(t["q"], k, k, t["cu"], t["cu"])
    for bad in ((t["q"].half(), k, k), (t["q"], k, k[:2]), (t["q"].transpose(1, 2), k, k), (t["q"][0], k, k)):
        with pytest.raises(ValueError):
            sfa.varlen_attention(*bad, t["cu"], t["cu"])
    with pytest.raises(ValueError):
        sfa.paged_read(t["k"], t["v"], t["table"], t["lens"], t["cu"].long(), 4)


@pytest.mark.parametrize("dtype", ["e4m3", "e5m2", 7, 4])
def test_read_refuses_types_it_does_not_write(dtype):
    t = tensors()
    with pytest.raises(ValueError, match="dtype"):
        sfa.paged_read(t["k"], t["v"], t["table"], t["lens"], t["cu"], 4, dtype=dtype)


@pytest.mark.parametrize("error", [RuntimeError("g++ failed"), FileNotFoundError("g++"), ImportError("torch")])
def test_library_builds_without_the_module_for_torch(monkeypatch, error):
    """The C library's users need neither g++ nor Python's headers."""
    from sparse_attention_serving_sfa_gb300 import _build

    def fails():
        raise error
    monkeypatch.setattr(_build, "stale", lambda: False)
    monkeypatch.setattr(_build, "tensors_stale", lambda: True)
    monkeypatch.setattr(_build, "build_tensors", fails)
    with pytest.warns(UserWarning, match="torch"):
        assert _build.build() == _build.LIB_PATH
