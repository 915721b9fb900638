"""Outputs and workspaces in the middle of larger buffers, to see that a call writes nothing
beside them; and which of the two attention kernels a call took."""
import torch

import sparse_attention_serving_sfa_gb300 as sfa
from tests import paged_testlib as P
from tests.test_gpu_paged import kw

ROOM = 4096


class Guard:
    def __init__(self):
        self.kept = []

    def tensor(self, shape, dtype, byte=None, value=None):
        """A new tensor of that shape with ROOM bytes to either side that must stay."""
        n = torch.empty(0, dtype=dtype).element_size()
        for s in shape:
            n *= s
        buf = torch.full((n + 2 * ROOM,), 0xA5, dtype=torch.uint8, device="cuda")
        self.kept.append((buf, n))
        x = buf[ROOM: ROOM + n]
        if byte is not None:
            x.fill_(byte)
        x = x.view(dtype).view(shape)
        return x if value is None else x.fill_(value)

    def copy(self, x):
        y = self.tensor(x.shape, x.dtype)
        y.view(torch.uint8).copy_(x.cuda().view(torch.uint8))
        return y

    def check(self):
        torch.cuda.synchronize()
        assert sfa.sfa_get_last_error() == sfa.SFA_OK
        for buf, n in self.kept:
            assert (buf[:ROOM] == 0xA5).all() and (buf[ROOM + n:] == 0xA5).all()


def few_row_workspace(dim):
    """Bytes of workspace that the kernel for few rows uses: parts of 16 rows with two fp32
    words of softmax state each, two for each of at most 320 ranges.  The other kernel writes
    down a cut item a range behind more than that, in every call."""
    return 2 * 320 * 16 * (dim + 2) * 4


def attend(c, call, lists=(), d=None, **more):
    """call() over cache c with everything it writes guarded: out, lse, and whether the
    tensor-core kernel ran.  The cache and the lists must stay as they are."""
    g = Guard()
    d = d or c.to("cuda")
    before = [d[n].view(torch.uint8).clone() for n in ("k", "v")]
    q, _, _ = c.split(d["qkv"])
    size = sfa.paged_shared_workspace_size if lists else sfa.paged_workspace_size
    ws = g.tensor((size(len(c.kv_lens), c.T, c.Hq, c.H, c.D),), torch.uint8, byte=0xFF)
    out = g.tensor((c.T, c.Hq, c.D), P.TORCH[c.dtype], value=9.0)
    lse = g.tensor((c.T, c.Hq), torch.float32, value=9.0)
    call(q, d["k"], d["v"], d["table"], d["lens"], d["cu"], *lists, out=out, lse=lse, workspace=ws, **kw(c, d), **more)
    g.check()
    assert all(torch.equal(d[n].view(torch.uint8), x) for n, x in zip(("k", "v"), before))
    plain = ws[few_row_workspace(c.D): sfa.paged_workspace_size(len(c.kv_lens), c.T, c.Hq, c.H, c.D)]
    return out.cpu(), lse.cpu(), bool((plain != 0xFF).any())
