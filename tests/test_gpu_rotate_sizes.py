"""rotate at the end of the range of its sizes."""
import ctypes as C

import pytest
import torch

import sparse_attention_prefill_gb300 as S
from tests import page_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dim", [64, 128])
def test_most_query_rows_of_a_batch(dim):
    """A batch padded to 2^31 - 1 query rows, of which the first few are a request's: others
    are not touched, so that they need not be there.  (The arrays lie in front of the rows,
    which the call would else take for theirs.)"""
    n, m, rot = 5, 900, 64
    mem = torch.zeros(1 << 16, dtype=torch.uint8, device=DEV)

    def part(at, like):
        t = mem[at:at + like.numel() * like.element_size()].view(like.dtype)
        t.copy_(like)
        return t

    rope = S.rope_freqs(rot)
    freq = part(0, rope["freq"])
    cu_q, kv_len = part(1024, torch.tensor([0, n], dtype=torch.int32)), part(2048, torch.tensor([m]))
    d_err = part(3200, torch.zeros(1, dtype=torch.int32))
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((n, 1, dim), generator=g, device=DEV).half()
    rows = part(4096, x.flatten())
    b = S.CPacked((1 << 31) - 1, 1, cu_q.data_ptr(), None, kv_len.data_ptr())
    r = S.CRope(freq.data_ptr(), None, rot, 0, 1.0, 0)
    lib = S.load()
    st = lib.csa2_rotate(C.byref(b), 1, dim, S.DT_F16, rows.data_ptr(), dim, C.byref(r), 0,
                         rows.data_ptr(), dim, d_err.data_ptr(),
                         torch.cuda.current_stream().cuda_stream)
    assert st == S.OK
    torch.cuda.synchronize()
    assert int(d_err.item()) == 0
    ok, _ = R.batch([n], [m], DEV)
    assert torch.equal(rows.view(x.shape), S.rotate(ok, x, rope))
    assert (mem[4096 + 2 * x.numel():] == 0).all()
