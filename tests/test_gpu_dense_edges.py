"""Dense-cache calls at the edges of what their arguments allow: malformed
device data, overlapping arguments, streams, sizes that choose rare variants."""
import pytest
import torch

import sparse_attention_prefill_gb300 as S
from tests.test_gpu_dense_attn import DEV, _derr

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _i64(x):
    return torch.tensor(x, dtype=torch.int64, device=DEV)


# ---------------------------------------------------------------------------
# moving rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("far", [2 ** 63 - 1, 2 ** 63 - 4, 2 ** 62, 20])
@pytest.mark.parametrize("src_far,dst_far", [(True, False), (False, True), (True, True)])
def test_rows_starts_past_every_buffer(far, in_place, src_far, dst_far):
    """A start so high that start + row does not fit 64 bits is out of range
    like any other; the other request's rows are moved all the same."""
    k = torch.arange(80, dtype=torch.float32, device=DEV).view(20, 1, 4)
    dst = k.clone() if in_place else torch.full((20, 1, 4), -1.0, device=DEV)
    want = dst.clone()
    want[10:13] = k[[11, 13, 15]]
    d = _derr()
    S.evict_rows(_i32([[[1, 3, 5]], [[0, 2, 4]]]), _i64([3, 3]),
                 _i64([10, far if src_far else 0]), _i64([10, far if dst_far else 0]),
                 [(dst if in_place else k, dst)], d_err=d)
    assert int(d.item()) == S.DERR_RANGE_ROW
    assert torch.equal(dst, want)
