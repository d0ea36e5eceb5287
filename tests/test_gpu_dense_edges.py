"""Dense-cache calls at the edges of what their arguments allow: malformed
device data, overlapping arguments, streams, sizes that choose rare variants."""
import pytest
import torch

import sparse_attention_prefill_gb300 as S
from tests import dense_ref as R
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


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows,heads,keep", [
    ([300, 12, 64, 65, 0], 3, 64), ([5200] * 8, 8, 1000), ([30000], 8, 4095), ([26000, 50], 2, 100),
    ([20] * 700, 2, 9)])
def test_select_shortens_kv_len_in_place(rows, heads, keep):
    """new_len may be kv_len: the selection goes by the lengths before."""
    start, pool = R.starts(rows)
    mass = torch.rand((heads, pool), device=DEV)
    st, n = _i64(start), _i64(rows)
    want, lens = S.evict_select(st, n.clone(), mass, keep, 2, 5)
    for _ in range(5):
        d = _derr()
        m = n.clone()
        idx, out = S.evict_select(st, m, mass, keep, 2, 5, new_len=m, d_err=d)
        assert out is m and int(d.item()) == 0
        assert torch.equal(m, lens) and torch.equal(idx, want)


def test_select_in_place_lengths_of_bad_requests():
    mass = torch.rand((2, 100), device=DEV)
    d = _derr()
    n = _i64([50, 50, 5, -2])
    idx, _ = S.evict_select(_i64([0, 90, -1, 0]), n, mass, 20, 1, 1, new_len=n, d_err=d)
    assert int(d.item()) == S.DERR_RANGE_ROW and n.tolist() == [20, 0, 0, 0]
    assert (idx[1:] == -1).all() and (idx[0] >= 0).all()
