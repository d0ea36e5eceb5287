"""Refusals of the dense-cache calls that concern several arguments at once
(no GPU needed: every call here is refused before a launch)."""
import ctypes as C

import pytest

import sparse_attention_prefill_gb300 as S
from sparse_attention_prefill_gb300 import build

AT = 1 << 30             # addresses far apart; never read
INV = S.ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    return S.load(build.build())


# 3 requests, 2 heads, 100 rows, 10 kept: kv_start, kv_len and new_len are 24
# bytes, mass is 800, idx 240
@pytest.mark.parametrize("kw", [
    dict(new=2 * AT + 8), dict(new=2 * AT - 8), dict(new=AT), dict(new=AT + 16), dict(new=3 * AT),
    dict(new=3 * AT + 792), dict(idx=AT), dict(idx=AT - 236), dict(idx=2 * AT + 20),
    dict(idx=3 * AT + 796), dict(idx=5 * AT + 20), dict(idx=5 * AT - 236), dict(idx=2 * AT, new=2 * AT)])
def test_select_outputs_that_overlap_are_refused(lib, kw):
    d = dict(idx=4 * AT, new=5 * AT)
    d.update(kw)
    assert lib.csa2_evict_select(3, 2, AT, 2 * AT, 3 * AT, 100, 10, 1, 2, d["idx"], d["new"], None,
                                 None) == INV


def _prefix_status(lib, n, ws_bytes, heads, kv, dim, groups, max_prefix, max_kv):
    """INV if the workspace is too small.  (Its address is not aligned, which is
    refused next: nothing is ever launched.)"""
    b = S.CPacked(n, n, AT, AT, AT)
    g = S.CPrefixGroups(groups, 0, AT, AT, AT, max_prefix)
    return lib.csa2_prefix_attn(C.byref(b), C.byref(g) if groups else None, heads, kv, dim,
                                S.DT_BF16, AT, heads * dim, AT, kv * dim, AT, kv * dim, 100, max_kv,
                                0.1, AT, None, AT + 16, ws_bytes, None, None)


@pytest.mark.parametrize("heads,kv,dim,groups,max_prefix,max_kv", [
    (64, 8, 128, 0, 0, 8192), (64, 8, 128, 1, 8192, 700), (16, 4, 64, 3, 900, 30000),
    (20, 1, 64, 2, 64, 64), (6, 2, 128, 0, 0, 0)])
@pytest.mark.parametrize("most", [300, 171, 115, 58])
def test_workspace_of_the_largest_batch_serves_every_smaller_one(lib, heads, kv, dim, groups,
                                                                 max_prefix, max_kv, most):
    sizes = (groups, heads, kv, dim, max_prefix, max_kv)
    need = S.csa2_prefix_attn_workspace(most, most, *sizes)
    for n in range(most, 0, -1):
        assert _prefix_status(lib, n, need, heads, kv, dim, groups, max_prefix,
                              max_kv) == S.ERR_UNSUPPORTED, n
        # and what it is told to take is enough
        own = S.csa2_prefix_attn_workspace(n, n, *sizes)
        assert _prefix_status(lib, n, own, heads, kv, dim, groups, max_prefix,
                              max_kv) == S.ERR_UNSUPPORTED, n


@pytest.mark.parametrize("heads,kv,dim,groups", [(64, 8, 128, 0), (6, 2, 64, 2), (3, 1, 128, 1)])
@pytest.mark.parametrize("n", [1, 7, 33, 200])
def test_least_workspace_is_one_part_a_side(lib, heads, kv, dim, groups, n):
    rows = (n * (heads // kv) + 31) // 32 * 32
    least = 4 * (dim + 1) * kv * rows * (2 if groups else 1)
    for size, status in ((least, S.ERR_UNSUPPORTED), (least - 4, INV), (0, INV), (-4, INV)):
        assert _prefix_status(lib, n, size, heads, kv, dim, groups, 5000, 5000) == status


@pytest.mark.parametrize("first,second", [(0, 1), (0, 7), (3, 6)])
def test_rows_one_destination_twice_is_refused(lib, first, second):
    arr = (S.CEvictBuf * 8)(*[S.CEvictBuf(AT, (2 + i) * AT, 10, 10, 64, 32, 64, 32, 32)
                              for i in range(8)])
    arr[second].dst = arr[first].dst
    assert lib.csa2_evict_rows(2, 2, AT, 4, AT, AT, AT, 8, arr, None, None) == INV
