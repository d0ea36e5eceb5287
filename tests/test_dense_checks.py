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
    dict(idx=3 * AT + 796), dict(idx=5 * AT + 20), dict(idx=5 * AT - 236),
    dict(idx=2 * AT, new=2 * AT)])
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


# 10 query rows of 8 x 128 (20480 bytes), 100 cache rows of 2 x 128 (51200
# bytes, or 1024 bytes apart), lse 320 bytes, mass 800, 2 requests, 1 group
def _attn(lib, prefix, **kw):
    d = dict(cu=AT, ks=2 * AT, kl=3 * AT, q=4 * AT, ldq=1024, k=5 * AT, v=6 * AT, ld=256,
             out=7 * AT, lse=8 * AT, ws=9 * AT, cug=10 * AT, ps=11 * AT, pl=12 * AT)
    d.update(kw)
    b = S.CPacked(10, 2, d["cu"], d["ks"], d["kl"])
    args = [8, 2, 128, S.DT_BF16, d["q"], d["ldq"], d["k"], d["ld"], d["v"], d["ld"], 100]
    if not prefix:
        return lib.csa2_prompt_attn(C.byref(b), *args, 0.1, d["out"], d["lse"], None, None)
    g = S.CPrefixGroups(1, 0, d["cug"], d["ps"], d["pl"], 50)
    return lib.csa2_prefix_attn(C.byref(b), C.byref(g), *args, 90, 0.1, d["out"], d["lse"], d["ws"],
                                1 << 24, None, None)


BOTH = [
    dict(out=5 * AT), dict(out=6 * AT + 51200 - 16), dict(out=5 * AT - 20480 + 16),
    dict(lse=7 * AT), dict(lse=7 * AT + 20476), dict(lse=4 * AT + 20000), dict(lse=6 * AT), dict(out=4 * AT + 16),
    dict(out=4 * AT, ldq=2048), dict(out=4 * AT + 2048, ldq=2048), dict(out=AT), dict(out=2 * AT),
    dict(lse=3 * AT + 12), dict(out=5 * AT + 512, ld=512)]


@pytest.mark.parametrize("prefix,kw", [(p, kw) for p in (False, True) for kw in BOTH] + [
    (True, dict(ws=5 * AT)), (True, dict(ws=4 * AT)), (True, dict(ws=7 * AT)),
    (True, dict(ws=8 * AT)),
    (True, dict(ws=6 * AT + 51200 - 256)), (True, dict(ws=10 * AT)), (True, dict(out=11 * AT)),
    (True, dict(out=12 * AT - 16))])
def test_attention_outputs_that_overlap_are_refused(lib, prefix, kw):
    assert _attn(lib, prefix, **kw) == INV


@pytest.mark.parametrize("kw", [
    dict(mass=4 * AT), dict(mass=5 * AT), dict(mass=5 * AT + 51200 - 4), dict(mass=8 * AT),
    dict(mass=8 * AT - 796), dict(old=13 * AT + 400, mass=13 * AT),
    dict(old=13 * AT - 4, mass=13 * AT),
    dict(mass=AT), dict(mass=3 * AT + 8)])
def test_mass_outputs_that_overlap_are_refused(lib, kw):
    d = dict(old=None)
    d.update(kw)
    b = S.CPacked(10, 2, AT, 2 * AT, 3 * AT)
    assert lib.csa2_attn_mass(C.byref(b), 8, 2, 128, S.DT_BF16, 4 * AT, 1024, 5 * AT, 256, 100,
                              8 * AT, 90, 0.1, d["old"], d["mass"], None, None) == INV


# ---------------------------------------------------------------------------
# arrays that are not aligned to their elements
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("prefix,kw", [(p, kw) for p in (False, True) for kw in (
    dict(cu=AT + 2), dict(ks=2 * AT + 4), dict(kl=3 * AT + 4), dict(lse=8 * AT + 2),
    dict(out=7 * AT + 8))] + [
    (True, dict(cug=10 * AT + 1)), (True, dict(ps=11 * AT + 4)), (True, dict(pl=12 * AT + 4))])
def test_attention_misaligned_arrays_are_refused(lib, prefix, kw):
    assert _attn(lib, prefix, **kw) == S.ERR_UNSUPPORTED


@pytest.mark.parametrize("at", range(6))
def test_mass_misaligned_arrays_are_refused(lib, at):
    off = [0] * 6
    off[at] = 4 if at in (1, 2) else 2
    b = S.CPacked(10, 2, AT + off[0], 2 * AT + off[1], 3 * AT + off[2])
    assert lib.csa2_attn_mass(C.byref(b), 8, 2, 128, S.DT_BF16, 4 * AT, 1024, 5 * AT, 256, 100,
                              8 * AT + off[3], 90, 0.1, 9 * AT + off[4], 13 * AT, 14 * AT + off[5],
                              None) == S.ERR_UNSUPPORTED


@pytest.mark.parametrize("at", range(5))
def test_select_misaligned_arrays_are_refused(lib, at):
    off = [0] * 5
    off[at] = 2 if at in (2, 4) else 4
    assert lib.csa2_evict_select(3, 2, AT + off[0], 2 * AT + off[1], 3 * AT, 100, 10, 1, 2,
                                 4 * AT + off[2], 5 * AT + off[3], 6 * AT + off[4],
                                 None) == S.ERR_UNSUPPORTED


@pytest.mark.parametrize("at", range(5))
def test_rows_misaligned_arrays_are_refused(lib, at):
    off = [0] * 5
    off[at] = 4 if 0 < at < 4 else 2
    arr = (S.CEvictBuf * 1)(S.CEvictBuf(8 * AT, 9 * AT, 10, 10, 64, 32, 64, 32, 32))
    assert lib.csa2_evict_rows(2, 2, AT + off[0], 4, 2 * AT + off[1], 3 * AT + off[2],
                               4 * AT + off[3], 1, arr, 5 * AT + off[4], None) == S.ERR_UNSUPPORTED
