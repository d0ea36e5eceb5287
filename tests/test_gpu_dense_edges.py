"""Dense-cache calls at the edges of what their arguments allow: malformed
device data, overlapping arguments, streams, sizes that choose rare variants."""
import math

import pytest
import torch

import sparse_attention_prefill_gb300 as S
from tests import dense_ref as R
from tests.test_gpu_dense_attn import BF, DEV, HF, _derr, _inputs

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


# ---------------------------------------------------------------------------
# waits that run out
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("heads,kv,dim,dtype", [(16, 2, 128, BF), (8, 4, 64, HF)])
def test_waits_of_every_length_run_out_and_recover(heads, kv, dim, dtype):
    """Limits around the time that the kernels' steps take, so that a wait runs
    out in any role and at any step, for some lanes of a warp just before it
    would have been met: the calls end and the next ones are right."""
    new, rows = [400, 3, 130, 1], [900, 700, 130, 2000]
    b, _, start, q, k, v = _inputs(new, rows, heads, kv, dim, dtype, seed=dim, extra=[1500])
    few, _, fstart, fq, fk, fv = _inputs([5, 2], [800, 3000], heads, kv, dim, dtype, seed=1)
    gr = dict(num_groups=1, cu_group=_i32([0, 4]), prefix_start=_i64(start[-1:]),
              prefix_len=_i64([1500]), max_prefix=1500)

    def calls(d):
        out = S.prompt_attn(b, q, k, v, d_err=d)
        return (*out, *S.prompt_attn(few, fq, fk, fv, d_err=d),
                *S.prefix_attn(b, gr, q, k, v, 2000, d_err=d),
                S.attn_mass(b, q, k, out[1], 2000, d_err=d))

    want = calls(None)
    d = _derr()
    try:
        for limit in (1, 300, 700, 1500, 3000, 6000, 12000, 25000, 50000, 99999, 100001, 200000):
            S.set_wait_limit_ns(limit)
            for _ in range(4):
                calls(d)
            torch.cuda.synchronize()
    finally:
        S.set_wait_limit_ns(0)
    assert int(d.item()) & S.DERR_TIMEOUT
    d = _derr()
    got = calls(d)
    assert int(d.item()) == 0
    for x, y in zip(want, got):
        assert torch.equal(x.nan_to_num(9.0), y.nan_to_num(9.0))


# ---------------------------------------------------------------------------
# streams
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("call", ["prompt", "prefix", "mass", "select"])
def test_side_stream_leaves_freed_memory_of_the_current_one(call):
    """Tensors freed while work on them is still queued on the current stream:
    what a call on another stream allocates must not be their memory."""
    rows = [700] * 20
    b, _, start, q, k, v = _inputs([1] * 20, rows, 16, 2, 128, BF)
    _, lse = S.prompt_attn(b, q, k, v)
    weight = torch.rand((2, k.shape[0]), device=DEV)
    run = {"prompt": lambda s: S.prompt_attn(b, q, k, v, stream=s),
           "prefix": lambda s: S.prefix_attn(b, None, q, k, v, 700, stream=s),
           "mass": lambda s: (S.attn_mass(b, q, k, lse, 700, stream=s),),
           "select": lambda s: S.evict_select(b["kv_start"], b["kv_len"], weight, 100,
                                               stream=s)}[call]
    want = run(None)
    sizes = [x.numel() * x.element_size() for x in want]
    sizes.append(S.csa2_prefix_attn_workspace(20, 20, 0, 16, 2, 128, 0, 700))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        used = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in sizes]
        torch.cuda._sleep(200_000_000)       # some 0.1 s
        read = [x.clone() for x in used]
        used.clear()
        got = run(side)
        side.synchronize()
        for x, y in zip(want, got):
            assert torch.equal(x, y)
        for x in read:
            assert (x == 7).all()


def test_side_stream_results_stay_while_the_current_stream_reads_them():
    """A result freed while the current stream has yet to read it: calls on the
    side stream must not be given its memory."""
    b, _, start, q, k, v = _inputs([300], [300], 8, 2, 128, BF)
    q2 = -q
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = S.prompt_attn(b, q, k, v)[0]
    torch.cuda.synchronize()
    out, lse = S.prompt_attn(b, q, k, v, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)
    read = out.clone()
    del out, lse
    for _ in range(3):
        S.prompt_attn(b, q2, k, v, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(read, want)


# ---------------------------------------------------------------------------
# malformed batches
# ---------------------------------------------------------------------------

def _is_range(cu, a, b, num_q):
    return 0 <= cu[a] <= cu[b] <= num_q


def _check_batch(call, cu, rows, num_q, groups, heads, kv, dim, seed=0):
    """Outputs of a batch whose cu_q or groups may be malformed: right for the
    requests that are ranges of rows, untouched for all other rows.  groups:
    (cu_group, prefix lengths) or None."""
    pre = list(groups[1]) if groups else []
    _, _, start, _, k, v = _inputs([1] * len(rows), rows, heads, kv, dim, BF, seed=seed, extra=pre)
    q = torch.randn((num_q, heads, dim), device=DEV).to(BF)
    b = dict(num_q=num_q, num_req=len(rows), cu_q=_i32(cu), kv_start=_i64(start[:len(rows)]),
             kv_len=_i64(rows))
    out = torch.full((num_q, heads, dim), 7.0, dtype=BF, device=DEV)
    lse = torch.full((num_q, heads), 7.0, device=DEV)
    d = _derr()
    if call == "prompt":
        S.prompt_attn(b, q, k, v, out=out, lse=lse, d_err=d)
    else:
        gr = None
        if groups:
            gr = dict(num_groups=len(pre), cu_group=_i32(groups[0]), max_prefix=max(pre),
                      prefix_start=_i64(start[len(rows):]), prefix_len=_i64(pre))
        need = S.csa2_prefix_attn_workspace(num_q, len(rows), len(pre), heads, kv, dim,
                                            max(pre, default=0), max(rows))
        ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)       # NaNs
        S.prefix_attn(b, gr, q, k, v, max(rows), out=out, lse=lse, workspace=ws, d_err=d)
    bad = not all(_is_range(cu, r, r + 1, num_q) for r in range(len(rows)))
    if groups:
        bad |= not all(0 <= x <= y <= len(rows) and _is_range(cu, x, y, num_q)
                       for x, y in zip(groups[0], groups[0][1:]))
    assert int(d.item()) == (S.DERR_BAD_EXTEND if bad else 0)
    mine = [0] * num_q
    for r in range(len(rows)):
        if _is_range(cu, r, r + 1, num_q):
            for i in range(cu[r], cu[r + 1]):
                mine[i] += 1
    for r in range(len(rows)):
        if not _is_range(cu, r, r + 1, num_q) or cu[r] == cu[r + 1]:
            continue
        at = slice(cu[r], cu[r + 1])
        n = cu[r + 1] - cu[r]
        kk, vv, off = k[start[r]:start[r] + rows[r]], v[start[r]:start[r] + rows[r]], 0
        for g in range(len(pre)):
            x, y = groups[0][g:g + 2]
            if 0 <= x <= r < y <= len(rows) and _is_range(cu, x, y, num_q):
                p = start[len(rows) + g]
                off = pre[g]
                kk, vv = torch.cat([k[p:p + off], kk]), torch.cat([v[p:p + off], vv])
        last = torch.clamp(off + rows[r] - n + torch.arange(n, device=DEV), min=off - 1)
        ref = R.attend(q[at], kk, vv, dim ** -0.5, last)
        assert max(mine[at]) == 1            # the cases have no row in two requests
        R.check_attention(out[at], lse[at], ref, BF, max(1, kk.shape[0]))
    free = torch.tensor([m == 0 for m in mine], device=DEV)
    assert (out[free] == 7).all() and (lse[free] == 7).all()


# heads, key heads: single tokens by the decode kernel and by tensor-core items
@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (16, 1, 64), (20, 1, 64), (64, 2, 128)])
@pytest.mark.parametrize("cu,num_q,cug", [
    ([0, 1, 2, 4], 3, [0, 3]), ([0, 1, 10 ** 9, 3], 3, [0, 2, 3]), ([0, 1, 2, 3], 5, [0, 1, 3]),
    ([0, 1, 2, 4], 3, [0, 2, 3]), ([0, 1, 1, 2], 2, [0, 2]), ([0, 1, 10 ** 9, 3], 3, None),
    ([0, 1, 2, 4], 3, None), ([0, 1, 2, 3], 3, [1, 4]), ([0, 1, 2, 3], 3, [2, 1, 3])])
def test_malformed_batches_of_single_tokens_behind_prefixes(heads, kv, dim, cu, num_q, cug):
    groups = None if cug is None else (cug, [300, 77][:len(cug) - 1])
    _check_batch("prefix", cu, [30, 200, 5], num_q, groups, heads, kv, dim)


@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (5, 1, 64)])
@pytest.mark.parametrize("call,cu,num_q,cug", [
    ("prompt", [0, 20, 50, 76], 75, None), ("prompt", [-4, 20, 50, 75], 80, None),
    ("prompt", [40, 75, 20, 40], 80, None), ("prefix", [0, 20, 50, 76], 75, None),
    ("prefix", [-4, 20, 50, 75], 80, None), ("prefix", [40, 75, 20, 40], 80, [0, 2]),
    ("prefix", [0, 20, 50, 76], 75, [0, 3]), ("prefix", [0, 20, 50, 76], 75, [0, 2, 3]),
    ("prefix", [0, 20, 10 ** 9, 75], 75, [0, 1, 2]), ("prefix", [-4, 20, 50, 75], 80, [0, 1, 3]),
    ("prefix", [3, 20, 50, 75], 80, [0, 2, 5])])
def test_malformed_batches_of_extends(call, heads, kv, dim, cu, num_q, cug):
    groups = None if cug is None else (cug, [300, 77][:len(cug) - 1])
    _check_batch(call, cu, [30, 200, 35], num_q, groups, heads, kv, dim)


@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (16, 1, 64)])
@pytest.mark.parametrize("cu,num_q,cug", [
    ([-1, 1, 2, 3], 3, None), ([0, 1, 2, -5], 3, None), ([0, 1, 2, -7, 2], 2, None),
    ([0, 3, 1, 1, 1, 1, 1, 1, 1], 8, None), ([5, 1, 2, 6, 6, 6, 6, 6, 6], 8, None),
    ([2, 3, 4, 4, 4, 5], 5, None), ([2 ** 31 - 1, 0, 1, 2], 3, None),
    ([-2 ** 31, 0, 1, 2], 3, None), ([-1, 1, 2, 3], 3, [0, 2, 3]), ([-1, 1, 2, 3], 3, [1, 3]),
    ([5, 1, 2, 6, 6, 6, 6, 6, 6], 8, [1, 2, 4])])
@pytest.mark.parametrize("call", ["prompt", "prefix"])
def test_single_tokens_of_malformed_batches_are_all_found(call, heads, kv, dim, cu, num_q, cug):
    """Single tokens whose request has not their number, nor one as far from it
    as the first query row."""
    groups = None if cug is None or call == "prompt" else (cug, [300, 77][:len(cug) - 1])
    rows = [30, 200, 5, 64, 1, 17, 2, 3][:len(cu) - 1]
    _check_batch(call, cu, rows, num_q, groups, heads, kv, dim)


@pytest.mark.parametrize("reqs,free", [(511, 1), (513, 3), (1600, 40)])
def test_rows_of_many_requests_are_told_from_free_ones(reqs, free):
    """More requests than a look at each takes one step; a group of 3 heads, so
    that tokens cross the blocks of the join."""
    cu = [free + i for i in range(reqs + 1)]
    cu[reqs // 2] = cu[reqs // 2 - 1]            # one of no token, the next of two
    cu[-1] += 2                                  # three
    _check_batch("prefix", cu, [2 + i % 7 for i in range(reqs)], cu[-1] + free,
                 ([0, reqs // 3], [40]), 6, 2, 64)


# ---------------------------------------------------------------------------
# workspaces
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("heads,kv,dim,dtype,new", [
    (16, 2, 128, BF, 1), (8, 2, 64, HF, 1), (20, 1, 64, BF, 1), (8, 2, 128, BF, 9)])
@pytest.mark.parametrize("grouped", [False, True])
def test_less_workspace_means_fewer_splits(heads, kv, dim, dtype, new, grouped):
    """From what the call would choose down to one part a side."""
    reqs, pre = 6, 3000
    rows = [2500 - 300 * i for i in range(reqs)]
    b, cu, start, q, k, v = _inputs([new] * reqs, rows, heads, kv, dim, dtype, seed=dim,
                                    extra=[pre])
    gr = dict(num_groups=1, cu_group=_i32([0, 4]), max_prefix=pre, prefix_start=_i64(start[-1:]),
              prefix_len=_i64([pre])) if grouped else None
    sides = 2 if grouped else 1
    part = 4 * (dim + 1) * kv * ((reqs * new * heads // kv + 31) // 32 * 32)
    need = S.csa2_prefix_attn_workspace(b["num_q"], reqs, sides - 1, heads, kv, dim, pre, 2500)
    assert need > sides * part and need % part == 0
    refs = []
    for r in range(reqs):
        at = slice(cu[r], cu[r + 1])
        kk, vv, off = k[start[r]:start[r] + rows[r]], v[start[r]:start[r] + rows[r]], 0
        if grouped and r < 4:
            p = start[-1]
            kk, vv, off = torch.cat([k[p:p + pre], kk]), torch.cat([v[p:p + pre], vv]), pre
        last = off + rows[r] - new + torch.arange(new, device=DEV)
        refs.append((at, R.attend(q[at], kk, vv, dim ** -0.5, last), kk.shape[0]))
    for parts in range(sides, need // part + 1):
        ws = torch.full((parts * part,), 255, dtype=torch.uint8, device=DEV)
        out, lse = S.prefix_attn(b, gr, q, k, v, 2500, workspace=ws)
        for at, ref, n in refs:
            R.check_attention(out[at], lse[at], ref, dtype, n)
    with pytest.raises(S.Csa2Error):
        S.prefix_attn(b, gr, q, k, v, 2500,
                      workspace=torch.empty(sides * part - 1, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("shift", [1, 7, 300])
def test_rows_close_up_in_place_through_another_view(shift):
    """The destination is a view further down the same memory, with starts that
    name the same rows: moved in order, as with one tensor for both."""
    rows, keep, heads = [6000, 900, 40], 4000, 2
    start, pool = R.starts(rows, gap=320)
    mass = torch.rand((heads, pool), device=DEV)
    c = torch.randn((pool, heads, 64), device=DEV).to(BF)
    idx, new_len = S.evict_select(_i64(start), _i64(rows), mass, keep, 2, 20)
    want = c.clone()
    for r, n in enumerate(rows):
        m = min(n, keep)
        for h in range(heads):
            want[start[r]:start[r] + m, h] = c[start[r] + idx[r, h, :m].long(), h]
    for down in (True, False):
        x, w = c.clone(), mass.clone()
        src, dst = (x, x[shift:]) if down else (x[shift:], x)
        s0 = _i64(start) - (0 if down else shift)
        d0 = _i64(start) - (shift if down else 0)
        d = _derr()
        S.evict_rows(idx, new_len, s0, d0, [(src, dst)], d_err=d)
        assert int(d.item()) == 0 and torch.equal(x, want)


def test_rows_between_columns_of_longer_rows():
    """Source and destination side by side in the same rows."""
    rows, heads = [700, 60], 3
    start, pool = R.starts(rows)
    x = torch.randn((pool, 2, heads, 32), device=DEV).to(BF)
    mass = torch.rand((heads, pool), device=DEV)
    idx, new_len = S.evict_select(_i64(start), _i64(rows), mass, 100, 2, 20)
    for a, b in ((0, 1), (1, 0)):
        y = x.clone()
        S.evict_rows(idx, new_len, _i64(start), _i64([0, 300]), [(y[:, a], y[:, b])])
        want = x.clone()
        for r, to in enumerate((0, 300)):
            m = int(new_len[r])
            for h in range(heads):
                want[to:to + m, b, h] = x[start[r] + idx[r, h, :m].long(), a, h]
        assert torch.equal(y, want)


# ---------------------------------------------------------------------------
# outputs in the queries' place, or between the rows of an input
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("heads,kv,dim,dtype", [(16, 2, 128, BF), (6, 2, 64, HF), (20, 1, 64, BF)])
@pytest.mark.parametrize("new", [[1, 1, 1], [3, 0, 40], [300, 17, 129], [0, 1, 2]])
@pytest.mark.parametrize("call", ["prompt", "prefix", "groups"])
def test_output_in_the_queries_place(heads, kv, dim, dtype, new, call):
    rows = [max(n, 400) for n in new]
    b, _, start, q, k, v = _inputs(new, rows, heads, kv, dim, dtype, seed=dim, lead=1, tail=2,
                                   extra=[500])
    gr = dict(num_groups=1, cu_group=_i32([0, 2]), max_prefix=500, prefix_start=_i64(start[-1:]),
              prefix_len=_i64([500])) if call == "groups" else None

    def run(q, out):
        if call == "prompt":
            return S.prompt_attn(b, q, k, v, out=out)
        return S.prefix_attn(b, gr, q, k, v, 400, out=out)

    out = q.clone()                      # rows of no request keep their values
    want, lse = run(q, out)
    x = q.clone()
    got, l2 = run(x, x)
    n = slice(1, 1 + sum(new))
    assert torch.equal(got.nan_to_num(9.0), want.nan_to_num(9.0)) and torch.equal(lse[n], l2[n])


def test_output_between_the_rows_of_an_input():
    """One row of output beside the one cache row that is read in longer rows."""
    x = torch.randn((40, 4, 64), device=DEV).to(BF)          # k, v and two heads of room
    q = torch.randn((1, 2, 64), device=DEV).to(BF)
    b, _ = R.batch([1], [40], [0], DEV)
    want, _ = S.prompt_attn(b, q, x[:, :1], x[:, 1:2])
    y = x.clone()
    S.prompt_attn(b, q, y[:, :1], y[:, 1:2], out=y[7:8, 2:])
    assert torch.equal(y[7, 2:], want[0])
    y[7, 2:] = x[7, 2:]
    assert torch.equal(x, y)


# ---------------------------------------------------------------------------
# shapes
# ---------------------------------------------------------------------------

def test_tensors_of_another_layout_are_refused():
    """As many values as the call wants, or more, in rows of another length."""
    b, _, start, q, k, v = _inputs([2, 1], [40, 30], 4, 2, 64, BF)
    pool = k.shape[0]
    out, lse = S.prompt_attn(b, q, k, v)
    mass = S.attn_mass(b, q, k, lse, 40)
    idx, n = S.evict_select(b["kv_start"], b["kv_len"], mass, 8)
    e = lambda *s: torch.empty(s, device=DEV)              # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)   # noqa: E731
    o = lambda *s: torch.empty(s, dtype=BF, device=DEV)    # noqa: E731
    for call in (lambda: S.prompt_attn(b, q, k, v, out=o(3, 4, 128)),
                 lambda: S.prompt_attn(b, q, k, v, out=o(3, 8, 64)),
                 lambda: S.prefix_attn(b, None, q, k, v, 40, lse=e(3, 5)),
                 lambda: S.attn_mass(b, q, k, e(3, 8), 40),
                 lambda: S.attn_mass(b, q, k, lse, 40, mass=e(2, pool + 1)),
                 lambda: S.attn_mass(b, q, k, lse, 40, mass_in=e(2, pool + 1)),
                 lambda: S.attn_mass(b, q, k, lse, 40, mass=e(pool, 2)),
                 lambda: S.evict_select(b["kv_start"], b["kv_len"], mass, 8, idx=i(2, 2, 9)),
                 lambda: S.evict_select(b["kv_start"], b["kv_len"], mass, 8, idx=i(4, 1, 8)),
                 lambda: S.csa2_evict_rows(2, 2, i(2, 4, 8), 8, n, b["kv_start"], b["kv_start"],
                                           [(k, k)], None)):
        with pytest.raises(S.Csa2Error):
            call()
    # more rows, or flat
    big = torch.empty((5, 4, 64), dtype=BF, device=DEV)
    S.prompt_attn(b, q, k, v, out=big, lse=e(99))
    assert torch.equal(big[:3], out)
    flat = torch.zeros(2 * pool, device=DEV)
    S.attn_mass(b, q, k, lse.view(-1), 40, mass=flat)
    assert torch.equal(flat.view(2, pool), mass)


def test_calls_on_a_side_stream_are_captured():
    """Outputs and workspaces allocated in a capture, on a stream forked in it."""
    b, _, start, q, k, v = _inputs([1] * 9, [300] * 9, 8, 2, 128, BF)
    weight = torch.rand((2, k.shape[0]), device=DEV)

    def calls(stream):
        out, lse = S.prefix_attn(b, None, q, k, v, 300, stream=stream)
        o2, _ = S.prompt_attn(b, q, k, v, stream=stream)
        mass = S.attn_mass(b, q, k, lse, 300, stream=stream)
        idx, n = S.evict_select(b["kv_start"], b["kv_len"], weight, 100, 3, 5, stream=stream)
        return out, lse, o2, mass, idx, n

    want = calls(None)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = calls(side)
        main.wait_stream(side)
    for _ in range(2):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert torch.equal(x, y)


# ---------------------------------------------------------------------------
# sizes that choose rare variants
# ---------------------------------------------------------------------------

def _check_masses(q, k, lse, mass, cu, start, new, rows, scale, which):
    for r in which:
        at = slice(start[r], start[r] + rows[r])
        last = rows[r] - new[r] + torch.arange(new[r], device=DEV)
        w, tol = R.mass(q[cu[r]:cu[r + 1]], k[at], lse[cu[r]:cu[r + 1]], scale, last)
        d = (mass[:, at].double() - w).abs()
        assert (d <= tol + w * 2.0 ** -23 + 1e-30).all(), r


@pytest.mark.parametrize("heads,dim,dtype,new", [
    (8, 64, HF, 70), (24, 128, BF, 131), (64, 128, BF, 1), (128, 64, BF, 3)])
def test_mass_four_key_tiles_an_item(heads, dim, dtype, new):
    """Enough rows that an item has four key tiles, the last of it in part."""
    kv, rows = 8, [9001, 7300, 8000, 7937, 1, 130, 12345, 15100]
    n = [min(new, m) for m in rows]
    assert (sum(rows) // 128 + 8) * kv >= 4 * 6 * 152
    b, cu, start, q, k, v = _inputs(n, rows, heads, kv, dim, dtype, seed=new)
    _, lse = S.prompt_attn(b, q, k, v)
    mass = S.attn_mass(b, q, k, lse, max(rows))
    _check_masses(q, k, lse, mass, cu, start, n, rows, dim ** -0.5, range(8))
    assert torch.equal(mass, S.attn_mass(b, q, k, lse, 10 ** 9))


def test_mass_of_many_requests_shortens_the_ring():
    """Thousands of requests leave shared memory for three key tiles: items that
    were meant to have four have two."""
    reqs = 8000
    rows = [1 + (53 * i) % 90 if i % 40 else 300 + i % 500 for i in range(reqs)]
    b, cu, start, q, k, v = _inputs([1] * reqs, rows, 128, 1, 128, BF, seed=3)
    _, lse = S.prompt_attn(b, q, k, v)
    mass = S.attn_mass(b, q, k, lse, max(rows))
    _check_masses(q, k, lse, mass, cu, start, [1] * reqs, rows, 128 ** -0.5,
                  list(range(0, reqs, 200)) + [1, 7, 3999, 7999])
    # every query's weights sum to one
    assert abs(float(mass.double().sum()) - reqs * 128) <= 1e-4 * reqs * 128


@pytest.mark.parametrize("rows,pool", [(12400, 0), (16500, 0), (20600, 0), (24700, 0), (28800, 0),
                                       (40000, 0), (700, 40000)])
@pytest.mark.parametrize("ties", [False, True])
def test_select_by_clusters_of_every_size(rows, pool, ties):
    """Three to eight CTAs to a request and head; a short request in a long pool."""
    keep, sink, recent, heads = min(rows // 3, 4000), 7, 100, 8
    g = torch.Generator(device=DEV).manual_seed(rows)
    mass = torch.rand((heads, max(rows + 9, pool)), generator=g, device=DEV)
    if ties:
        mass = (mass * 50).floor()
    for start in (0, 9):
        idx, n = S.evict_select(_i64([start]), _i64([rows]), mass, keep, sink, recent)
        assert n.tolist() == [keep]
        for h in range(heads):
            order = mass[h, start:start + rows].clone()
            order[:sink] = order[rows - recent:] = math.inf
            want = torch.sort(order, descending=True, stable=True).indices[:keep].sort().values
            assert torch.equal(idx[0, h].long(), want)


def test_mass_of_whole_prompts():
    """Every query of two prompts, many query tiles to a key tile."""
    rows = [2500, 701]
    b, cu, start, q, k, v = _inputs(rows, rows, 8, 1, 128, BF, seed=12)
    _, lse = S.prompt_attn(b, q, k, v)
    mass = S.attn_mass(b, q, k, lse, 2500)
    _check_masses(q, k, lse, mass, cu, start, rows, rows, 128 ** -0.5, range(2))
    assert abs(float(mass.double().sum()) - 3201 * 8) <= 1e-4 * 3201 * 8


def test_mass_without_queries_is_carried_over():
    b, _, start, _, k, _ = _inputs([0, 0], [300, 40], 4, 2, 64, BF)
    old = torch.rand((2, k.shape[0]), device=DEV)
    new = torch.full_like(old, 5.0)
    q = torch.empty((0, 4, 64), dtype=BF, device=DEV)
    S.attn_mass(b, q, k, torch.empty((0, 4), device=DEV), 300, mass_in=old, mass=new)
    held = torch.zeros(k.shape[0], dtype=torch.bool, device=DEV)
    for s, n in zip(start, (300, 40)):
        held[s:s + n] = True
    assert torch.equal(new[:, held], old[:, held]) and (new[:, ~held] == 5).all()


@pytest.mark.parametrize("new", [1, 5])
def test_many_groups_and_many_key_heads(new):
    """More groups than a warp has lanes, every third request in none; 200 key
    heads of their own."""
    reqs, kv, dim = 120, 200, 64
    rows = [new + 3 * i % 50 for i in range(reqs)]
    pre = [30 + i for i in range(reqs // 3)]
    b, cu, start, q, k, v = _inputs([new] * reqs, rows, kv, kv, dim, BF, seed=new, extra=pre)
    # group g: requests 3 g and 3 g + 1, behind it a group of request 3 g + 2
    # without a prefix
    cug, ps, pl = [0], [], []
    for g in range(reqs // 3):
        cug += [3 * g + 2, 3 * g + 3]
        ps += [start[reqs + g], 0]
        pl += [pre[g], 0]
    gr = dict(num_groups=len(pl), cu_group=_i32(cug), prefix_start=_i64(ps), prefix_len=_i64(pl),
              max_prefix=max(pre))
    out, lse = S.prefix_attn(b, gr, q, k, v, max(rows))
    for r in list(range(0, reqs, 11)) + [2, 119]:
        at = slice(cu[r], cu[r + 1])
        kk, vv, off = k[start[r]:start[r] + rows[r]], v[start[r]:start[r] + rows[r]], 0
        if r % 3 != 2:
            p, off = start[reqs + r // 3], pre[r // 3]
            kk, vv = torch.cat([k[p:p + off], kk]), torch.cat([v[p:p + off], vv])
        last = off + rows[r] - new + torch.arange(new, device=DEV)
        ref = R.attend(q[at], kk, vv, dim ** -0.5, last)
        R.check_attention(out[at], lse[at], ref, BF, kk.shape[0])


@pytest.mark.parametrize("new", [[1, 1], [70, 3]])
def test_without_lse_and_without_groups_in_a_dict(new):
    b, _, _, q, k, v = _inputs(new, [200, 90], 8, 2, 64, HF, seed=2)
    none = dict(num_groups=0, cu_group=_i32([0]), prefix_start=_i64([]), prefix_len=_i64([]),
                max_prefix=0)
    out, lse = S.prompt_attn(b, q, k, v, want_lse=False)
    assert lse is None and torch.equal(out, S.prompt_attn(b, q, k, v)[0])
    want = S.prefix_attn(b, None, q, k, v, 200)
    out, lse = S.prefix_attn(b, none, q, k, v, 200, want_lse=False)
    assert lse is None and torch.equal(out, want[0])
    got = S.prefix_attn(b, none, q, k, v, 200)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_runs_over_one_another_past_two_to_the_32_items():
    """Runs of a malformed batch that all hold every row: more items than the grid
    has, or 32 bits; flagged, and every row written is one of the batch's."""
    reqs, num_q = 140001, 1 << 16
    q = torch.randn((num_q, 20, 64), device=DEV).to(BF)
    k = torch.randn((100, 1, 64), device=DEV).to(BF)
    b = dict(num_q=num_q, num_req=reqs, kv_start=_i64([0] * reqs), kv_len=_i64([100] * reqs),
             cu_q=_i32([0, num_q] * (reqs // 2 + 1)))
    room = torch.full((num_q + 4096, 20, 64), 7.0, dtype=BF, device=DEV)
    d = _derr()
    S.prompt_attn(b, q, k, k, out=room[2048:2048 + num_q], d_err=d)
    assert int(d.item()) == S.DERR_BAD_EXTEND
    assert (room[:2048] == 7).all() and (room[2048 + num_q:] == 7).all()


@pytest.mark.parametrize("to,ok", [
    ([100, 600, 900], [1, 1, 1]),              # closed up in place
    ([1500, 2500, 3500], [1, 1, 1]),           # elsewhere in the same tensor
    ([70, 600, 900], [1, 1, 1]),               # the first moves down over itself
    ([130, 600, 900], [0, 1, 1]),              # up over itself
    ([100, 200, 300], [1, 0, 0]),              # closed up over the others' sources
    ([850, 1500, 1900], [0, 1, 1]), ([0, 1500, 899], [1, 1, 1])])
def test_rows_moved_within_one_tensor(to, ok):
    """Requests at 100, 600 and 900 of 400, 250 and 90 rows, of which the first
    and the last among others stay."""
    start, rows, keep, heads = [100, 600, 900], [400, 250, 90], 60, 2
    c = torch.randn((4000, heads, 32), device=DEV).to(BF)
    idx = torch.empty((3, heads, keep), dtype=torch.int32, device=DEV)
    for r, n in enumerate(rows):
        for h in range(heads):
            pick = torch.randperm(n - 2, device=DEV)[:keep - 2] + 1
            idx[r, h] = torch.cat([pick, torch.tensor([0, n - 1], device=DEV)]).sort().values
    want = c.clone()
    for r in range(3):
        for h in range(heads):
            if ok[r]:
                want[to[r]:to[r] + keep, h] = c[start[r] + idx[r, h].long(), h]
    d = _derr()
    S.evict_rows(idx, _i64([keep] * 3), _i64(start), _i64(to), [(c, c)], d_err=d)
    assert int(d.item()) == (0 if all(ok) else S.DERR_RANGE_ROW)
    assert torch.equal(c, want)
