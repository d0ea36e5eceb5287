"""Accumulated attention weight, selection of the rows that stay and their
move (csa2_attn_mass, csa2_evict_select, csa2_evict_rows), and the chain they
are used in: prompt, weight, eviction, decode on what is left."""
import math

import pytest
import torch

import sparse_attention_prefill_gb300 as S
from tests import dense_ref as R
from tests.test_gpu_dense_attn import BF, DEV, HF, _derr, _inputs

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# accumulated attention weight
# ---------------------------------------------------------------------------

def _check_mass(b, cu, start, q, k, new, rows, scale, lse, mass, old, untouched):
    seen = torch.zeros(k.shape[0], dtype=torch.bool, device=DEV)
    for r in range(len(new)):
        at = slice(start[r], start[r] + rows[r])
        seen[at] = True
        last = rows[r] - new[r] + torch.arange(new[r], device=DEV)
        w, tol = R.mass(q[cu[r]:cu[r + 1]], k[at], lse[cu[r]:cu[r + 1]], scale, last)
        base = 0.0 if old is None else old[:, at].double()
        # the old value's addition rounds once more
        d = (mass[:, at].double() - base - w).abs()
        t = tol + (w + base) * 2.0 ** -23 + 1e-30
        assert (d <= t).all(), (r, float((d - t).max()))
    assert (mass[:, ~seen] == untouched).all()


@pytest.mark.parametrize("heads,kv,dim,dtype", [
    (8, 1, 128, BF), (64, 8, 128, BF), (6, 2, 64, HF), (4, 4, 128, HF), (5, 1, 64, BF),
    (128, 1, 64, BF), (28, 4, 128, BF)])
@pytest.mark.parametrize("acc", [False, True])
def test_mass_ragged(heads, kv, dim, dtype, acc):
    new = [130, 1, 0, 37, 128, 9, 260, 5]
    rows = [130, 1, 40, 300, 129, 4, 519, 0]
    b, cu, start, q, k, v = _inputs(new, rows, heads, kv, dim, dtype, lead=3, tail=4)
    _, lse = S.prompt_attn(b, q, k, v)
    lse[:cu[0]] = lse[cu[-1]:] = math.nan
    old = torch.rand((kv, k.shape[0]), device=DEV) if acc else None
    mass = torch.full((kv, k.shape[0]), 7.0, device=DEV)
    d = _derr()
    S.attn_mass(b, q, k, lse, 519, mass_in=old, mass=mass, d_err=d)
    assert int(d.item()) == 0
    _check_mass(b, cu, start, q, k, new, rows, dim ** -0.5, lse, mass, old, 7.0)
    if acc:                                            # in place, the same bits
        S.attn_mass(b, q, k, lse, 519, mass_in=old, mass=old)
        for r in range(len(new)):
            at = slice(start[r], start[r] + rows[r])
            assert torch.equal(old[:, at], mass[:, at])


@pytest.mark.parametrize("reqs,m,heads,kv", [(1, 5000, 8, 1), (70, 300, 64, 8), (200, 129, 4, 4)])
def test_mass_decode(reqs, m, heads, kv):
    rows = [max(1, m - 3 * i) for i in range(reqs)]
    b, cu, start, q, k, v = _inputs([1] * reqs, rows, heads, kv, 128, BF, seed=m)
    _, lse = S.prefix_attn(b, None, q, k, v, m)
    mass = S.attn_mass(b, q, k, lse, m)
    _check_mass(b, cu, start, q, k, [1] * reqs, rows, 128 ** -0.5, lse, mass, None, 0.0)
    # every query's weights sum to one
    assert abs(float(mass.double().sum()) - reqs * heads) <= 1e-4 * reqs * heads


@pytest.mark.parametrize("hint", [0, 40, 10 ** 9])
def test_mass_hint_only_steers_the_grid(hint):
    """Many rows and windows of queries, one, two and four key tiles an item."""
    rows = [2000 + 700 * i for i in range(8)]
    b, cu, start, q, k, v = _inputs([70] * 8, rows, 32, 8, 64, BF, seed=4)
    _, lse = S.prompt_attn(b, q, k, v)
    mass = S.attn_mass(b, q, k, lse, hint)
    _check_mass(b, cu, start, q, k, [70] * 8, rows, 64 ** -0.5, lse, mass, None, 0.0)
    assert torch.equal(mass, S.attn_mass(b, q, k, lse, hint))


def test_mass_counts_lse_of_a_joint_softmax_and_skips_empty_rows():
    """lse from elsewhere; -inf adds nothing though the row sees keys."""
    b, cu, start, q, k, _ = _inputs([6], [200], 4, 2, 64, BF, seed=2)
    lse = torch.randn((6, 4), device=DEV) + 8
    lse[2, 1] = -math.inf
    mass = S.attn_mass(b, q, k, lse, 200)
    _check_mass(b, cu, start, q, k, [6], [200], 64 ** -0.5, lse, mass, None, 0.0)


def test_mass_bad_requests_and_wait():
    b, cu, start, q, k, v = _inputs([20, 30], [20, 60], 4, 2, 64, BF)
    _, lse = S.prompt_attn(b, q, k, v)
    want = S.attn_mass(b, q, k, lse, 60)
    d = _derr()
    mass = torch.full_like(want, 7.0)
    S.attn_mass(dict(b, kv_start=b["kv_start"] + torch.tensor([0, 10 ** 9], device=DEV)), q, k,
                lse, 60, mass=mass, d_err=d)
    assert int(d.item()) == S.DERR_RANGE_ROW
    one = slice(start[0], start[0] + 20)
    assert torch.equal(mass[:, one], want[:, one])
    mass[:, one] = 7
    assert (mass == 7).all()
    S.set_wait_limit_ns(1)
    try:
        d = _derr()
        for _ in range(3):
            S.attn_mass(b, q, k, lse, 60, d_err=d)
        torch.cuda.synchronize()
    finally:
        S.set_wait_limit_ns(0)
    assert int(d.item()) & S.DERR_TIMEOUT
    assert torch.equal(S.attn_mass(b, q, k, lse, 60), want)


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------

def _select_ref(mass, start, rows, keep, sink, recent):
    """Stable order on the host: NaN below everything, ties to the lower row."""
    r, h = len(rows), mass.shape[0]
    idx = torch.full((r, h, keep), -1, dtype=torch.int32)
    m = mass.cpu().double()
    for i, n in enumerate(rows):
        for a in range(h):
            x = m[a, start[i]:start[i] + n].tolist()
            if n <= keep:
                ids = list(range(n))
            else:
                must = set(range(sink)) | set(range(n - recent, n))
                rest = [j for j in range(n) if j not in must]
                rest.sort(key=lambda j: (-math.inf if x[j] != x[j] else x[j], x[j] == x[j], -j),
                          reverse=True)
                ids = sorted(must | set(rest[:keep - sink - recent]))
            idx[i, a, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
    return idx.to(DEV)


def _select(mass, start, rows, keep, sink, recent, d=None):
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device=DEV)    # noqa: E731
    return S.evict_select(i64(start), i64(rows), mass, keep, sink, recent, d_err=d)


@pytest.mark.parametrize("rows,heads,keep,sink,recent", [
    ([1, 0, 2], 1, 1, 0, 0), ([300, 12, 64, 65], 3, 64, 4, 16), ([5000], 2, 1023, 0, 1),
    ([2048, 2049], 8, 2048, 100, 1948), ([700] * 40, 8, 350, 1, 7), ([9000], 1, 8999, 0, 0),
    ([4097, 100], 2, 33, 33, 0), ([4097], 2, 33, 0, 33)])
@pytest.mark.parametrize("kind", ["normal", "ties", "special"])
def test_select(rows, heads, keep, sink, recent, kind):
    g = torch.Generator(device=DEV).manual_seed(len(rows) + keep)
    start, pool = R.starts(rows)
    mass = torch.randn((heads, pool), generator=g, device=DEV).exp()
    if kind == "ties":
        mass = (mass * 2).floor()
    if kind == "special":
        u = torch.rand((heads, pool), generator=g, device=DEV)
        mass = torch.where(u < 0.2, math.nan, torch.where(u < 0.4, math.inf, torch.where(
            u < 0.5, -math.inf, torch.where(u < 0.6, -0.0, torch.where(u < 0.7, 0.0, -mass)))))
    d = _derr()
    idx, new_len = _select(mass, start, rows, keep, sink, recent, d)
    assert int(d.item()) == 0
    assert new_len.tolist() == [min(n, keep) for n in rows]
    assert torch.equal(idx, _select_ref(mass, start, rows, keep, sink, recent))


def test_select_long_rows():
    """Slices longer than a CTA holds; checked by counting."""
    n, keep, sink, recent = 400000, 150001, 10, 500
    mass = torch.randn((2, n), device=DEV).exp()
    mass[1] = (mass[1] * 4).floor()
    idx, new_len = _select(mass, [0], [n], keep, sink, recent)
    assert new_len.tolist() == [keep]
    for h in range(2):
        order = mass[h].clone()
        order[:sink] = order[n - recent:] = math.inf
        want = torch.sort(order, descending=True, stable=True).indices[:keep].sort().values
        assert torch.equal(idx[0, h].long(), want)


def test_select_bad_request_is_flagged():
    mass = torch.rand((2, 100), device=DEV)
    d = _derr()
    idx, new_len = _select(mass, [0, 90, -1, 0], [50, 50, 5, -2], 20, 1, 1, d)
    assert int(d.item()) == S.DERR_RANGE_ROW and new_len.tolist() == [20, 0, 0, 0]
    assert (idx[1:] == -1).all() and (idx[0] >= 0).all()


# ---------------------------------------------------------------------------
# the move
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dim,dtype,heads", [(128, BF, 8), (64, HF, 1), (6, torch.float32, 3),
                                             (512, torch.uint8, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_move(dim, dtype, heads, in_place):
    rows, keep = [1500, 40, 3000, 0], 700
    start, pool = R.starts(rows)
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device=DEV)    # noqa: E731
    mass = torch.rand((heads, pool), device=DEV)
    k = (torch.randn((pool, heads, dim), device=DEV) * 50).to(dtype)
    scale = torch.rand((pool, heads, 3), device=DEV)
    idx, new_len = _select(mass, start, rows, keep, 2, 20)
    src = [k, scale, mass.t()]
    if in_place:
        dst, to = [x.clone() for x in src[:2]] + [mass.clone().t()], start
        orig = [x.clone() for x in dst]
        pairs = [(x, x) for x in dst]
    else:
        to = [3 + keep * i for i in range(4)]
        dst = [torch.full((keep * 4 + 9,) + x.shape[1:], 9, device=DEV).to(x.dtype) for x in src]
        orig = [x.clone() for x in dst]
        pairs = list(zip(src, dst))
    d = _derr()
    S.evict_rows(idx, new_len, i64(start), i64(to), pairs, d_err=d)
    assert int(d.item()) == 0
    for x, o, y in zip(src, orig, dst):
        want = o.clone()
        for r, n in enumerate(rows):
            m = min(n, keep)
            for h in range(heads):
                want[to[r]:to[r] + m, h] = x[start[r] + idx[r, h, :m].long(), h]
        assert torch.equal(y, want)


def test_rows_interleaved_cache_in_place_on_a_side_stream():
    """K and V as views of one buffer, closed up in place on another stream."""
    rows, keep, heads = [900, 300], 128, 4
    start, pool = R.starts(rows)
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device=DEV)    # noqa: E731
    c = torch.randn((pool, 2, heads, 64), device=DEV).to(BF)
    c0 = c.clone()
    mass = torch.rand((heads, pool), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    st = i64(start)
    idx, new_len = S.evict_select(st, i64(rows), mass, keep, 1, 1, stream=side)
    S.evict_rows(idx, new_len, st, st, [(c[:, 0], c[:, 0]), (c[:, 1], c[:, 1])], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = c0.clone()
    for r, s in enumerate(start):
        for h in range(heads):
            want[s:s + keep, :, h] = c0[s + idx[r, h].long(), :, h]
    assert torch.equal(c, want)


def test_rows_bad_indices_are_flagged():
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device=DEV)    # noqa: E731
    k = torch.arange(40, dtype=torch.float32, device=DEV).view(10, 1, 4)
    dst = torch.full((3, 1, 4), -1.0, device=DEV)
    idx = torch.tensor([[[1, -1, 99, 4, 5]]], dtype=torch.int32, device=DEV)
    d = _derr()
    S.evict_rows(idx, i64([5]), i64([0]), i64([0]), [(k, dst)], d_err=d)
    assert int(d.item()) == S.DERR_RANGE_ROW
    assert torch.equal(dst[0], k[1]) and (dst[1:] == -1).all()
    S.evict_rows(idx, i64([-3]), i64([0]), i64([0]), [(k, dst)])
    d = _derr()
    S.evict_rows(idx, i64([1]), i64([0]), i64([-1]), [(k, dst)], d_err=d)
    assert int(d.item()) == S.DERR_RANGE_ROW


# ---------------------------------------------------------------------------
# the chain
# ---------------------------------------------------------------------------

def test_prompt_weight_eviction_decode_chain():
    """Two requests behind one system prompt: their prompts, the weight that
    the 128-token tails (csa2_tail_layout) put on their own rows, eviction of
    K, V and weight in place, and a decode step over the prefix and the rows
    left, with its weight added; the whole run captured and replayed too."""
    h, kv, dim, keep = 8, 2, 128, 256
    rows, pre = [900, 500], 700
    b, cu, start, q, k, v = _inputs(rows, rows, h, kv, dim, BF, seed=6, extra=[pre])
    k0, v0 = k.clone(), v.clone()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)    # noqa: E731
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device=DEV)    # noqa: E731
    gr = dict(num_groups=1, cu_group=i32([0, 2]), prefix_start=i64(start[-1:]),
              prefix_len=i64([pre]), max_prefix=pre)
    tail = S.tail_layout(i32(rows), i64(rows), 128)
    qd = torch.randn((2, h, dim), device=DEV).to(BF)
    qt = torch.empty((256, h, dim), dtype=BF, device=DEV)
    lt = torch.empty((256, h), dtype=torch.float32, device=DEV)
    bt = dict(b, num_q=256, cu_q=tail["cu_tail"])
    kept = torch.empty(2, dtype=torch.int64, device=DEV)
    idx = torch.empty((2, kv, keep), dtype=torch.int32, device=DEV)
    bd = dict(num_q=2, num_req=2, cu_q=i32([0, 1, 2]), kv_start=b["kv_start"], kv_len=kept)
    mass = torch.zeros((kv, k.shape[0]), device=DEV)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    d = _derr()

    def chain():
        k.copy_(k0)
        v.copy_(v0)
        out, lse = S.prefix_attn(b, gr, q, k, v, max(rows), d_err=d)
        S.rows_gather(tail["src_row"][:256], q, qt, d_err=d)
        S.rows_gather(tail["src_row"][:256], lse, lt, d_err=d)
        S.attn_mass(bt, qt, k, lt, max(rows), mass=mass, d_err=d)
        S.evict_select(b["kv_start"], b["kv_len"], mass, keep, 4, 32, idx=idx, new_len=kept,
                       d_err=d)
        S.evict_rows(idx, kept, b["kv_start"], b["kv_start"],
                     [(k, k), (v, v), (mass.t(), mass.t())], d_err=d)
        od, ld = S.prefix_attn(bd, gr, qd, k, v, keep, workspace=ws, d_err=d)
        S.attn_mass(bd, qd, k, ld, keep, mass_in=mass, mass=mass, d_err=d)
        return out, lse, od, ld

    out, lse, od, ld = chain()
    assert int(d.item()) == 0
    scale = dim ** -0.5
    for r in range(2):
        at = slice(start[r], start[r] + rows[r])
        p = slice(start[2], start[2] + pre)
        ref = R.attend(q[cu[r]:cu[r + 1]], torch.cat([k0[p], k0[at]]), torch.cat([v0[p], v0[at]]),
                       scale, pre + torch.arange(rows[r], device=DEV))
        R.check_attention(out[cu[r]:cu[r + 1]], lse[cu[r]:cu[r + 1]], ref, BF, pre + rows[r])
        tl = slice(cu[r + 1] - 128, cu[r + 1])
        w, tol = R.mass(q[tl], k0[at], lse[tl], scale,
                        torch.arange(rows[r] - 128, rows[r], device=DEV))
        for g in range(kv):
            ids = idx[r, g].long()
            assert (ids[1:] > ids[:-1]).all() and ids[:4].tolist() == [0, 1, 2, 3]
            assert ids[-32:].tolist() == list(range(rows[r] - 32, rows[r]))
            # no row left out weighs more than one chosen, beyond the bound
            rest = torch.ones(rows[r], dtype=torch.bool, device=DEV)
            rest[ids] = False
            assert float((w[g] - tol[g])[rest].max()) <= float((w[g] + tol[g])[ids[4:-32]].min())
            src = start[r] + ids
            to = slice(start[r], start[r] + keep)
            assert torch.equal(k[to, g], k0[src, g]) and torch.equal(v[to, g], v0[src, g])
        to = slice(start[r], start[r] + keep)
        ref = R.attend(qd[r:r + 1], torch.cat([k0[p], k[to]]), torch.cat([v0[p], v[to]]), scale,
                       torch.tensor([pre + keep - 1], device=DEV))
        R.check_attention(od[r:r + 1], ld[r:r + 1], ref, BF, pre + keep)
        w2, tol2 = R.mass(qd[r:r + 1], k[to], ld[r:r + 1], scale,
                          torch.tensor([keep - 1], device=DEV))
        for g in range(kv):
            ids = idx[r, g].long()
            both = w[g][ids] + w2[g]
            t = tol[g][ids] + tol2[g] + both * 2.0 ** -22
            assert ((mass[g, to].double() - both).abs() <= t).all()
    m1 = mass.clone()
    graph = torch.cuda.CUDAGraph()
    mass.zero_()
    with torch.cuda.graph(graph):
        g_out = chain()
    mass.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip((out, lse, od, ld), g_out):
        assert torch.equal(x, y)
    for r in range(2):
        to = slice(start[r], start[r] + keep)
        assert torch.equal(mass[:, to], m1[:, to])
