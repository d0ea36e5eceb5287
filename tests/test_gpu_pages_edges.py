"""Calls on 8-bit pages at the edges: waits that run out, streams, graphs, workspaces,
arguments in place, pages far out, empty caches, other layouts."""
import math

import pytest
import torch

import sparse_attention_prefill_gb300 as S
from tests import page_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


def _derr():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _normal(shape, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _case(new, rows, heads, kv, dim, page, dtype, seed=0, **kw):
    b, cu = R.batch(new, rows, DEV, **kw)
    c = R.make_cache(rows, kv, dim, page, seed=seed)
    return b, cu, c, _normal((b["num_q"], heads, dim), dtype, seed + 1)


# single tokens of up to 8 and 16 heads and more, few and many rows to a request
KINDS = [([1] * 9, [900, 70, 1, 3000, 200, 17, 64, 33, 5000], 8, 1),
         ([1] * 3, [2000, 31, 700], 24, 2), ([1] * 4, [900, 40, 2500, 7], 40, 1),
         ([5, 2], [800, 3000], 8, 2), ([400, 3, 130, 1], [900, 700, 130, 2000], 8, 2)]


@pytest.mark.parametrize("dim,page,dtype", [(128, 64, BF), (64, 16, HF)])
def test_waits_of_every_length_run_out_and_recover(dim, page, dtype):
    """Limits around the time that the kernels' steps take, so that a wait runs out in any
    role and at any step: the calls end and the next ones are right."""
    cases = [_case(n, r, h, kv, dim, page, dtype, seed=i) for i, (n, r, h, kv) in enumerate(KINDS)]
    none = torch.empty(0, dtype=torch.uint8, device=DEV)

    def calls(d):
        return [t for b, _, c, q in cases for ws in (None, none)
                for t in S.page_attn(b, q, c, max_kv=5000, workspace=ws, d_err=d)]

    want = calls(None)
    d = _derr()
    try:
        for limit in (1, 300, 700, 1500, 3000, 6000, 12000, 25000, 50000, 99999, 100001, 200000):
            S.set_wait_limit_ns(limit)
            for _ in range(3):
                calls(d)
            torch.cuda.synchronize()
    finally:
        S.set_wait_limit_ns(0)
    assert int(d.item()) & S.DERR_TIMEOUT
    d = _derr()
    got = calls(d)
    assert int(d.item()) == 0
    for x, y in zip(want, got):
        assert torch.equal(x, y)


@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_same_bits_whatever_the_workspace_held(kind):
    """The same call gives the same bits, on another stream and in a graph, too, and with
    any contents of the workspace; the sharing of caches changes the last bits alone."""
    new, rows, heads, kv = KINDS[kind]
    b, cu, c, q = _case(new, rows, heads, kv, 128, 32, BF, seed=kind)
    out, lse = S.page_attn(b, q, c, max_kv=5000)
    need = S.csa2_page_attn_workspace(b["num_q"], b["num_req"], heads, kv, 128, 5000)
    for fill in (0, 255):
        ws = torch.full((need + 512,), fill, dtype=torch.uint8, device=DEV)
        o, l = S.page_attn(b, q, c, max_kv=5000, workspace=ws)
        assert torch.equal(o, out) and torch.equal(l, lse)
        assert (ws[need:] == fill).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, l = S.page_attn(b, q, c, max_kv=5000, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, out) and torch.equal(l, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, l = S.page_attn(b, q, c, max_kv=5000)
    o.zero_()
    for _ in range(2):
        graph.replay()
    assert torch.equal(o, out) and torch.equal(l, lse)
    # a hint that is too short changes what is shared, not what is computed
    for hint in (0, 100):
        o, l = S.page_attn(b, q, c, max_kv=hint)
        assert torch.allclose(l, lse, rtol=0, atol=1e-5)
        assert torch.allclose(o.float(), out.float(), rtol=2.0 ** -7, atol=1e-2)


def test_two_calls_at_once_in_one_graph():
    """Two batches on two streams of one graph, a workspace each."""
    cases = [_case(*KINDS[i][:2], *KINDS[i][2:], 64, 32, HF, seed=i) for i in (0, 3)]
    want = [S.page_attn(b, q, c, max_kv=5000) for b, _, c, q in cases]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = [S.page_attn(b, q, c, max_kv=5000, stream=s)
               for (b, _, c, q), s in zip(cases, (None, side))]
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(5):
        for o, l in got:
            o.zero_(), l.zero_()
        graph.replay()
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_output_in_the_queries_place_and_strided_queries(kind):
    new, rows, heads, kv = KINDS[kind]
    b, cu, c, q = _case(new, rows, heads, kv, 64, 16, BF, seed=kind)
    out, lse = S.page_attn(b, q, c, max_kv=5000)
    wide = _normal((q.shape[0], heads + 3, 64), BF, 9)
    wide[:, 1:1 + heads] = q
    o, l = S.page_attn(b, wide[:, 1:1 + heads], c, max_kv=5000, want_lse=False)
    assert l is None and torch.equal(o, out)
    p = q.clone()
    o, _ = S.page_attn(b, p, c, max_kv=5000, out=p)
    assert o is p and torch.equal(p, out)


def test_codes_as_float8_and_pages_between_others():
    """K and V page by page in one array, as float8, read as they are."""
    rows, heads, kv, dim, page = [100, 333], 6, 2, 64, 32
    b, cu, c, q = _case([1, 1], rows, heads, kv, dim, page, HF, seed=2)
    n = c["k"].shape[0]
    both = torch.full((n, 3, kv, page, dim), R.NAN, dtype=torch.uint8, device=DEV)
    both[:, 0], both[:, 2] = c["k"], c["v"]
    f = both.view(torch.float8_e4m3fn)
    out, lse = S.page_attn(b, q, c, max_kv=333)
    o, l = S.page_attn(b, q, dict(c, k=f[:, 0], v=f[:, 2]), max_kv=333)
    assert torch.equal(o, out) and torch.equal(l, lse)
    k, v = _normal((2, kv, dim), HF, 5), _normal((2, kv, dim), HF, 6)
    keep = both[:, 1].clone()
    fresh = dict(c, k=f[:, 0], v=f[:, 2], k_scale=c["k_scale"].clone(),
                 v_scale=c["v_scale"].clone())
    S.page_append(b, k, v, c)
    S.page_append(b, k, v, fresh)
    for x in ("k_scale", "v_scale"):
        assert torch.equal(fresh[x], c[x])
    assert torch.equal(both[:, 1], keep)
    used = c["table"][c["table"] >= 0].long()
    assert torch.equal(both[:, 2][used], c["v"][used])


@pytest.mark.parametrize("n", [1, 40])
def test_pages_past_four_gigabytes(n):
    """Pages at the ends of a pool of 4.8 GB a side, in an order that crosses it."""
    page, kv, dim, heads, m = 64, 8, 128, 16, 300
    pages = 73000
    assert pages * kv * page * dim > 1 << 32
    k, v = (torch.empty((pages, kv, page, dim), dtype=torch.uint8, device=DEV) for _ in range(2))
    ids = [pages - 1, 0, 65536, pages - 2, 70000]
    c = dict(k=k, v=v, k_scale=torch.zeros((pages, kv), device=DEV),
             v_scale=torch.zeros((pages, kv), device=DEV),
             table=torch.tensor([ids], dtype=torch.int32, device=DEV))
    kk, vv = _normal((m, kv, dim), BF, 1), _normal((m, kv, dim), BF, 2)
    b, _ = R.batch([m], [m], DEV)
    S.page_append(b, kk, vv, c)
    for x, rows in (("k", kk), ("v", vv)):
        got = R.held(c, 0, m, x)
        assert ((got - rows.double()).abs() <= rows.double().abs() * 2.0 ** -4 + 2.0 ** -9).all()
    b, cu = R.batch([n], [m], DEV)
    q = _normal((n, heads, dim), BF, 3)
    d = _derr()
    out, lse = S.page_attn(b, q, c, max_kv=m, d_err=d)
    assert int(d.item()) == 0
    ref = R.attend(q, R.held(c, 0, m, "k"), R.held(c, 0, m, "v"), dim ** -0.5,
                   m - n + torch.arange(n, device=DEV))
    R.check_attention(out, lse, ref, BF, m)


def test_empty_caches_and_batches():
    """No pages at all, tables of no width, no queries: nothing is read or written."""
    kv, dim, page, heads = 2, 64, 16, 4
    b, _ = R.batch([1, 3], [0, 0], DEV)
    q = _normal((4, heads, dim), BF, 1)
    for pages, width in ((0, 3), (0, 0), (5, 0)):
        c = dict(k=torch.zeros((pages, kv, page, dim), dtype=torch.uint8, device=DEV),
                 v=torch.zeros((pages, kv, page, dim), dtype=torch.uint8, device=DEV),
                 k_scale=torch.ones((pages, kv), device=DEV),
                 v_scale=torch.ones((pages, kv), device=DEV),
                 table=torch.zeros((2, width), dtype=torch.int32, device=DEV))
        d = _derr()
        for ws in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
            out, lse = S.page_attn(b, q, c, max_kv=0, workspace=ws, d_err=d)
            assert (out == 0).all() and (lse == -math.inf).all()
        x = _normal((4, kv, dim), BF, 2)
        S.page_append(dict(b, cu_q=torch.zeros(3, dtype=torch.int32, device=DEV)), x, x, c, d_err=d)
        assert int(d.item()) == 0
        # rows that there is no place for
        S.page_append(dict(b, kv_len=torch.tensor([1, 3], device=DEV)), x, x, c, d_err=d)
        assert int(d.item()) == S.DERR_RANGE_ROW
        assert (c["k"] == 0).all() and (c["k_scale"] == 1).all()
    e = dict(num_q=0, num_req=0, cu_q=torch.zeros(1, dtype=torch.int32, device=DEV),
             kv_len=torch.zeros(0, dtype=torch.int64, device=DEV))
    out, lse = S.page_attn(e, q[:0], c, max_kv=0)
    assert out.shape == (0, heads, dim)
    assert S.rotate(e, q[:0], S.rope_freqs(32)).shape == (0, heads, dim)


def test_rotation_and_append_in_a_graph_on_a_side_stream():
    """A decode step captured once and replayed as the lengths go on: what is read from the
    device at each replay is the batch, not what it was at the capture."""
    heads, kv, dim, page = 8, 2, 64, 16
    rows = [40, 7]
    c = R.make_cache([r + 8 for r in rows], kv, dim, page, seed=3)
    rope = dict(S.rope_freqs(64), interleaved=True)
    b, cu = R.batch([1, 1], rows, DEV)
    q, k, v = (_normal((2, h, dim), HF, i) for i, h in enumerate((heads, kv, kv)))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    twin = {x: t.clone() for x, t in c.items()}
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        qr = S.rotate(b, q, rope, stream=side)
        S.page_append(b, k, v, c, rope=rope, stream=side)
        out, lse = S.page_attn(b, qr, c, max_kv=48, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for step in range(6):
        b["kv_len"] += 1
        for i, t in enumerate((q, k, v)):
            t.copy_(_normal(t.shape, HF, 10 * step + i))
        graph.replay()
        S.page_append(b, k, v, twin, rope=rope)
        o, l = S.page_attn(b, S.rotate(b, q, rope), twin, max_kv=48)
        assert torch.equal(o, out) and torch.equal(l, lse)
    for x in c:
        assert torch.equal(c[x], twin[x])


def test_many_key_heads_and_requests():
    heads = kv = 96
    rows = [1 + (31 * i) % 75 for i in range(400)]
    b, cu, c, q = _case([1] * 400, rows, heads, kv, 64, 16, BF, seed=4)
    out, lse = S.page_attn(b, q, c, max_kv=75, sm_scale=0.02)
    for r in range(0, 400, 37):
        ref = R.attend(q[r:r + 1], R.held(c, r, rows[r], "k"), R.held(c, r, rows[r], "v"), 0.02,
                       torch.tensor([rows[r] - 1], device=DEV))
        R.check_attention(out[r:r + 1], lse[r:r + 1], ref, BF, rows[r],
                          float(c["v_scale"].max()))


@pytest.mark.parametrize("single", [True, False])
def test_requests_all_over_one_another(single):
    """Every other request has all query rows: the calls end in the time of a few batches,
    say so, and touch nothing but these rows."""
    n, heads, kv, dim, page = 2000, 4, 1, 64, 16
    r = n if single else 300
    cu = torch.tensor(([2, n] * r)[:r + 1], dtype=torch.int32, device=DEV)
    b = dict(num_q=n, num_req=r, cu_q=cu, kv_len=torch.full((r,), n, device=DEV))
    c = R.make_cache([n], kv, dim, page, seed=1)
    c["table"] = c["table"].expand(r, -1).contiguous()
    q = _normal((n, heads, dim), HF, 2)
    out = torch.full_like(q, 7.0)
    k = _normal((n, kv, dim), HF, 3)
    a, z = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    d = _derr()
    S.rotate(b, q, S.rope_freqs(64), d_err=d)
    a.record()
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        S.page_attn(b, q, c, max_kv=n, out=out, workspace=ws, d_err=d)
    S.page_append(b, k, k, c, rope=S.rope_freqs(64), d_err=d)
    z.record()
    z.synchronize()
    assert int(d.item()) == S.DERR_BAD_EXTEND
    assert (out[:2] == 7).all() and (out[2:] != 7).any(2).all()
    assert a.elapsed_time(z) < 500
