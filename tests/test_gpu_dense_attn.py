"""Prompt attention and shared-prefix attention (csa2_prompt_attn,
csa2_prefix_attn) against the definition in 64 bits."""
import math

import pytest
import torch

import sparse_attention_prefill_gb300 as S
from tests import dense_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, HF = torch.bfloat16, torch.float16


def _derr():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _inputs(new, rows, heads, kv, dim, dtype, seed=0, lead=0, tail=0, extra=()):
    """Requests, then `extra` runs (prefixes) in one pool whose other rows are
    NaN; q rows of no request are NaN too."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    start, pool = R.starts(list(rows) + list(extra))
    b, cu = R.batch(new, rows, start[:len(rows)], DEV, lead, tail)
    q = torch.full((b["num_q"], heads, dim), math.nan, dtype=dtype, device=DEV)
    n = cu[-1] - cu[0]
    q[cu[0]:cu[-1]] = torch.randn((n, heads, dim), generator=g, device=DEV).to(dtype)
    k, v = (torch.full((pool, kv, dim), math.nan, dtype=dtype, device=DEV) for _ in range(2))
    for s, m in zip(start, list(rows) + list(extra)):
        k[s:s + m] = torch.randn((m, kv, dim), generator=g, device=DEV).to(dtype)
        v[s:s + m] = torch.randn((m, kv, dim), generator=g, device=DEV).to(dtype)
    return b, cu, start, q, k, v


def _ref(q, k, v, cu, start, new, rows, r, scale, prefix=None):
    kk, vv = k[start[r]:start[r] + rows[r]], v[start[r]:start[r] + rows[r]]
    off = 0
    if prefix:
        p, n = prefix
        kk, vv = torch.cat([k[p:p + n], kk]), torch.cat([v[p:p + n], vv])
        off = n
    last = off + rows[r] - new[r] + torch.arange(new[r], device=DEV)
    if prefix:
        last = torch.clamp(last, min=off - 1)
    return R.attend(q[cu[r]:cu[r + 1]], kk, vv, scale, last), max(1, kk.shape[0])


SHAPES = [  # heads, key heads, dim, type
    (8, 1, 128, BF), (64, 8, 128, BF), (6, 2, 64, HF), (4, 4, 128, HF), (5, 1, 64, BF),
    (48, 3, 64, BF), (128, 1, 128, BF), (12, 4, 128, HF),
]


@pytest.mark.parametrize("heads,kv,dim,dtype", SHAPES)
def test_prompt_ragged(heads, kv, dim, dtype):
    # whole prompts, extends, one token, nothing new, nothing cached, more
    # queries than rows, tile edges
    new = [130, 1, 0, 37, 128, 5, 9, 260]
    rows = [130, 1, 40, 300, 128, 0, 4, 519]
    b, cu, start, q, k, v = _inputs(new, rows, heads, kv, dim, dtype, lead=3, tail=4)
    out = torch.full((b["num_q"], heads, dim), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((b["num_q"], heads), 7.0, device=DEV)
    d = _derr()
    S.prompt_attn(b, q, k, v, out=out, lse=lse, d_err=d)
    assert int(d.item()) == 0
    for r in range(len(new)):
        if new[r]:
            ref, n = _ref(q, k, v, cu, start, new, rows, r, dim ** -0.5)
            R.check_attention(out[cu[r]:cu[r + 1]], lse[cu[r]:cu[r + 1]], ref, dtype, n)
    # rows of no request keep their values
    for t in (out, lse):
        assert (t[:cu[0]] == 7).all() and (t[cu[-1]:] == 7).all()


@pytest.mark.parametrize("n,m", [(1, 1), (1, 127), (1, 129), (2, 1000), (127, 127), (129, 129),
                                 (31, 4000), (700, 2100), (2049, 2049)])
@pytest.mark.parametrize("heads,kv,dim,dtype", [(8, 2, 128, BF), (3, 1, 64, HF)])
def test_prompt_one_request(n, m, heads, kv, dim, dtype):
    b, cu, start, q, k, v = _inputs([n], [m], heads, kv, dim, dtype, seed=n + m)
    out, lse = S.prompt_attn(b, q, k, v, sm_scale=0.2)
    ref, keys = _ref(q, k, v, cu, start, [n], [m], 0, 0.2)
    R.check_attention(out, lse, ref, dtype, keys)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_prompt_growing_and_large_logits(dtype):
    """The running maximum moves at almost every tile, up to logits of 1e3."""
    b, cu, start, q, k, v = _inputs([64], [1500], 4, 1, 128, dtype, seed=3)
    grow = torch.linspace(0.01, 40, k.shape[0], device=DEV)[:, None, None]
    k = torch.where(k.isnan(), k, q[:1, :1].float().sign() * grow).to(dtype)
    out, lse = S.prompt_attn(b, q, k, v)
    ref, keys = _ref(q, k, v, cu, start, [64], [1500], 0, 128 ** -0.5)
    R.check_attention(out, lse, ref, dtype, keys)


def test_prompt_many_small_weights_f16():
    """Thousands of keys far below one: their share is not lost in f16."""
    m = 6000
    b, cu, start, q, k, v = _inputs([3], [m], 2, 1, 64, HF, seed=4)
    q[:] = 0
    q[:, :, 0] = 1
    k[start[0]:start[0] + m] = 0
    k[start[0], :, 0] = 13.0
    v[start[0]:start[0] + m] = 1
    v[start[0]] = -1
    out, lse = S.prompt_attn(b, q, k, v, sm_scale=1.0)
    ref, keys = _ref(q, k, v, cu, start, [3], [m], 0, 1.0)
    R.check_attention(out, lse, ref, HF, keys)


def test_strided_rows():
    """q, k and v inside one fused projection's rows, and an interleaved cache."""
    n, h, kv, d = 150, 8, 2, 64
    x = torch.randn((n, (h + 2 * kv) * d), device=DEV).to(BF)
    q, k, v = (y.view(n, -1, d) for y in x.split([h * d, kv * d, kv * d], 1))
    b, cu = R.batch([n], [n], [0], DEV)
    out, lse = S.prompt_attn(b, q, k, v)
    o2, l2 = S.prompt_attn(b, q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    c = torch.randn((n, 2, kv, d), device=DEV).to(BF)
    out, lse = S.prompt_attn(b, q, c[:, 0], c[:, 1])
    o2, l2 = S.prompt_attn(b, q, c[:, 0].contiguous(), c[:, 1].contiguous())
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("call", ["prompt", "prefix"])
def test_bad_requests_are_flagged(call):
    new, rows = [20, 30, 25], [20, 60, 25]
    b, cu, start, q, k, v = _inputs(new, rows, 4, 2, 64, BF)
    good, _ = S.prompt_attn(b, q, k, v)

    def run(b, d):
        if call == "prompt":
            return S.prompt_attn(b, q, k, v, d_err=d)
        return S.prefix_attn(b, None, q, k, v, 60, d_err=d)

    for bad in (dict(kv_start=b["kv_start"] + torch.tensor([0, 10 ** 9, 0], device=DEV)),
                dict(kv_start=b["kv_start"] - torch.tensor([0, 50, 0], device=DEV)),
                dict(kv_len=b["kv_len"] * torch.tensor([1, -1, 1], device=DEV))):
        d = _derr()
        out, lse = run(dict(b, **bad), d)
        assert int(d.item()) == S.DERR_RANGE_ROW
        assert (out[20:50] == 0).all() and (lse[20:50] == -math.inf).all()
        assert torch.allclose(out[:20].float(), good[:20].float(), atol=2 ** -6)
        assert torch.allclose(out[50:].float(), good[50:].float(), atol=2 ** -6)
    for cu_bad in ([0, 20, 10, 75], [0, 20, 50, 76], [0, 20, 10 ** 9, 75], [-4, 20, 50, 75]):
        d = _derr()
        run(dict(b, cu_q=torch.tensor(cu_bad, dtype=torch.int32, device=DEV)), d)
        assert int(d.item()) & S.DERR_BAD_EXTEND


@pytest.mark.parametrize("heads,kv,dim,dtype", SHAPES)
def test_prefix_groups(heads, kv, dim, dtype):
    """Two groups, a request in none, an empty prefix, several tokens a request."""
    new = [1, 3, 1, 0, 40, 1, 2]
    rows = [17, 3, 300, 9, 140, 1, 0]
    pre = [1000, 0, 333]
    cug = [0, 2, 4, 6]                      # the last request is in no group
    b, cu, start, q, k, v = _inputs(new, rows, heads, kv, dim, dtype, seed=5, lead=2, tail=3,
                                    extra=pre)
    gr = dict(num_groups=3, cu_group=torch.tensor(cug, dtype=torch.int32, device=DEV),
              prefix_start=torch.tensor(start[len(new):], dtype=torch.int64, device=DEV),
              prefix_len=torch.tensor(pre, dtype=torch.int64, device=DEV), max_prefix=1000)
    out = torch.full((b["num_q"], heads, dim), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((b["num_q"], heads), 7.0, device=DEV)
    d = _derr()
    need = S.csa2_prefix_attn_workspace(b["num_q"], len(new), 3, heads, kv, dim, 1000, 300)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)       # NaNs
    S.prefix_attn(b, gr, q, k, v, 300, out=out, lse=lse, workspace=ws, d_err=d)
    assert int(d.item()) == 0
    for r in range(len(new)):
        if not new[r]:
            continue
        g = next((i for i in range(3) if cug[i] <= r < cug[i + 1]), None)
        p = None if g is None else (start[len(new) + g], pre[g])
        ref, n = _ref(q, k, v, cu, start, new, rows, r, dim ** -0.5, p)
        R.check_attention(out[cu[r]:cu[r + 1]], lse[cu[r]:cu[r + 1]], ref, dtype, n)
    for t in (out, lse):
        assert (t[:cu[0]] == 7).all() and (t[cu[-1]:] == 7).all()


@pytest.mark.parametrize("reqs,heads,kv,dim,prefix,hint", [
    (1, 8, 1, 128, 1, 1), (1, 8, 8, 64, 20000, 20000), (40, 16, 2, 128, 3001, 3001),
    (300, 8, 8, 64, 130, 130), (9, 64, 8, 128, 5000, 10), (33, 5, 1, 64, 700, 100000),
    (12, 16, 1, 128, 900, 900), (20, 24, 2, 64, 900, 900), (7, 34, 2, 128, 300, 300),
    (6, 128, 1, 64, 500, 500)])
def test_prefix_decode(reqs, heads, kv, dim, prefix, hint):
    """Decode batches of one group; max_prefix and max_kv only steer the splits."""
    rows = [1 + (37 * i) % 400 for i in range(reqs)]
    b, cu, start, q, k, v = _inputs([1] * reqs, rows, heads, kv, dim, BF, seed=reqs,
                                    extra=[prefix])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)    # noqa: E731
    gr = dict(num_groups=1, cu_group=i32([0, reqs]), max_prefix=hint,
              prefix_start=torch.tensor(start[-1:], device=DEV),
              prefix_len=torch.tensor([prefix], device=DEV))
    out, lse = S.prefix_attn(b, gr, q, k, v, hint)
    for r in range(0, reqs, max(1, reqs // 9)):
        ref, n = _ref(q, k, v, cu, start, [1] * reqs, rows, r, dim ** -0.5, (start[-1], prefix))
        R.check_attention(out[r:r + 1], lse[r:r + 1], ref, BF, n)


@pytest.mark.parametrize("reqs,m", [(1, 30000), (3, 129), (70, 2000)])
def test_decode_without_groups(reqs, m):
    rows = [max(1, m - 11 * i) for i in range(reqs)]
    b, cu, start, q, k, v = _inputs([1] * reqs, rows, 16, 4, 128, HF, seed=m)
    out, lse = S.prefix_attn(b, None, q, k, v, m)
    for r in range(0, reqs, max(1, reqs // 7)):
        ref, n = _ref(q, k, v, cu, start, [1] * reqs, rows, r, 128 ** -0.5)
        R.check_attention(out[r:r + 1], lse[r:r + 1], ref, HF, n)


@pytest.mark.parametrize("heads,kv", [(8, 1), (12, 1), (40, 2)])
def test_decode_strided_cache_and_uneven_tokens(heads, kv):
    """An interleaved cache, requests of no, one, two and three tokens (not a
    token each, though as many as requests), rows in front and behind."""
    new, rows = [2, 0, 1, 0, 3, 0], [2, 40, 300, 7, 65, 1]
    b, cu, start, q, k, v = _inputs(new, rows, heads, kv, 128, BF, seed=heads, lead=0, tail=0)
    c = torch.stack([k, v], 1)
    for call in (lambda k, v: S.prompt_attn(b, q, k, v),
                 lambda k, v: S.prefix_attn(b, None, q, k, v, 300)):
        out, lse = call(c[:, 0], c[:, 1])
        for r in range(len(new)):
            if new[r]:
                ref, n = _ref(q, k, v, cu, start, new, rows, r, 128 ** -0.5)
                R.check_attention(out[cu[r]:cu[r + 1]], lse[cu[r]:cu[r + 1]], ref, BF, n)


@pytest.mark.parametrize("n", [1, 3, 300])
def test_rows_past_two_to_the_32_bytes(n):
    """Requests at the end of pools whose byte offsets pass 32 bits."""
    kv, dim, m, pool = 8, 128, 333, (1 << 21) + 5000
    k = torch.empty((pool, kv, dim), dtype=BF, device=DEV)
    v = torch.empty((pool, kv, dim), dtype=BF, device=DEV)
    start = pool - m
    k[start:] = torch.randn((m, kv, dim), device=DEV).to(BF)
    v[start:] = torch.randn((m, kv, dim), device=DEV).to(BF)
    q = torch.randn((n, 16, dim), device=DEV).to(BF)
    b, cu = R.batch([n], [m], [start], DEV)
    ref, keys = _ref(q, k, v, cu, [start], [n], [m], 0, dim ** -0.5)
    for out, lse in (S.prompt_attn(b, q, k, v), S.prefix_attn(b, None, q, k, v, m)):
        R.check_attention(out, lse, ref, BF, keys)
    mass = torch.zeros((kv, pool), device=DEV)
    S.attn_mass(b, q, k, lse, m, mass=mass)
    w, tol = R.mass(q, k[start:], lse, dim ** -0.5, m - n + torch.arange(n, device=DEV))
    assert ((mass[:, start:].double() - w).abs() <= tol + w * 2.0 ** -22 + 1e-30).all()
    assert (mass[:, :start] == 0).all()


def test_decode_bad_requests_are_flagged():
    rows = [20, 60, 25]
    b, cu, start, q, k, v = _inputs([1, 1, 1], rows, 8, 2, 128, BF)
    good, _ = S.prompt_attn(b, q, k, v)
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device=DEV)    # noqa: E731
    for bad in (dict(kv_start=b["kv_start"] + i64([0, 10 ** 9, 0])),
                dict(kv_len=b["kv_len"] * i64([1, -1, 1]))):
        for call in (lambda b, d: S.prompt_attn(b, q, k, v, d_err=d),
                     lambda b, d: S.prefix_attn(b, None, q, k, v, 60, d_err=d)):
            d = _derr()
            out, lse = call(dict(b, **bad), d)
            assert int(d.item()) == S.DERR_RANGE_ROW
            assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
            assert torch.allclose(out[::2].float(), good[::2].float(), atol=2 ** -6)
    for cu_bad in ([0, 1, 10 ** 9, 3], [0, 2, 1, 3], [-1, 1, 2, 3], [0, 1, 2, 4],
                   [0, -5, 2, 3]):
        d = _derr()
        S.prompt_attn(dict(b, cu_q=torch.tensor(cu_bad, dtype=torch.int32, device=DEV)), q, k, v,
                      d_err=d)
        assert int(d.item()) == S.DERR_BAD_EXTEND, cu_bad


def test_two_calls_at_once_with_a_workspace_each():
    """Two shared-prefix calls on two streams, replayed from one graph."""
    args = []
    for seed in (1, 2):
        rows = [100 + 50 * seed] * 20
        b, cu, start, q, k, v = _inputs([1] * 20, rows, 16, 2, 128, BF, seed=seed, extra=[2000])
        gr = dict(num_groups=1, cu_group=torch.tensor([0, 20], dtype=torch.int32, device=DEV),
                  prefix_start=torch.tensor(start[-1:], device=DEV),
                  prefix_len=torch.tensor([2000], device=DEV), max_prefix=2000)
        need = S.csa2_prefix_attn_workspace(20, 20, 1, 16, 2, 128, 2000, 200)
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        args.append((b, gr, q, k, v, 200, ws))
    want = [S.prefix_attn(*a[:6], workspace=a[6]) for a in args]
    got = [tuple(torch.empty_like(x) for x in w) for w in want]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        S.prefix_attn(*args[0][:6], workspace=args[0][6], out=got[0][0], lse=got[0][1])
        S.prefix_attn(*args[1][:6], workspace=args[1][6], out=got[1][0], lse=got[1][1],
                      stream=side)
        main.wait_stream(side)
    for _ in range(3):
        for g in got:
            g[0].zero_(), g[1].zero_()
        graph.replay()
        for w, g in zip(want, got):
            assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


@pytest.mark.parametrize("grouped", [True, False])
def test_calls_in_a_row_keep_the_stream_order(grouped):
    """The call's kernels overlap one another, but nothing in front of the call
    or behind it: inputs written just before and just after, one workspace."""
    reqs, heads, kv, dim, prefix = 40, 32, 4, 128, 2500
    rows = [(37 * i) % 400 + 1 for i in range(reqs)]
    b, _, start, q, k, v = _inputs([1] * reqs, rows, heads, kv, dim, BF, extra=[prefix])
    groups = dict(num_groups=1, max_prefix=prefix,
                  cu_group=torch.tensor([0, reqs - 3], dtype=torch.int32, device=DEV),
                  prefix_start=torch.tensor([start[-1]], dtype=torch.int64, device=DEV),
                  prefix_len=torch.tensor([prefix], dtype=torch.int64, device=DEV))
    g = groups if grouped else None
    g0 = torch.Generator(device=DEV).manual_seed(5)
    qs = [torch.randn(q.shape, generator=g0, device=DEV).to(BF) for _ in range(12)]
    ks = [k + i for i in range(3)]
    want = []
    for i, x in enumerate(qs):
        want.append(S.prefix_attn(b, g, x, ks[i % 3], v, max(rows)))
        torch.cuda.synchronize()
    n = S.csa2_prefix_attn_workspace(reqs, reqs, 1 if grouped else 0, heads, kv, dim,
                                     prefix if grouped else 0, max(rows))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    qb, kb = torch.empty_like(q), torch.empty_like(k)
    got = []
    for i, x in enumerate(qs):
        qb.copy_(x)
        kb.copy_(ks[i % 3])
        S.prefix_attn(b, g, qb, kb, v, max(rows), out=out, lse=lse, workspace=ws)
        qb.fill_(math.nan)
        kb.fill_(math.nan)
        got.append((out.clone(), lse.clone()))
        out.fill_(9.0)
        ws.fill_(255)
    for (o, l), (wo, wl) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)


def test_prefix_bad_groups_are_flagged():
    new, rows = [1, 1, 1], [30, 40, 50]
    b, cu, start, q, k, v = _inputs(new, rows, 4, 2, 64, BF, extra=[200])
    own, _ = S.prefix_attn(b, None, q, k, v, 50)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)    # noqa: E731
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device=DEV)    # noqa: E731
    for cug, ps, pl, bit in (([0, 9], start[-1], 200, S.DERR_BAD_EXTEND),
                             ([-1, 3], start[-1], 200, S.DERR_BAD_EXTEND),
                             ([0, 3], 10 ** 8, 200, S.DERR_RANGE_ROW),
                             ([0, 3], start[-1], 10 ** 8, S.DERR_RANGE_ROW)):
        d = _derr()
        gr = dict(num_groups=1, cu_group=i32(cug), prefix_start=i64([ps]), prefix_len=i64([pl]),
                  max_prefix=200)
        out, _ = S.prefix_attn(b, gr, q, k, v, 50, d_err=d)
        assert int(d.item()) == bit
        assert torch.allclose(out.float(), own.float(), atol=2 ** -6)


def test_same_bits_and_streams_and_graph():
    """The same call gives the same bits, on another stream and replayed."""
    new, rows = [1, 30, 4], [900, 30, 500]
    b, cu, start, q, k, v = _inputs(new, rows, 8, 2, 128, BF, seed=8, extra=[800])
    gr = dict(num_groups=1, cu_group=torch.tensor([0, 3], dtype=torch.int32, device=DEV),
              prefix_start=torch.tensor(start[-1:], device=DEV),
              prefix_len=torch.tensor([800], device=DEV), max_prefix=800)
    o1, l1 = S.prompt_attn(b, q, k, v)
    o2, l2 = S.prefix_attn(b, gr, q, k, v, 900)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p1, m1 = S.prompt_attn(b, q, k, v, stream=side)
    p2, m2 = S.prefix_attn(b, gr, q, k, v, 900, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o1, p1) and torch.equal(o2, p2)
    assert torch.equal(l1, m1) and torch.equal(l2, m2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g1, _ = S.prompt_attn(b, q, k, v)
        g2, _ = S.prefix_attn(b, gr, q, k, v, 900)
    q.copy_(-q)
    graph.replay()
    o1, _ = S.prompt_attn(b, q, k, v)
    o2, _ = S.prefix_attn(b, gr, q, k, v, 900)
    assert torch.equal(o1, g1) and torch.equal(o2, g2)


def test_empty_batches():
    b, _ = R.batch([], [], [], DEV)
    z = torch.empty((0, 4, 64), dtype=BF, device=DEV)
    out, lse = S.prompt_attn(b, z, z, z)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    b, _ = R.batch([2], [0], [0], DEV)                  # an empty pool
    q = torch.randn((2, 4, 64), device=DEV).to(BF)
    for out, lse in (S.prompt_attn(b, q, z, z), S.prefix_attn(b, None, q, z, z, 0)):
        assert (out == 0).all() and (lse == -math.inf).all()


def test_waits_run_out_then_recover():
    b, cu, start, q, k, v = _inputs([400], [400], 8, 2, 128, BF, seed=9)
    want, _ = S.prompt_attn(b, q, k, v)
    S.set_wait_limit_ns(1)
    try:
        d = _derr()
        for _ in range(3):
            S.prompt_attn(b, q, k, v, d_err=d)
            S.prefix_attn(b, None, q, k, v, 400, d_err=d)
        torch.cuda.synchronize()
    finally:
        S.set_wait_limit_ns(0)
    assert int(d.item()) & S.DERR_TIMEOUT
    d = _derr()
    out, _ = S.prompt_attn(b, q, k, v, d_err=d)
    assert int(d.item()) == 0 and torch.equal(out, want)
