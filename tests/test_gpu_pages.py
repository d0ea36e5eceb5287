"""Rotary positions, appending to 8-bit pages and attention over them (csa2_rotate,
csa2_page_append, csa2_page_attn) against the definitions in 64 bits."""
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


def _positions(new, rows):
    return torch.cat([torch.arange(m - n, m, device=DEV) for n, m in zip(new, rows)])


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def _check_rotated(y, x, pos, rope, dtype, inverse=False):
    ref = R.rotate(x, pos, rope, inverse)
    tol = R.rotate_error(x, rope) + ref.abs() * R.HALF_STEP[dtype] * 1.001
    if dtype == HF:
        tol = tol + 2.0 ** -25
    d = (y.double() - ref).abs()
    assert (d <= tol + 1e-38).all(), float((d / (tol + 1e-38)).max())


@pytest.mark.parametrize("heads,dim,rot,inter,dtype", [
    (1, 64, 64, False, BF), (3, 128, 128, False, BF), (64, 128, 128, True, HF),
    (5, 128, 96, False, HF), (7, 64, 16, True, BF), (33, 64, 32, False, HF),
    (16, 128, 16, False, BF), (130, 128, 112, True, BF),
])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotate(heads, dim, rot, inter, dtype, inverse):
    new, rows = [1, 13, 0, 40, 7], [1, 13, 9, 500000, 3000]
    b, cu = R.batch(new, rows, DEV, lead=3, tail=2)
    x = _normal((b["num_q"], heads, dim), dtype)
    rope = S.rope_freqs(rot, scaling="ramp", factor=4, original=4096)
    rope["interleaved"] = inter
    out = torch.full_like(x, 7.0)
    d = _derr()
    S.rotate(b, x, rope, inverse=inverse, out=out, d_err=d)
    assert int(d.item()) == 0
    at = slice(cu[0], cu[-1])
    _check_rotated(out[at], x[at], _positions(new, rows), rope, dtype, inverse)
    assert torch.equal(out[at][..., rot:], x[at][..., rot:])
    assert (out[:cu[0]] == 7).all() and (out[cu[-1]:] == 7).all()


def test_rotate_given_positions():
    """Positions of their own: far, negative, repeated; no batch is read."""
    pos = torch.tensor([0, 5, 5, -3, 2 ** 31 + 7, 10 ** 6, 2 ** 24 + 1], device=DEV)
    x = _normal((7, 4, 64), BF)
    rope = dict(freq=torch.tensor([1.0, 0.5, 0.01, 2e-5, 3.0, 1e-9, 0.0, -0.25], device=DEV,
                                  dtype=torch.float64), amplitude=0.75)
    y = S.rotate(dict(num_q=7), x, rope, pos=pos)
    # 2^31 times a frequency of 3 in 64 bits is off by 2^-20 itself
    ref = R.rotate(x, pos, rope)
    tol = R.rotate_error(x, rope) * 4 + ref.abs() * R.HALF_STEP[BF] * 1.001
    assert ((y.double() - ref).abs() <= tol).all()
    back = S.rotate(dict(num_q=7), y, rope, pos=pos, inverse=True)
    # amplitude 0.75 twice, and two roundings of each of a pair's channels
    h = 8
    n = (x[..., :h].double().square() + x[..., h:16].double().square()).sqrt()
    d = (back.double() - x.double() * 0.5625)[..., :16].abs()
    assert (d <= 0.5625 * 4 * 2.0 ** -8 * torch.cat([n, n], 2)).all()


def test_rotate_in_place_and_views():
    """q and k inside one fused projection's rows, each rotated where it is."""
    n, h, kv, d = 37, 8, 2, 64
    b, _ = R.batch([n], [n + 100], DEV)
    x = _normal((n, (h + 2 * kv) * d), HF)
    keep = x.clone()
    q, k, v = (y.view(n, -1, d) for y in x.split([h * d, kv * d, kv * d], 1))
    q0, k0 = q.contiguous(), k.contiguous()
    rope = S.rope_freqs(64)
    S.rotate(b, q, rope, out=q)
    S.rotate(b, k, rope, out=k)
    assert torch.equal(q, S.rotate(b, q0, rope)) and torch.equal(k, S.rotate(b, k0, rope))
    assert torch.equal(x[:, -kv * d:], keep[:, -kv * d:])


def test_rotate_gradient_by_differences():
    """<g, R x> has the gradient R^T g: against differences of R along directions."""
    n, h, d = 9, 2, 64
    b, _ = R.batch([n], [n + 77], DEV)
    for inter in (False, True):
        rope = dict(S.rope_freqs(32, scaling="linear", factor=2), interleaved=inter,
                    amplitude=1.25)
        x, g = _normal((n, h, d), HF, 1), _normal((n, h, d), HF, 2)
        grad = S.rotate(b, g, rope, inverse=True).double()
        for seed in range(3):
            e = _normal((n, h, d), HF, 3 + seed)
            a = S.rotate(b, (x + e), rope).double()
            z = S.rotate(b, (x - e), rope).double()
            lhs = float((g.double() * (a - z)).sum() / 2)
            step = (((x + e).double() - (x - e).double()) / 2)
            rhs = float((grad * step).sum())
            # roundings of a, z and grad: half a step each of values of norm <= 1.25 |.|
            tol = 2.0 ** -11 * 1.3 * float((g.double().abs() * 1.25
                                             * (x.double().abs() + e.double().abs()) * 1.5).sum()
                                            + (grad.abs() * step.abs()).sum())
            assert abs(lhs - rhs) <= tol, (lhs, rhs, tol)


def test_rotate_bad_requests():
    b, cu = R.batch([4, 5, 3], [10, 11, 12], DEV)
    b["cu_q"] = torch.tensor([0, 4, 2, 12], dtype=torch.int32, device=DEV)   # request 1: [4, 2)
    x = _normal((12, 2, 64), BF)
    rope = S.rope_freqs(64)
    out, d = torch.full_like(x, 7.0), _derr()
    S.rotate(b, x, rope, out=out, d_err=d)
    assert int(d.item()) == S.DERR_BAD_EXTEND
    _check_rotated(out[:2], x[:2], torch.arange(6, 8, device=DEV), rope, BF)
    _check_rotated(out[4:], x[4:], torch.arange(4, 12, device=DEV), rope, BF)


# ---------------------------------------------------------------------------
# appending
# ---------------------------------------------------------------------------

def _check_append(new, rows, cu, before, after, sides, errs, page):
    """Every touched block's scale and codes, and that nothing else changed."""
    for side, x, err in zip("kv", sides, errs):
        c0, c1 = before[side].clone(), after[side]
        s0, s1 = before[side + "_scale"].clone(), after[side + "_scale"]
        for r, (n, m) in enumerate(zip(new, rows)):
            if not n:
                continue
            ids = before["table"][r].tolist()
            for p in range((m - n) // page, (m + page - 1) // page):
                lo, hi, at = max(p * page, m - n), min((p + 1) * page, m), ids[p]
                old = lo - p * page
                q = slice(cu[r] + lo - (m - n), cu[r] + hi - (m - n))
                top, off = x[q].abs().amax((0, 2)), err[q].amax((0, 2))
                for h in range(x.shape[1]):
                    allowed = {R.need(float(top[h]) + t * float(off[h])) for t in (-1, 0, 1)}
                    if old:
                        allowed = {max(a, float(s0[at, h])) for a in allowed}
                    assert float(s1[at, h]) in allowed, (side, r, p, h)
                s = s1[at].double()
                ratio = (s0[at].double() / s)[:, None, None]
                want = R.e4m3(R.values(c0[at, :, :old].contiguous()) * ratio)
                assert torch.equal(R.values(c1[at, :, :old].contiguous()), want), (side, r, p)
                got = R.values(c1[at, :, old:old + hi - lo].contiguous()).transpose(0, 1) \
                    * s[:, None]
                want = x[q]
                # half a step: 2^-4 of the value, or of the smallest normal one
                tol = torch.maximum(want.abs() * 2.0 ** -4, 2.0 ** -10 * s[:, None]) * 1.0001 \
                    + err[q]
                assert ((got - want).abs() <= tol).all(), (side, r, p)
                if not float(err.max()):
                    assert torch.equal(got, R.e4m3(want / s[:, None]) * s[:, None])
                c0[at, :, :old + hi - lo] = c1[at, :, :old + hi - lo]
                s0[at] = s1[at]
        assert torch.equal(c0, c1) and torch.equal(s0, s1)      # the rest is as it was


def _copy(c):
    both = c["k"]._base if c["k"]._base is not None else None
    if both is None:
        return {k: v.clone() for k, v in c.items()}
    b = both.clone()
    return dict({k: v.clone() for k, v in c.items()}, k=b[:, 0], v=b[:, 1])


RAGGED = ([130, 1, 0, 37, 64, 5, 200, 1], [130, 1, 40, 300, 128, 7, 519, 64])
SHAPES = [(1, 64, 16, BF), (2, 128, 64, BF), (4, 64, 32, HF), (3, 128, 128, HF),
          (8, 128, 16, BF), (2, 64, 128, BF), (5, 64, 64, HF), (1, 128, 32, HF)]


@pytest.mark.parametrize("kv,dim,page,dtype", SHAPES)
@pytest.mark.parametrize("rotated", [False, True])
def test_append_ragged(kv, dim, page, dtype, rotated):
    new, rows = RAGGED
    b, cu = R.batch(new, rows, DEV, lead=2, tail=3)
    c = R.make_cache(rows, kv, dim, page, seed=page + dim, spread=0.0, strided=kv == 2)
    before = _copy(c)
    gain = torch.exp(1.5 * _normal((b["num_q"], kv, 1), torch.float32, 5))
    k, v = ((_normal((b["num_q"], kv, dim), torch.float32, s) * gain).to(dtype) for s in (1, 2))
    rope = None
    if rotated:
        rope = dict(S.rope_freqs(dim // 2 if page == 32 else dim, scaling="base", factor=4),
                    interleaved=page == 64)
    d = _derr()
    S.page_append(b, k, v, c, rope=rope, d_err=d)
    assert int(d.item()) == 0
    at, pos = slice(cu[0], cu[-1]), _positions(new, rows)
    kk, ke = k.double(), torch.zeros_like(k, dtype=torch.float64)
    if rotated:
        kk[at], ke[at] = R.rotate(k[at], pos, rope), R.rotate_error(k[at], rope)
    _check_append(new, rows, cu, before, c, (kk, v.double()), (ke, torch.zeros_like(ke)), page)


@pytest.mark.parametrize("kv,dim,page,dtype", SHAPES)
@pytest.mark.parametrize("inter", [False, True])
def test_append_few_rows_and_one_long(kv, dim, page, dtype, inter):
    """No more rows than requests, and one with many: blocks go to warps."""
    new = [1] * 50 + [150] + [2] * 9 + [0] * 170
    rows = [1 + 7 * i for i in range(50)] + [190] + [2 + 30 * i for i in range(9)] + [3] * 170
    b, cu = R.batch(new, rows, DEV, lead=1)
    c = R.make_cache(rows, kv, dim, page, seed=page + dim, spread=0.0)
    before = _copy(c)
    gain = torch.exp(1.5 * _normal((b["num_q"], kv, 1), torch.float32, 5))
    k, v = ((_normal((b["num_q"], kv, dim), torch.float32, s) * gain).to(dtype) for s in (1, 2))
    rope = dict(S.rope_freqs(dim if page > 32 else 16, base=500.0), interleaved=inter)
    d = _derr()
    S.page_append(b, k, v, c, rope=rope, d_err=d)
    assert int(d.item()) == 0
    at, pos = slice(cu[0], cu[-1]), _positions(new, rows)
    kk, ke = k.double(), torch.zeros_like(k, dtype=torch.float64)
    kk[at], ke[at] = R.rotate(k[at], pos, rope), R.rotate_error(k[at], rope)
    _check_append(new, rows, cu, before, c, (kk, v.double()), (ke, torch.zeros_like(ke)), page)


@pytest.mark.parametrize("page", [16, 64])
def test_append_row_by_row_is_appending_at_once(page):
    """Blocks filled one row at a time, their rows of growing strength, hold what they
    would if they were filled at once, but for codes that fall below 2^-6."""
    m, kv, dim = 70, 2, 64
    one, all_ = (R.make_cache([m], kv, dim, page, seed=3) for _ in range(2))
    grow = torch.exp2(torch.arange(m, device=DEV) / 9)[:, None, None]
    k, v = ((_normal((m, kv, dim), torch.float32, s) * grow).to(BF) for s in (1, 2))
    for i in range(m):
        b, _ = R.batch([1], [i + 1], DEV)
        S.page_append(b, k[i:i + 1], v[i:i + 1], one)
    b, _ = R.batch([m], [m], DEV)
    S.page_append(b, k, v, all_)
    for s in "kv":
        assert torch.equal(one[s + "_scale"], all_[s + "_scale"])
        x, y = R.values(one[s]), R.values(all_[s])
        fine = (x == y) | (x.isnan() & y.isnan())
        # rounded more than once below the normal range: a step of 2^-9 at most
        assert ((x - y).abs()[~fine] <= 2.0 ** -9).all() and (y.abs()[~fine] <= 2.0 ** -6).all()


def test_append_values_at_the_edges():
    """Zeros, the largest value of a scale and the one above, tiny and huge rows, NaN
    and infinities."""
    page, kv, dim = 16, 1, 64
    x = torch.zeros((9, 1, dim), device=DEV)
    x[1, 0, 3] = 448
    x[2, 0, 3] = -450                    # the next bf16 above 448
    x[3, 0, 0] = 1e-30
    x[4, 0, 0] = 3e38
    x[5, 0, 1], x[5, 0, 2] = math.nan, 5
    x[6, 0, 60] = -math.inf
    x[7, 0, 0] = 7 * 2.0 ** -20
    x = x.to(BF)
    c = R.make_cache([1] * 9, kv, dim, page, seed=1)
    b, _ = R.batch([1] * 9, [1] * 9, DEV)
    d = _derr()
    S.page_append(b, x, x, c, d_err=d)
    assert int(d.item()) == S.DERR_SCALE | S.DERR_NONFINITE
    for s in "kv":
        for r, scale in enumerate([R.LOW, 1.0, 2.0, R.LOW, R.HIGH, R.LOW, R.LOW, 2.0 ** -26]):
            at = int(c["table"][r, 0])
            assert float(c[s + "_scale"][at, 0]) == scale, (s, r)
            row = R.values(c[s][at, 0, 0].contiguous())
            want = x[r, 0].double()
            want = torch.zeros_like(want) if not want.isfinite().all() else want / scale
            assert torch.equal(row, R.e4m3(want)), (s, r)


def test_append_given_positions_and_old_scales():
    """Positions of their own turn the keys, not their places; a block's older scale
    that is no power of two, out of range or NaN."""
    page, kv, dim = 16, 2, 128
    rows, new = [5, 5, 5, 5], [1, 1, 1, 1]
    c = R.make_cache(rows, kv, dim, page, seed=2)
    old = [0.37, 2.0 ** -40, math.nan, 3.0]
    for r, s in enumerate(old):
        for x in ("k_scale", "v_scale"):
            c[x][int(c["table"][r, 0])] = s
    before = _copy(c)
    b, cu = R.batch(new, rows, DEV)
    k, v = (_normal((4, kv, dim), HF, s) for s in (1, 2))
    pos = torch.tensor([10 ** 6, 0, -4, 77], device=DEV)
    rope = S.rope_freqs(128)
    d = _derr()
    S.page_append(b, k, v, c, rope=rope, pos=pos, d_err=d)
    assert int(d.item()) == S.DERR_SCALE
    for x in ("k_scale", "v_scale"):
        for r, s in ((1, R.LOW), (2, R.LOW)):
            before[x][int(c["table"][r, 0])] = s
    # (an old scale that is no power of two and stays: codes are E4M3(x / scale))
    _check_append(new, rows, cu, before, c, (R.rotate(k, pos, rope), v.double()),
                  (R.rotate_error(k, rope) + 1e-6, torch.full_like(v, 1e-6).double()), page)


def test_append_bad_batches():
    """Only the requests that are malformed are left out."""
    page, kv, dim = 16, 1, 64
    rows, new = [20, 33, 40, 17], [20, 3, 4, 17]
    c = R.make_cache(rows, kv, dim, page, seed=6, extra=40)
    fresh = _copy(c)
    k, v = (_normal((sum(new), kv, dim), BF, s) for s in (1, 2))
    ok, cu = R.batch(new, rows, DEV)
    S.page_append(ok, k, v, c)

    def check(b, bits, bad, cache=None):
        x, d = _copy(fresh) if cache is None else cache, _derr()
        S.page_append(b, k, v, x, d_err=d)
        assert int(d.item()) == bits
        for r in range(4):
            ids = fresh["table"][r, :(rows[r] + 15) // 16].long()
            for s in ("k", "v", "k_scale", "v_scale"):
                want = (fresh if r in bad else c)[s][ids]
                assert torch.equal(x[s][ids], want), (r, s)
        return x

    check(dict(ok, cu_q=torch.tensor([0, 20, 50, 27, 44], dtype=torch.int32, device=DEV)),
          S.DERR_BAD_EXTEND, (1, 2))       # [20, 50) is past num_q, [50, 27) descends
    check(dict(ok, kv_len=torch.tensor([20, 33, -1, 17], device=DEV)), S.DERR_RANGE_ROW, (2,))
    check(dict(ok, kv_len=torch.tensor([20, 1 << 40, 40, 17], device=DEV)), S.DERR_RANGE_ROW,
          (1,))
    # a page of none; the others of the request are written
    for none in (-1, 1 << 30):
        x = _copy(fresh)
        x["table"][0, 1] = none
        d = _derr()
        S.page_append(ok, k, v, x, d_err=d)
        assert int(d.item()) == S.DERR_RANGE_ROW
        a, z = int(fresh["table"][0, 0]), int(fresh["table"][0, 1])
        assert torch.equal(x["k"][a], c["k"][a]) and torch.equal(x["k"][z], fresh["k"][z])
    # more queries than rows: those in front of position 0 are left out
    x, d = _copy(fresh), _derr()
    S.page_append(dict(ok, kv_len=torch.tensor([20, 33, 40, 9], device=DEV)), k, v, x, d_err=d)
    assert int(d.item()) == S.DERR_BAD_EXTEND
    y = _copy(fresh)
    b, _ = R.batch([9], [9], DEV)
    S.page_append(b, k[-9:], v[-9:], dict(y, table=fresh["table"][3:]))
    at = int(fresh["table"][3, 0])
    assert torch.equal(x["k"][at], y["k"][at]) and torch.equal(x["v"][at], y["v"][at])


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _check_attn(out, lse, b, cu, new, rows, c, q, scale, dtype, which=None):
    for r in which if which is not None else range(len(new)):
        n, m = new[r], rows[r]
        if not n:
            continue
        at = slice(cu[r], cu[r + 1])
        k, v = R.held(c, r, m, "k"), R.held(c, r, m, "v")
        last = m - n + torch.arange(n, device=DEV)
        ids = c["table"][r, :(m + c["k"].shape[2] - 1) // c["k"].shape[2]].long()
        top = float(c["v_scale"][ids].max()) if m else 1.0
        R.check_attention(out[at], None if lse is None else lse[at],
                          R.attend(q[at], k, v, scale, last), dtype, max(1, m), top)


ATTN = [  # heads, key heads, dim, page, type
    (8, 1, 128, 64, BF), (16, 2, 64, 16, HF), (6, 2, 64, 32, BF), (4, 4, 128, 16, HF),
    (5, 1, 64, 128, BF), (32, 2, 128, 32, BF), (24, 2, 128, 128, HF), (9, 1, 64, 64, HF),
    (40, 1, 128, 16, BF), (128, 1, 64, 32, HF), (34, 2, 64, 128, BF), (128, 1, 128, 64, BF),
]


@pytest.mark.parametrize("heads,kv,dim,page,dtype", ATTN)
def test_attn_single_tokens(heads, kv, dim, page, dtype):
    rows = [1, 17, 0, 300, 128, 31, 2500, 64, 4097]
    new = [1] * len(rows)
    b, cu = R.batch(new, rows, DEV, lead=2, tail=3)
    c = R.make_cache(rows, kv, dim, page, seed=page + dim, strided=kv == 2)
    q = _normal((b["num_q"], heads, dim), dtype, 3)
    q[:cu[0]], q[cu[-1]:] = math.nan, math.nan
    scale = 0.3 * dim ** -0.5
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        out = torch.full((b["num_q"], heads, dim), 7.0, dtype=dtype, device=DEV)
        lse = torch.full((b["num_q"], heads), 7.0, device=DEV)
        d = _derr()
        S.page_attn(b, q, c, max_kv=max(rows), sm_scale=scale, out=out, lse=lse, workspace=ws,
                    d_err=d)
        assert int(d.item()) == 0
        _check_attn(out, lse, b, cu, new, rows, c, q, scale, dtype)
        for t in (out, lse):
            assert (t[:cu[0]] == 7).all() and (t[cu[-1]:] == 7).all()


@pytest.mark.parametrize("shared", [False, True])
def test_attn_single_tokens_of_any_number(shared):
    """One long cache, many short ones, several tokens to a request among idle ones: items
    that one, two and many CTAs share."""
    heads, kv, dim, page, dtype = 6, 2, 64, 32, BF
    for new, rows in (([1], [70000]), ([1] * 700, [1 + (37 * i) % 190 for i in range(700)]),
                      ([3, 0, 0, 0, 2, 0], [900, 5, 0, 40, 1, 7]),
                      ([1] * 5, [33000, 1, 20000, 64, 3]), ([1, 0, 1], [0, 0, 31])):
        b, cu = R.batch(new, rows, DEV, lead=1)
        c = R.make_cache(rows, kv, dim, page, seed=len(rows))
        q = _normal((b["num_q"], heads, dim), dtype, 3)
        out = torch.full((b["num_q"], heads, dim), 7.0, dtype=dtype, device=DEV)
        lse = torch.full((b["num_q"], heads), 7.0, device=DEV)
        d = _derr()
        ws = None if shared else torch.empty(0, dtype=torch.uint8, device=DEV)
        S.page_attn(b, q, c, max_kv=max(rows), sm_scale=0.03, out=out, lse=lse, workspace=ws,
                    d_err=d)
        assert int(d.item()) == 0
        which = range(len(new)) if len(new) < 100 else range(0, 700, 13)
        _check_attn(out, lse, b, cu, new, rows, c, q, 0.03, dtype, which=which)
        assert (out[:1] == 7).all() and (out[1:] != 7).any(2).all()


@pytest.mark.parametrize("heads,kv,dim,page,dtype", ATTN)
def test_attn_ragged(heads, kv, dim, page, dtype):
    # whole prompts, extends, one token, nothing new, nothing cached, more queries
    # than rows, tile edges
    new = [130, 1, 0, 37, 128, 5, 9, 260]
    rows = [130, 1, 40, 300, 128, 0, 4, 519]
    b, cu = R.batch(new, rows, DEV, lead=3, tail=4)
    c = R.make_cache(rows, kv, dim, page, seed=page + dim, strided=kv == 2)
    q = _normal((b["num_q"], heads, dim), dtype, 3)
    out = torch.full((b["num_q"], heads, dim), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((b["num_q"], heads), 7.0, device=DEV)
    d = _derr()
    scale = 0.3 * dim ** -0.5
    S.page_attn(b, q, c, max_kv=max(rows), sm_scale=scale, out=out, lse=lse, d_err=d)
    assert int(d.item()) == 0
    _check_attn(out, lse, b, cu, new, rows, c, q, scale, dtype)
    for t in (out, lse):
        assert (t[:cu[0]] == 7).all() and (t[cu[-1]:] == 7).all()


@pytest.mark.parametrize("n,m", [(2, 1000), (127, 127), (129, 129), (31, 4000), (700, 2100),
                                 (2049, 2049), (16, 9001), (4, 20000)])
@pytest.mark.parametrize("heads,kv,dim,page,dtype", [(8, 2, 128, 16, BF), (3, 1, 64, 64, HF),
                                                     (8, 1, 64, 32, BF), (8, 2, 128, 128, HF)])
def test_attn_one_request(n, m, heads, kv, dim, page, dtype):
    b, cu = R.batch([n], [m], DEV)
    c = R.make_cache([m], kv, dim, page, seed=n + m)
    q = _normal((n, heads, dim), dtype, 3)
    d = _derr()
    out, lse = S.page_attn(b, q, c, max_kv=m, sm_scale=0.02, d_err=d)
    assert int(d.item()) == 0
    _check_attn(out, lse, b, cu, [n], [m], c, q, 0.02, dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n", [1, 70])
def test_attn_scales_of_any_size(n, dtype):
    """Blocks whose scales lie 2^40 apart, in K and in V."""
    rows, heads, kv, dim, page = [400], 8, 1, 128, 16
    b, cu = R.batch([n], rows, DEV)
    c = R.make_cache(rows, kv, dim, page, seed=8)
    e = torch.arange(c["v_scale"].shape[0], device=DEV).float()[:, None]
    c["v_scale"] = torch.exp2(-32 + (e * 7) % 41) * 1.3
    c["k_scale"] = torch.exp2(-12 - (e * 5) % 17)
    q = _normal((n, heads, dim), dtype, 3)
    out, lse = S.page_attn(b, q.clone(), c, max_kv=400, sm_scale=1.0)
    k, v = R.held(c, 0, 400, "k"), R.held(c, 0, 400, "v")
    last = 400 - n + torch.arange(n, device=DEV)
    R.check_attention(out, lse, R.attend(q, k, v, 1.0, last), dtype, 400,
                      float(c["v_scale"].max()))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n", [1, 64])
def test_attn_growing_and_large_logits(n, dtype):
    """The running maximum moves at almost every block, up to logits of 1e3."""
    m, heads, kv, dim, page = 1500, 4, 1, 128, 32
    b, cu = R.batch([n], [m], DEV)
    c = R.make_cache([m], kv, dim, page, seed=3, spread=0.0)
    q = _normal((n, heads, dim), dtype, 4)
    grow = torch.linspace(0.1, 400, m, device=DEV)
    ids = c["table"][0].tolist()
    for i in range(m):
        x = q[0, 0].float().sign() * grow[i]
        c["k"][ids[i // page], 0, i % page] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    c["k_scale"][:] = 0.1
    out, lse = S.page_attn(b, q, c, max_kv=m)
    _check_attn(out, lse, b, cu, [n], [m], c, q, dim ** -0.5, dtype)


@pytest.mark.parametrize("scale", [1e-20, 1.0, 1e20])
def test_attn_queries_of_any_size(scale):
    """bf16 queries far outside f16's range."""
    rows, heads, kv, dim = [200, 33], 8, 2, 64
    b, cu = R.batch([1, 1], rows, DEV)
    c = R.make_cache(rows, kv, dim, 32, seed=5, spread=0.0)
    q = (_normal((2, heads, dim), torch.float32, 3) * scale).to(BF)
    q[0, 1] = 0
    out, lse = S.page_attn(b, q, c, max_kv=200, sm_scale=0.05 / scale)
    _check_attn(out, lse, b, cu, [1, 1], rows, c, q, 0.05 / scale, BF)


@pytest.mark.parametrize("n", [1, 50])
def test_attn_bad_pages_and_requests(n):
    """Rows of a page that is none are not seen; requests of more rows than the table
    has room for have none; scales out of range are flagged."""
    rows, heads, kv, dim, page = [100, 200, 90], 4, 2, 64, 16
    new = [n] * 3
    b, cu = R.batch(new, rows, DEV)
    c = R.make_cache(rows, kv, dim, page, seed=9, spread=0.0)
    q = _normal((3 * n, heads, dim), BF, 3)
    for none in (-1, 1 << 30):
        x = dict(c, table=c["table"].clone())
        x["table"][1, 3] = none
        d = _derr()
        out, lse = S.page_attn(b, q, x, max_kv=200, sm_scale=0.02, d_err=d)
        assert int(d.item()) == S.DERR_RANGE_ROW
        _check_attn(out, lse, b, cu, new, rows, c, q, 0.02, BF, which=(0, 2))
        k, v = R.held(c, 1, 200, "k"), R.held(c, 1, 200, "v")
        see = torch.cat([torch.arange(48), torch.arange(64, 200)]).to(DEV)
        last = (see[None, :] <= 200 - n + torch.arange(n, device=DEV)[:, None]).sum(1) - 1
        ref = R.attend(q[cu[1]:cu[2]], k[see], v[see], 0.02, last)
        R.check_attention(out[cu[1]:cu[2]], lse[cu[1]:cu[2]], ref, BF, 200)
    for bad in (1 << 40, -5):
        d = _derr()
        out, lse = S.page_attn(dict(b, kv_len=torch.tensor([100, bad, 90], device=DEV)), q, c,
                               max_kv=200, sm_scale=0.02, d_err=d)
        assert int(d.item()) == S.DERR_RANGE_ROW
        _check_attn(out, lse, b, cu, new, rows, c, q, 0.02, BF, which=(0, 2))
        assert (out[cu[1]:cu[2]] == 0).all() and (lse[cu[1]:cu[2]] == -math.inf).all()
    x = dict(c, v_scale=c["v_scale"].clone())
    x["v_scale"][int(c["table"][0, 1])] = 2.0 ** -50
    d = _derr()
    out, lse = S.page_attn(b, q, x, max_kv=200, sm_scale=0.02, d_err=d)
    assert int(d.item()) == S.DERR_SCALE
    x["v_scale"][int(c["table"][0, 1])] = R.LOW
    _check_attn(out, lse, b, cu, new, rows, x, q, 0.02, BF)


def test_attn_malformed_batch():
    rows, new, heads, kv, dim = [50, 60, 70], [4, 5, 3], 4, 2, 64
    b, cu = R.batch(new, rows, DEV)
    c = R.make_cache(rows, kv, dim, 16, seed=9, spread=0.0)
    q = _normal((12, heads, dim), BF, 3)
    out = torch.full_like(q, 7.0)
    d = _derr()
    bad = dict(b, cu_q=torch.tensor([0, 4, 20, 12], dtype=torch.int32, device=DEV))
    S.page_attn(bad, q, c, max_kv=70, sm_scale=0.02, out=out, d_err=d)
    assert int(d.item()) == S.DERR_BAD_EXTEND
    _check_attn(out, None, b, cu, new, rows, c, q, 0.02, BF, which=(0,))
    assert (out[4:] == 7).all()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,page,dim", [(BF, 64, 128), (HF, 16, 64)])
def test_serving_steps(dtype, page, dim):
    """Prompts, an extend and decode steps of a batch: queries rotated, keys rotated and
    appended, attention over the pages; against rows that are rotated and held the
    same way, in 64 bits."""
    heads, kv = 8, 2
    lens = [100, 1, 37]
    total = [n + 25 for n in lens]
    c = R.make_cache(total, kv, dim, page, seed=4)
    for s in "kv":
        c[s].fill_(R.NAN)
    rope = S.rope_freqs(dim, scaling="ramp", factor=4, original=64)
    done = [0, 0, 0]
    for step, new in enumerate([lens, [20, 0, 3], [1, 1, 1], [1, 1, 1], [1, 1, 1]]):
        done = [a + n for a, n in zip(done, new)]
        b, cu = R.batch(new, done, DEV)
        nq = b["num_q"]
        q, k, v = (_normal((nq, h, dim), dtype, 10 * step + i)
                   for i, h in enumerate((heads, kv, kv)))
        d = _derr()
        qr = S.rotate(b, q, rope, d_err=d)
        S.page_append(b, k, v, c, rope=rope, d_err=d)
        out, lse = S.page_attn(b, qr, c, max_kv=max(done), d_err=d)
        assert int(d.item()) == 0
        _check_attn(out, lse, b, cu, new, done, c, qr, dim ** -0.5, dtype)
        # the last row of each request as it was meant to be held
        for r, n in enumerate(new):
            if n:
                i = cu[r + 1] - 1
                pos = torch.tensor([done[r] - 1], device=DEV)
                want = R.rotate(k[i:i + 1], pos, rope)[0]
                got = R.held(c, r, done[r], "k")[-1]
                assert ((got - want).abs() <= want.abs().amax() * 2.0 ** -4).all()
