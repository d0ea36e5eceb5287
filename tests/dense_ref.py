"""Definitions of the dense-cache operators in 64 bits, row by row, and the
error bounds the kernels are held to."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def starts(lens, gap=5):
    """First rows of runs in a pool with unused rows around them, and its size."""
    at, out = gap, []
    for n in lens:
        out.append(at)
        at += n + gap
    return out, at


def batch(new, rows, start, device, lead=0, tail=0):
    """Packed dict; `lead` query rows in front of the first request and `tail`
    behind the last belong to none."""
    cu = [lead]
    for n in new:
        cu.append(cu[-1] + n)
    return dict(num_q=cu[-1] + tail, num_req=len(new),
                cu_q=torch.tensor(cu, dtype=torch.int32, device=device),
                kv_start=torch.tensor(start, dtype=torch.int64, device=device),
                kv_len=torch.tensor(rows, dtype=torch.int64, device=device)), cu


def attend(q, keys, values, scale, last):
    """One request: q [n, H, D] over keys, values [m, Hkv, D] in float64; query
    i sees the keys <= last[i].  Returns out, lse, sum of |weights * values|
    and the largest sum_d |q k| * scale per row."""
    n, h, d = q.shape
    kv = keys.shape[1]
    q, keys, values = q.double(), keys.double(), values.double()
    k = keys.repeat_interleave(h // kv, 1)
    v = values.repeat_interleave(h // kv, 1)
    see = (torch.arange(keys.shape[0], device=q.device)[None, :] <= last[:, None])[:, None, :]
    x = torch.einsum("nhd,mhd->nhm", q, k) * scale
    mag = (torch.einsum("nhd,mhd->nhm", q.abs(), k.abs()) * scale * see).amax(2) \
        if keys.shape[0] else torch.zeros(n, h, device=q.device, dtype=torch.float64)
    x = torch.where(see, x, -math.inf)
    if not keys.shape[0]:
        z = torch.zeros_like(q)
        return z, torch.full((n, h), -math.inf, device=q.device, dtype=torch.float64), z, mag
    lse = torch.logsumexp(x, 2)
    w = torch.where(see, torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[..., None]), 0.0)
    v = torch.where(see.any(0).any(0)[:, None, None], v, 0.0)
    return (torch.einsum("nhm,mhd->nhd", w, v), lse, torch.einsum("nhm,mhd->nhd", w, v.abs()),
            mag)


def check_attention(out, lse, ref, dtype, n_keys):
    """|error| bounds.  Weights are rounded to the inputs' type (half a step
    each, so at most u * sum w|v|) and the output once more (u * |out|).  A
    logit of D <= 128 fp32 terms is off by at most 2^-17 of sum |q k| (128
    additions of 2^-24), which moves every weight by that much relatively, and
    the sum under it too; sums over the keys add n * 2^-24, the exponential
    2^-22, and an f16 weight below its normal range 2^-32."""
    ro, rl, ra, mag = ref
    u = HALF_STEP[dtype]
    dl = 2.0 ** -17 * mag + 2.0 ** -22
    tol = u * (ra + ro.abs()) * 1.01 + ra * (2 * dl + n_keys * 2.0 ** -23)[..., None] \
        + n_keys * 2.0 ** -32 + 1e-30
    if dtype == torch.float16:
        tol = tol + 2.0 ** -24            # outputs below f16's normal range
    bad = (out.double() - ro).abs() > tol
    assert not bad.any(), (float((out.double() - ro).abs().max()), int(bad.sum()))
    if lse is not None:
        inf = rl.isinf()
        assert (lse.double()[inf] == -math.inf).all()
        d = (lse.double() - rl).abs()[~inf]
        t = (dl + n_keys * 2.0 ** -24 + rl.abs() * 2.0 ** -22)[~inf]
        assert (d <= t).all(), (float(d.max()), float(t.min()))


def mass(q, keys, lse, scale, last):
    """One request: float64 weights [Hkv, m] and the bound on their error."""
    n, h, d = q.shape
    kv = keys.shape[1]
    q, keys, lse = q.double(), keys.double(), lse.double()
    k = keys.repeat_interleave(h // kv, 1)
    see = (torch.arange(keys.shape[0], device=q.device)[None, :] <= last[:, None])[:, None, :]
    x = torch.einsum("nhd,mhd->nhm", q, k) * scale
    mag = torch.einsum("nhd,mhd->nhm", q.abs(), k.abs()) * scale
    w = torch.where(see & (lse > -math.inf)[..., None], torch.exp(x - lse[..., None]), 0.0)
    # the logit's 2^-17, the roundings of c s and lse' (2^-24 each of values
    # near |lse|), the exponential's 2^-22, the additions
    rel = 2.0 ** -17 * mag + 2.0 ** -22 * (1 + torch.where(lse.isinf(), 0.0, lse).abs())[..., None] \
        + n * h // kv * 2.0 ** -24
    fold = lambda y: y.sum(0).reshape(kv, h // kv, -1).sum(1)   # noqa: E731
    return fold(w), fold(w * rel)
