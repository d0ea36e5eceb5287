"""Definitions of the operators on 8-bit pages in 64 bits, and the error bounds the
kernels are held to."""
import math

import torch

# torch.finfo(t).eps / 2: bf16 has 8 significant bits, a step of at most 2^-7 of the
# value, so rounding is off by 2^-8 of it
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LOW, HIGH = 2.0 ** -32, 2.0 ** 32
NAN = 0x7f


def batch(new, rows, device, lead=0, tail=0):
    """Packed dict; `lead` query rows in front of the first request and `tail` behind
    the last belong to none."""
    cu = [lead]
    for n in new:
        cu.append(cu[-1] + n)
    return dict(num_q=cu[-1] + tail, num_req=len(new),
                cu_q=torch.tensor(cu, dtype=torch.int32, device=device),
                kv_len=torch.tensor(rows, dtype=torch.int64, device=device)), cu


def rotation(pos, rope):
    """Complex factors [n, rot / 2] in 64 bits."""
    f = rope["freq"].double()
    a = pos.double()[:, None] * f[None, :]
    return torch.polar(torch.full_like(a, float(rope.get("amplitude", 1.0))), a)


def rotate(x, pos, rope, inverse=False):
    x = x.double().clone()
    z = rotation(pos, rope)[:, None, :]
    if inverse:
        z = z.conj()
    h = rope["freq"].numel()
    if rope.get("interleaved"):
        a, b = x[..., 0:2 * h:2].clone(), x[..., 1:2 * h:2].clone()
    else:
        a, b = x[..., :h].clone(), x[..., h:2 * h].clone()
    u, w = a * z.real - b * z.imag, a * z.imag + b * z.real
    if rope.get("interleaved"):
        x[..., 0:2 * h:2], x[..., 1:2 * h:2] = u, w
    else:
        x[..., :h], x[..., h:2 * h] = u, w
    return x


def rotate_error(x, rope):
    """Bound on an fp32 rotation's error, before the result is rounded: per pair
    amplitude * (|a| + |b|) times the angle's 2^-22 (half turns to 2^-25, frequencies
    and positions exact), sine and cosine 2 units of 2^-23 at most, amplitude,
    products and sum 2^-24 each."""
    x = x.double().abs()
    h = rope["freq"].numel()
    err = torch.zeros_like(x)
    amp = abs(float(rope.get("amplitude", 1.0)))
    if rope.get("interleaved"):
        m = amp * (x[..., 0:2 * h:2] + x[..., 1:2 * h:2]) * 2.0 ** -20
        err[..., 0:2 * h:2], err[..., 1:2 * h:2] = m, m
    else:
        m = amp * (x[..., :h] + x[..., h:2 * h]) * 2.0 ** -20
        err[..., :h], err[..., h:2 * h] = m, m
    return err


def need(amax):
    """Smallest power of two with amax <= 448 times it, within the scales' range."""
    if not amax > 448 * LOW:
        return LOW
    return min(HIGH, 2.0 ** math.ceil(math.log2(amax / 448)))


def e4m3(x):
    """Nearest E4M3 value of float64 x, ties to even, saturating."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -30))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def held(cache, r, m, side):
    """Rows of request r, [m, kv, D] in 64 bits."""
    k = cache[side]
    page = k.shape[2]
    ids = cache["table"][r, :(m + page - 1) // page].long()
    s = cache[side + "_scale"][ids].double()[:, :, None, None]
    x = (values(k[ids].contiguous().view(torch.uint8)) * s).transpose(1, 2)
    return x.reshape(-1, k.shape[1], k.shape[3])[:m]


def make_cache(rows, kv, dim, page, seed=0, device="cuda", extra=3, spread=1.0, strided=False):
    """Pages in random order full of normal rows, each block of its own strength;
    rows behind a request's last, and pages of nobody, are NaN codes."""
    g = torch.Generator(device=device).manual_seed(seed)
    count = [(m + page - 1) // page for m in rows]
    n = sum(count) + extra
    order = torch.randperm(n, generator=g, device=device).to(torch.int32)
    table = torch.full((max(1, len(rows)), max(count + [0]) + 1), -7, dtype=torch.int32,
                       device=device)
    if strided:                        # K and V page by page in one array
        both = torch.full((n, 2, kv, page, dim), NAN, dtype=torch.uint8, device=device)
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = (torch.full((n, kv, page, dim), NAN, dtype=torch.uint8, device=device)
                for _ in range(2))
    c = dict(k=k, v=v, table=table)
    for side in "kv":
        s = torch.exp2(torch.randint(-9, -5, (n, kv), generator=g, device=device).float())
        c[side + "_scale"] = s * torch.exp(spread * torch.randn((n, kv), generator=g,
                                                                device=device))
    at = 0
    for r, m in enumerate(rows):
        ids = order[at:at + count[r]]
        table[r, :count[r]] = ids
        at += count[r]
        for i, p in enumerate(ids.tolist()):
            here = min(page, m - i * page)
            for side in "kv":
                x = torch.randn((kv, here, dim), generator=g, device=device) * 60
                c[side][p, :, :here] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return c


def attend(q, keys, vals, scale, last):
    """One request: q [n, H, D] over keys, vals [m, Hkv, D]; query i sees the keys <=
    last[i].  Returns out, lse, sum of |weights * values|, largest sum_d |q k| * scale."""
    n, h, d = q.shape
    kv, m = keys.shape[1], keys.shape[0]
    if not m:
        z = torch.zeros((n, h, d), dtype=torch.float64, device=q.device)
        return z, torch.full((n, h), -math.inf, dtype=torch.float64, device=q.device), z, z[..., 0]
    q = q.double()
    k, v = (x.repeat_interleave(h // kv, 1) for x in (keys, vals))
    see = (torch.arange(m, device=q.device)[None, :] <= last[:, None])[:, None, :]
    x = torch.einsum("nhd,mhd->nhm", q, k) * scale
    mag = (torch.einsum("nhd,mhd->nhm", q.abs(), k.abs()) * scale * see).amax(2)
    x = torch.where(see, x, -math.inf)
    lse = torch.logsumexp(x, 2)
    w = torch.where(see, torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[..., None]), 0.0)
    return (torch.einsum("nhm,mhd->nhd", w, v), lse, torch.einsum("nhm,mhd->nhd", w, v.abs()),
            mag)


def check_attention(out, lse, ref, dtype, n_keys, v_scale=1.0):
    """|error| bounds.  Weights times their block's scale are rounded to f16 (2^-11 of
    each) and the output to its type.  A logit of D <= 128 exact products added in fp32
    is off by at most 2^-17 of sum |q k|, its factors (the row's, the block's, the
    softmax's and the logarithm of V's scale) by 2^-21 of that and 2^-19 in all, which
    moves every weight by that much relatively, and the sum under it too; sums over
    the keys add n 2^-24, the exponential 2^-22.  A weight under f16's normal range is
    off by 2^-33 of the largest, times a code of at most 448."""
    ro, rl, ra, mag = ref
    dl = 2.0 ** -16.9 * mag + 2.0 ** -18
    tol = 2.0 ** -11 * ra * 1.01 + HALF_STEP[dtype] * ro.abs() * 1.01 \
        + ra * (2 * dl + n_keys * 2.0 ** -23)[..., None] \
        + n_keys * 2.0 ** -33 * 448 * v_scale + 1e-30
    if dtype == torch.float16:
        tol = tol + 2.0 ** -24            # outputs below f16's normal range
    d = (out.double() - ro).abs()
    bad = ~(d <= tol)
    assert not bad.any(), (float(d.max()), int(bad.sum()), float((d / tol).max()))
    if lse is not None:
        inf = rl.isinf()
        assert (lse.double()[inf] == -math.inf).all()
        d = (lse.double() - rl).abs()[~inf]
        t = (dl + n_keys * 2.0 ** -24 + rl.abs() * 2.0 ** -22)[~inf]
        assert (d <= t).all(), (float(d.max()), float(t.min()))
