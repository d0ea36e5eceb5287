"""How exact rotations are: pairs of channels that nearly cancel show the fp32 result, which a
16-bit output hides otherwise.  Angles of the reference come from integers."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import sparse_attention_prefill_gb300 as S
from tests import page_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inverse_of_two_pi(digits=80):
    """1 / 2 pi by pi = 16 atan(1/5) - 4 atan(1/239)."""
    unit = 10 ** (digits + 10)

    def atan(n):
        s, t, k = 0, unit // n, 1
        while t:
            s += t // k if k % 4 == 1 else -(t // k)
            t //= n * n
            k += 2
        return s

    return Fraction(unit, 2 * (16 * atan(5) - 4 * atan(239)))


PER_RADIAN = _inverse_of_two_pi()


def angles(pos, freq):
    """[positions, pairs] radians within a half turn, to 2^-52 of their value."""
    out = np.empty((len(pos), len(freq)))
    for i, p in enumerate(pos):
        for j, f in enumerate(freq):
            t = p * Fraction(f) * PER_RADIAN
            out[i, j] = float((t - round(t)) / PER_RADIAN)
    return out


def cancelling(a, seed):
    """f16 pairs (x, y) [2, *a.shape]: x cos a - y sin a nearly 0, then y cos a + x sin a."""
    rng = np.random.default_rng(seed)
    c, s = np.cos(a), np.sin(a)

    def pair(u, w):                      # y = x u / w or x = y w / u, the best of 256
        big = rng.uniform(512, 1024, (256,) + a.shape).astype(np.float16).astype(np.float64)
        flip = np.abs(u) > np.abs(w)
        small = (big * np.where(flip, w, u) / np.where(flip, u, w)).astype(np.float16)
        small = small.astype(np.float64)
        x, y = np.where(flip, small, big), np.where(flip, big, small)
        best = np.argmin(np.abs(x * u - y * w), 0)[None]
        return [np.take_along_axis(v, best, 0)[0] for v in (x, y)]

    x0, y0 = pair(c, s)
    x1, y1 = pair(s, -c)
    return np.stack([x0, x1]), np.stack([y0, y1])


def check(pos, freq, interleaved, amplitude, inverse, seed):
    """Cosine and sine, times the amplitude, are off by 0.82 units of the last place (2^-23 of
    the value at most) and 2^-48 of the amplitude near their zeros, products and their sum
    by 2^-24 each, and the angle by p 2^-64 turns."""
    a = angles(pos, freq) * (-1 if inverse else 1)
    x, y = cancelling(a, seed)
    n, h = a.shape
    rows = np.zeros((n, 2, 2 * h), np.float16)
    first, second = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else \
        (slice(0, h), slice(h, 2 * h))
    rows[..., first], rows[..., second] = x.transpose(1, 0, 2), y.transpose(1, 0, 2)
    rope = dict(freq=torch.tensor(freq, dtype=torch.float64, device=DEV), amplitude=amplitude,
                interleaved=interleaved)
    amp = float(np.float32(amplitude))
    got = S.rotate(dict(num_q=n), torch.from_numpy(rows).to(DEV), rope,
                   pos=torch.tensor(pos, device=DEV), inverse=inverse).cpu().double().numpy()
    c, s = np.cos(a), np.sin(a)
    turned = 2 * np.pi * 2.0 ** -64 * np.abs(np.array(pos, np.float64))[:, None]
    worst = 0.0
    for k in range(2):
        for ref, m, at in ((x[k] * c - y[k] * s, np.abs(x[k] * c) + np.abs(y[k] * s), first),
                           (y[k] * c + x[k] * s, np.abs(y[k] * c) + np.abs(x[k] * s), second)):
            tol = amp * (m * 1.33 * 2.0 ** -23
                         + (np.abs(x[k]) + np.abs(y[k])) * (2.0 ** -48 + turned)) \
                + amp * np.abs(ref) * (2.0 ** -24 + 2.0 ** -11 * 1.001) + 2.0 ** -25
            worst = max(worst, float((np.abs(got[:, k, at] - amp * ref) / tol).max()))
    assert worst <= 1, worst
    return worst


FREQS = [1.0, 3.0, 0.25, -0.5, 0.7071, 100.0, 1e-3, -1e-7, 2.0 ** -12, 2.0 ** -11, 1.9e-4, 4097.0,
         -1e6, 1e-9, 0.0, 2.0 ** 40] * 2


@pytest.mark.parametrize("inverse", [False, True])
def test_far_positions(inverse):
    """Frequencies near 1, held to 2^-56 of a turn, would be some ten units off at 2^33."""
    pos = [2 ** 31 + 7, 2 ** 33 + 1, -(2 ** 33) - 5, 2 ** 34 - 3, 3 * 2 ** 33 + 11, 2 ** 35]
    check(pos, FREQS, inverse, 1.0, inverse, seed=1)


@pytest.mark.parametrize("interleaved,amplitude", [(False, 1.0), (True, 1.0),
                                                   (False, 0.1 * np.log(8.0) + 1), (True, 0.6)])
@pytest.mark.parametrize("inverse", [False, True])
def test_positions_of_long_contexts(interleaved, amplitude, inverse):
    """Within one unit of cosine and sine, where two would show."""
    rng = np.random.default_rng(5)
    pos = [int(p) for p in rng.integers(1, 1 << 20, 150)] + [0, 1, 2, 3]
    freq = [10000.0 ** (-2 * i / 64) for i in range(32)]
    check(pos, freq, interleaved, amplitude, inverse, seed=2)


@pytest.mark.parametrize("new,interleaved,dtype", [([4000, 96], False, torch.bfloat16),
                                                   ([1] * 300, True, torch.float16)])
def test_codes_of_rotated_keys_are_those_of_64_bits(new, interleaved, dtype):
    """An appended key's code is another one than the 64-bit rotation's only where that lies
    as near to the middle of two codes as the error of the fp32 rotation allows."""
    kv, dim, page = 8, 128, 64
    rows = [n + (0 if n > 1 else 64 * (3 + i % 50)) for i, n in enumerate(new)]
    c = R.make_cache(new, kv, dim, page, seed=3)
    if new[0] == 1:                      # the first rows of pages further on
        table = torch.zeros((len(new), 60), dtype=torch.int32, device=DEV)
        table[torch.arange(len(new)), torch.tensor(rows) // page] = c["table"][:, 0]
        c["table"] = table
    g = torch.Generator(device=DEV).manual_seed(4)
    b, cu = R.batch(new, rows, DEV)
    k = torch.randn((b["num_q"], kv, dim), generator=g, device=DEV).to(dtype)
    rope = dict(S.rope_freqs(dim), interleaved=interleaved)
    S.page_append(b, k, k, c, rope=rope)
    pos = torch.cat([torch.arange(m - n, m, device=DEV) for n, m in zip(new, rows)])
    u = R.rotate(k, pos, rope)
    z = R.rotation(pos, rope)
    h = dim // 2
    x = k.double().abs()
    p, q = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :h], x[..., h:])
    co, si = z.real.abs()[:, None], z.imag.abs()[:, None]
    # (the turn's 2^-64 a position, and the reference's angles, half a step of 64 bits)
    angle = (2.0 ** -48 + pos.double()[:, None] * (2.0 ** -61 + rope["freq"] * 2.0 ** -52))[:, None]
    e0 = (p * co + q * si) * 1.33 * 2.0 ** -23 + (p + q) * angle
    e1 = (q * co + p * si) * 1.33 * 2.0 ** -23 + (p + q) * angle
    err = (torch.stack([e0, e1], 3).flatten(2) if interleaved else torch.cat([e0, e1], 2)) \
        + u.abs() * 2.0 ** -24
    req = torch.repeat_interleave(torch.arange(len(new), device=DEV), torch.tensor(new, device=DEV))
    block, slot = c["table"].long()[req, pos // page], pos % page
    scale = c["k_scale"].double()[block][..., None]
    got = R.values(c["k"][block, :, slot].contiguous())
    want = R.e4m3(u / scale)
    differ = got != want
    middle = (got + want) / 2 * scale
    assert ((u - middle).abs() <= err)[differ].all()
    assert ((got - want).abs() * 8 <= torch.maximum(got.abs(), want.abs()).clamp_min(2.0 ** -6)
            )[differ].all()
    assert int(differ.sum()) <= differ.numel() * 1e-4
