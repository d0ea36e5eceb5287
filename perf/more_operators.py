"""Workloads of the paged 8-bit cache: rotary positions, keys and values appended
to pages with the rotation on the way, and attention over what the pages hold.

``run`` makes one pass through one operator: with ``own`` false in elementary
torch operations in 32 bits (angles in 64), with ``own`` true through the
package's calls.

A page holds ``page`` rows of one request, E4M3 codes [kv_heads, page, dim], with
one fp32 scale for each page and head; a table names each request's pages in
order.  Appending picks the smallest power of two under which a block's rows stay
within 448, never below the scale that older rows of the block have, and rescales
those where the new one is larger.

Queries, keys and values are normal, keys with a few strong channels as the
projections give them; positions reach the 512K contexts that the package's mixed
workload has.  Sizes: 64 query heads on 8 key heads, 8 requests of 8192 tokens, 256
decode requests and 64-token extends are the package's own; the rest is generic.
"""
import math
import random

import torch

own = False

DEV = "cuda"
CHUNK = 1 << 28            # scores held at a time by the plain forms
TOP = 448.0                # the largest E4M3 value
LOW, HIGH = 2.0 ** -32, 2.0 ** 32        # range of a block's scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # queries of one small decode step: latency
        dict(name="rotate_step_small", op="rotate", reqs=5, tokens=5, cached=3000, heads=16, dim=64,
             rot=32, layout="interleaved", scaling="none", inverse=False, dtype="float16", lens=11),
        # queries of eight prompts behind long contexts, frequencies scaled by their wavelength
        dict(name="rotate_prompts", op="rotate", reqs=8, tokens=16001, cached=500000, heads=64,
             dim=128, rot=128, layout="half", scaling="ramp", inverse=False, dtype="bfloat16",
             lens=12),
        # the gradient of rotated queries, half of each head rotated
        dict(name="rotate_gradient", op="rotate", reqs=12, tokens=12345, cached=0, heads=24,
             dim=64, rot=32, layout="interleaved", scaling="linear", inverse=True,
             dtype="float16", lens=13),
        # one decode step of four requests: latency
        dict(name="append_step_small", op="append", reqs=4, tokens=4, cached=700, kv_heads=4,
             dim=64, page=16, rot=64, layout="half", scaling="none", dtype="float16", lens=21),
        # one decode step of a serving batch
        dict(name="append_step", op="append", reqs=256, tokens=256, cached=4000, kv_heads=8,
             dim=128, page=64, rot=128, layout="half", scaling="none", dtype="bfloat16", lens=22),
        # ragged extends, most of them begin inside a page
        dict(name="append_extends", op="append", reqs=12, tokens=3001, cached=1500, kv_heads=8,
             dim=64, page=32, rot=32, layout="interleaved", scaling="base", dtype="float16",
             lens=23),
        # eight prompts
        dict(name="append_prompts", op="append", reqs=8, tokens=65536, cached=0, kv_heads=8,
             dim=128, page=64, rot=128, layout="half", scaling="ramp", dtype="bfloat16", lens=24),
        # four decode requests: latency
        dict(name="attn_step_small", op="attn", reqs=4, tokens=4, cached=1001, heads=16,
             kv_heads=4, dim=64, page=16, dtype="float16", lens=31),
        # a decode step of ordinary caches
        dict(name="attn_step", op="attn", reqs=61, tokens=61, cached=9000, heads=64, kv_heads=8,
             dim=128, page=64, dtype="bfloat16", lens=32),
        # a decode step of long caches
        dict(name="attn_step_long", op="attn", reqs=96, tokens=96, cached=32768, heads=64,
             kv_heads=8, dim=128, page=64, dtype="bfloat16", lens=33),
        # 64-token extends over cached prompts
        dict(name="attn_extends", op="attn", reqs=16, tokens=1024, cached=8192, heads=64,
             kv_heads=8, dim=128, page=32, dtype="bfloat16", lens=34),
        # one long prompt
        dict(name="attn_prompt_long", op="attn", reqs=1, tokens=16384, cached=0, heads=32,
             kv_heads=4, dim=128, page=128, dtype="bfloat16", lens=35),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "attn", "attn"])
    dim = rng.choice([64, 128])
    c = dict(op=op, dim=dim, dtype=rng.choice(["bfloat16", "float16"]),
             lens=rng.randrange(1 << 30))
    kv = rng.choice([1, 2, 4, 8])
    if op != "attn":
        c.update(rot=rng.choice([r for r in (16, 32, 64, 96, 128) if r <= dim]),
                 layout=rng.choice(["half", "interleaved"]),
                 scaling=rng.choice(["none", "linear", "base", "ramp"]))
    if op == "rotate":
        tokens = _log(rng, 1, 15000)
        c.update(reqs=rng.randint(1, min(tokens, 40)), tokens=tokens,
                 cached=rng.choice([0, _log(rng, 10, 500000)]), heads=kv * rng.choice([1, 3, 8]),
                 inverse=rng.random() < 0.4)
        return c
    c.update(kv_heads=kv, page=rng.choice([16, 32, 64, 128]))
    kind = rng.choice(["step", "step", "extend", "prompt"])
    if op == "append":
        if kind == "step":
            n = _log(rng, 2, 300)
            c.update(reqs=n, tokens=n, cached=_log(rng, 20, 5000))
        elif kind == "extend":
            c.update(reqs=rng.randint(1, 24), tokens=_log(rng, 60, 6000),
                     cached=_log(rng, 20, 3000))
        else:
            c.update(reqs=rng.randint(1, 12), tokens=_log(rng, 60, 40000), cached=0)
        return c
    c["heads"] = kv * rng.choice([g for g in (1, 2, 3, 5, 8, 16) if kv * g <= 64])
    if kind == "step":
        n = _log(rng, 2, 120)
        c.update(reqs=n, tokens=n, cached=_log(rng, 300, 12000))
    elif kind == "extend":
        c.update(reqs=rng.randint(1, 16), tokens=_log(rng, 40, 1500),
                 cached=_log(rng, 200, 6000))
    else:
        c.update(reqs=rng.randint(1, 8), tokens=_log(rng, 60, 9000), cached=0)
    return c


def _dtype(case):
    return {"bfloat16": torch.bfloat16, "float16": torch.float16}[case["dtype"]]


def _lens(case):
    """New tokens of each request, and rows of its cache with these."""
    rng = random.Random(case["lens"])
    r, n = case["reqs"], case["tokens"]
    if n == r:
        new = [1] * r
    elif n % r == 0 and n // r >= 64:
        new = [n // r] * r                    # equal extends or prompts
    else:
        w = [rng.uniform(0.3, 1.0) ** 3 for _ in range(r)]
        new = [max(1, int(n * x / sum(w))) for x in w]
        new[0] = max(1, n - sum(new[1:]))
    c = case["cached"]
    old = [c if i == 0 else (_log(rng, max(1, c // 16), c) if c else 0) for i in range(r)]
    return new, [a + b for a, b in zip(new, old)]


def _pairs(new, rows):
    """Visible (query, key) pairs: query i of n sees the keys up to m - n + i."""
    return sum(n * (m - n) + n * (n + 1) / 2 for n, m in zip(new, rows))


def work(case):
    new, rows = _lens(case)
    d, n = case["dim"], sum(new)
    if case["op"] == "rotate":
        return {"bytes": 4 * n * case["heads"] * d, "flops": 3 * n * case["heads"] * case["rot"]}
    kv, page = case["kv_heads"], case["page"]
    if case["op"] == "append":
        blocks = sum((m + page - 1) // page - (m - k) // page for k, m in zip(new, rows))
        # two bytes in and one out for each channel of K and V; the blocks' scales and pages
        return {"bytes": 6 * n * kv * d + 8 * kv * blocks + 4 * blocks,
                "flops": n * kv * (4 * d + 3 * case["rot"])}
    blocks = sum((m + page - 1) // page for m in rows)
    b = n * case["heads"] * (4 * d + 4) + sum(rows) * kv * 2 * d + blocks * (8 * kv + 4)
    return {"bytes": b, "flops": 4 * d * case["heads"] * _pairs(new, rows)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _frequencies(case):
    """Radians per position of each pair of channels, and the amplitude: as they
    are; divided by the factor; of a larger base; or divided by the factor only
    where a pair turns less than once over the original context, with a ramp up
    to 32 turns."""
    rot, kind, factor, original = case["rot"], case["scaling"], 8.0, 65536
    base = 10000.0 * (factor ** (rot / (rot - 2)) if kind == "base" else 1.0)
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    if kind == "linear":
        return f / factor, 1.0
    if kind == "ramp":
        turns = original * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1
    return f, 1.0


def _gains(g, kv, dim):
    """Strengths of the key channels, of mean square 1: one in sixteen strong."""
    x = torch.where(torch.rand((kv, dim), generator=g, device=DEV) < 1 / 16, 4.0, 0.8)
    return x / x.square().mean(1, keepdim=True).sqrt()


def _block_scale(amax):
    """Smallest power of two with amax <= 448 times it."""
    f, e = torch.frexp(amax)
    e = torch.where(f > 0.875, e - 8, e - 9)
    s = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=amax.device), e.double())
    return torch.where(amax > 0, s, LOW).clamp(LOW, HIGH).float()


def _filled(g, pages, kv, page, dim, gain):
    """Codes [pages, kv, page, dim] and scales of pages that are full of normal rows."""
    x = torch.randn((pages, kv, page, dim), generator=g, device=DEV)
    if gain is not None:
        x *= gain[None, :, None, :]
    s = _block_scale(x.abs().amax((2, 3)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt, d = _dtype(case), case["dim"]
    new, rows = _lens(case)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    normal = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=dt)   # noqa: E731
    i64 = lambda v: torch.tensor(v, dtype=torch.int64, device=DEV)   # noqa: E731
    s = dict(case=case, new=new, rows=rows, cu=cu,
             d_err=torch.zeros(1, dtype=torch.int32, device=DEV))
    s["batch"] = dict(num_q=cu[-1], num_req=len(new),
                      cu_q=torch.tensor(cu, dtype=torch.int32, device=DEV), kv_len=i64(rows))
    if case["op"] != "attn":
        f, a = _frequencies(case)
        s["rope"] = dict(freq=f.to(DEV), amplitude=a, interleaved=case["layout"] == "interleaved")
    if case["op"] == "rotate":
        s["x"] = normal(cu[-1], case["heads"], d)
        return s
    kv, page = case["kv_heads"], case["page"]
    count = [(m + page - 1) // page for m in rows]
    pages = sum(count) + 3                                     # three belong to nobody
    gain = _gains(g, kv, d)
    k, ks = _filled(g, pages, kv, page, d, gain)
    v, vs = _filled(g, pages, kv, page, d, None)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(new), max(count) + 1), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(count):
        table[r, :n] = order[at:at + n]
        at += n
    s["cache"] = dict(k=k, v=v, k_scale=ks, v_scale=vs, table=table)
    if case["op"] == "append":
        s["k"] = (normal(cu[-1], kv, d).float() * gain).to(dt)
        s["v"] = normal(cu[-1], kv, d)
        # the blocks' older rows come from shorter ranges, so that some have to be rescaled
        for x in (ks, vs):
            x *= torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.3, 0.5, 1.0)
    else:
        s["q"] = normal(cu[-1], case["heads"], d)
        s["scale"] = d ** -0.5
    return s


# ---------------------------------------------------------------------------
# plain forms, in 32 bits
# ---------------------------------------------------------------------------

def _row_requests(s):
    """Request of each query row, and its row in the request's cache."""
    n = torch.tensor(s["new"], device=DEV)
    req = torch.repeat_interleave(torch.arange(len(s["new"]), device=DEV), n)
    b = s["batch"]
    i = torch.arange(b["num_q"], device=DEV) - b["cu_q"].long()[req]
    return req, b["kv_len"][req] - n[req] + i


def _rotated(x, pos, rope, inverse=False):
    """x [n, heads, dim] in 32 bits, its first channels rotated by pos."""
    f = rope["freq"]
    rot = 2 * f.numel()
    angle = pos.double()[:, None] * f[None, :]
    c = (torch.cos(angle) * rope["amplitude"]).float()[:, None, :]
    t = (torch.sin(angle) * rope["amplitude"]).float()[:, None, :]
    if inverse:
        t = -t
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if rope["interleaved"] else \
        (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * c - b * t, b * c + a * t
    y = torch.stack([u, w], 3).flatten(2) if rope["interleaved"] else torch.cat([u, w], 2)
    return torch.cat([y, x[..., rot:]], 2)


def _plain_rotate(s):
    pos = _row_requests(s)[1]
    return _rotated(s["x"], pos, s["rope"], s["case"]["inverse"]).to(s["x"].dtype)


def _append_blocks(s, x, codes, scale, req, row):
    """Rows x [n, heads, dim] into the blocks of one side of the cache."""
    page, table = codes.shape[2], s["cache"]["table"].long()
    block, slot = table[req, row // page], row % page
    need = torch.zeros_like(scale)
    need.index_reduce_(0, block, x.abs().amax(2), "amax")
    old_rows = torch.zeros(scale.shape[0], dtype=torch.int64, device=DEV)
    first = s["batch"]["cu_q"].long()[:-1]                     # each request's first new row
    old_rows[block[first]] = slot[first]
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=DEV)
    touched[block] = True
    now = _block_scale(need)
    now = torch.where((old_rows > 0)[:, None], torch.maximum(now, scale), now)
    now = torch.where(touched[:, None], now, scale)
    # older rows of the blocks that are filled up
    at = block[first]
    have = codes[at].view(torch.float8_e4m3fn).float()
    have = (have * (scale[at] / now[at])[:, :, None, None]).to(torch.float8_e4m3fn)
    keep = torch.arange(page, device=DEV)[None, :] < old_rows[at][:, None]
    codes[at] = torch.where(keep[:, None, :, None], have.view(torch.uint8), codes[at])
    codes[block, :, slot] = (x / now[block][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(now)


def _cache_values(s):
    c = s["cache"]
    return [c["k"].view(torch.float8_e4m3fn), c["v"].view(torch.float8_e4m3fn), c["k_scale"],
            c["v_scale"]]


def _plain_append(s):
    req, row = _row_requests(s)
    c = s["cache"]
    _append_blocks(s, _rotated(s["k"], row, s["rope"]), c["k"], c["k_scale"], req, row)
    _append_blocks(s, s["v"].float(), c["v"], c["v_scale"], req, row)
    return _cache_values(s)


def _held(s, r, side):
    """Rows of request r in 32 bits, [heads, rows, dim]."""
    c = s["cache"]
    codes, scale, m = c[side], c[side + "_scale"], s["rows"][r]
    kv, page, d = codes.shape[1:]
    at = c["table"][r, :(m + page - 1) // page].long()
    x = codes[at].view(torch.float8_e4m3fn).float() * scale[at][:, :, None, None]
    return x.transpose(0, 1).reshape(kv, -1, d)[:, :m]


def _plain_attn(s):
    q = s["q"]
    h, d = q.shape[1:]
    out, lse = torch.empty_like(q), q.new_empty(q.shape[:2], dtype=torch.float32)
    for r, (n, m) in enumerate(zip(s["new"], s["rows"])):
        k, v = _held(s, r, "k"), _held(s, r, "v")
        kv = k.shape[0]
        grp = h // kv
        step = max(1, CHUNK // (h * m))
        for a in range(0, n, step):
            b = min(n, a + step)
            at, seen = slice(s["cu"][r] + a, s["cu"][r] + b), m - n + b
            qh = q[at].float().reshape(b - a, kv, grp, d).transpose(0, 1).reshape(kv, -1, d)
            x = torch.matmul(qh, k[:, :seen].transpose(1, 2)) * s["scale"]
            if b - a > 1:
                last = (m - n + torch.arange(a, b, device=DEV)).repeat_interleave(grp)
                x.masked_fill_(torch.arange(seen, device=DEV)[None, :] > last[:, None], -math.inf)
            top = x.amax(2, keepdim=True)
            p = torch.exp(x - top)
            total = p.sum(2, keepdim=True)
            o = torch.matmul(p, v[:, :seen]) / total
            out[at] = o.reshape(kv, b - a, grp, d).transpose(0, 1).reshape(b - a, h, d).to(q.dtype)
            z = top + torch.log(total)
            lse[at] = z.reshape(kv, b - a, grp).transpose(0, 1).reshape(b - a, h)
    return out, lse


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------

def _own(s):
    import sparse_attention_prefill_gb300 as S
    op, b = s["case"]["op"], s["batch"]
    if op == "rotate":
        return S.rotate(b, s["x"], s["rope"], inverse=s["case"]["inverse"], d_err=s["d_err"])
    if op == "append":
        S.page_append(b, s["k"], s["v"], s["cache"], rope=s["rope"], d_err=s["d_err"])
        return _cache_values(s)
    return S.page_attn(b, s["q"], s["cache"], max_kv=max(s["rows"]), sm_scale=s["scale"],
                       d_err=s["d_err"])


def run(state):
    if own:
        return _own(state)
    return {"rotate": _plain_rotate, "append": _plain_append,
            "attn": _plain_attn}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _turn(x, pos, rope, sign):
    """Each pair of channels as a complex number, times amplitude * e^(i angle)."""
    x = x.double().clone()
    rot = 2 * rope["freq"].numel()
    w = torch.polar(torch.full((pos.numel(), rot // 2), float(rope["amplitude"]),
                               dtype=torch.float64, device=DEV),
                    sign * pos.double()[:, None] * rope["freq"][None, :])[:, None, :]
    if rope["interleaved"]:
        z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:2], rot // 2, 2).contiguous()) * w
        x[..., :rot] = torch.view_as_real(z).reshape(*x.shape[:2], rot)
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * w
        x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
    return x


def _nearest_code(x):
    """Nearest E4M3 value, ties to the even mantissa."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -20))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-TOP, TOP)


def exact(case, seed):
    s = prepare(case, seed)
    pos = torch.cat([torch.arange(m - n, m, device=DEV) for n, m in zip(s["new"], s["rows"])])
    if case["op"] == "rotate":
        return _turn(s["x"], pos, s["rope"], -1 if case["inverse"] else 1)
    c = s["cache"]
    if case["op"] == "append":
        return _exact_append(s, c, [_turn(s["k"], pos, s["rope"], 1), s["v"].double()])
    q = s["q"].double()
    h, d = q.shape[1:]
    out, lse = torch.empty_like(q), q.new_empty(q.shape[:2])
    for r, (n, m) in enumerate(zip(s["new"], s["rows"])):
        page = c["k"].shape[2]
        at = c["table"][r, :(m + page - 1) // page].long()
        for j in range(c["k"].shape[1]):
            kk, vv = ((c[x][at, j].view(torch.float8_e4m3fn).double()
                       * c[x + "_scale"][at, j].double()[:, None, None]).reshape(-1, d)[:m]
                      for x in "kv")
            grp = h // c["k"].shape[1]
            step = max(1, CHUNK // 4 // (m * grp))
            for a in range(0, n, step):
                b = min(n, a + step)
                seen, rows = m - n + b, slice(s["cu"][r] + a, s["cu"][r] + b)
                x = torch.einsum("ngd,md->ngm", q[rows, j * grp:(j + 1) * grp], kk[:seen])
                x = x * s["scale"]
                see = (torch.arange(seen, device=DEV)[None, :]
                       <= torch.arange(m - n + a, m - n + b, device=DEV)[:, None])
                x = torch.where(see[:, None, :], x, -math.inf)
                z = torch.logsumexp(x, 2)
                lse[rows, j * grp:(j + 1) * grp] = z
                out[rows, j * grp:(j + 1) * grp] = torch.einsum(
                    "ngm,md->ngd", torch.exp(x - z[..., None]), vv[:seen])
    return out, lse


def _exact_append(s, c, sides):
    codes = [c[x].view(torch.float8_e4m3fn).double() for x in "kv"]
    scales = [c[x + "_scale"].double() for x in "kv"]
    page = c["k"].shape[2]
    for x, have, scale in zip(sides, codes, scales):
        top = x.abs().amax(2)
        for r, (n, m) in enumerate(zip(s["new"], s["rows"])):
            ids = c["table"][r].tolist()
            for p in range((m - n) // page, (m + page - 1) // page):
                lo, hi = max(p * page, m - n), min((p + 1) * page, m)
                rows = slice(s["cu"][r] + lo - (m - n), s["cu"][r] + hi - (m - n))
                at, old = ids[p], lo - p * page
                need = torch.exp2(torch.ceil(torch.log2(top[rows].amax(0) / TOP)))
                now = torch.maximum(need, scale[at]) if old else need
                have[at, :, :old] = _nearest_code(have[at, :, :old]
                                                  * (scale[at] / now)[:, None, None])
                have[at, :, old:old + hi - lo] = _nearest_code(
                    (x[rows] / now[:, None]).transpose(0, 1))
                scale[at] = now
    return codes + scales
