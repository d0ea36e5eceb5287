"""Workloads of the dense-cache operators: the prompt attention, the attention
over a shared prefix, the accumulated attention weight of cached rows and the
eviction that goes by it.

``run`` makes one pass through one operator: with ``own`` false in elementary
torch operations in 32 bits, with ``own`` true through the package's calls.
Queries, keys and values are N(0, 1) as after the projections' normalisation;
accumulated weights are log-normal, with exact ties and exact zeros as a cache
has them (fresh rows no query has looked at yet).

Sizes: 64 query heads, 128-token tails, 8 requests of 8192 tokens and 256
decode requests are the package's own workloads; the rest is generic.
"""
import math
import random

import torch

own = False

DEV = "cuda"
CHUNK = 1 << 28            # scores held at a time by the plain forms


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a few short extends over cached prefixes, one request idle: latency
        dict(name="prompt_extend_small", op="prompt", reqs=5, tokens=61, cached=700, idle=True,
             heads=16, kv_heads=4, dim=64, dtype="float16", lens=11),
        # a batch of ragged prompts, one of them most of the batch
        dict(name="prompt_packed_ragged", op="prompt", reqs=7, tokens=9001, cached=0, idle=False,
             heads=64, kv_heads=8, dim=128, dtype="bfloat16", lens=12),
        # narrow heads, three query heads to a key head, over a cached part
        dict(name="prompt_narrow_heads", op="prompt", reqs=12, tokens=12345, cached=1500,
             idle=False, heads=24, kv_heads=8, dim=64, dtype="float16", lens=13),
        # one long prompt
        dict(name="prompt_long", op="prompt", reqs=1, tokens=16384, cached=0, idle=False,
             heads=32, kv_heads=4, dim=128, dtype="bfloat16", lens=14),
        # four decode requests behind one system prompt: latency
        dict(name="prefix_decode_small", op="prefix", reqs=4, groups=1, prefix=1001, rest=90,
             heads=16, kv_heads=4, dim=64, dtype="float16", lens=21),
        # two system prompts, 48 decode requests of ordinary length
        dict(name="prefix_decode_groups", op="prefix", reqs=48, groups=2, prefix=8192, rest=700,
             heads=64, kv_heads=8, dim=128, dtype="bfloat16", lens=22),
        # 256 decode requests behind one long document
        dict(name="prefix_decode_large", op="prefix", reqs=256, groups=1, prefix=32768, rest=2048,
             heads=64, kv_heads=8, dim=128, dtype="bfloat16", lens=23),
        # the weight that the 128-token tails of eight prompts put on their cache
        dict(name="mass_prompt_tails", op="mass", reqs=8, queries=128, rows=8192, fresh=True,
             heads=64, kv_heads=8, dim=128, dtype="bfloat16", lens=31),
        # one decode step's weight added to the accumulated one
        dict(name="mass_decode_step", op="mass", reqs=61, queries=1, rows=9000, fresh=False,
             heads=64, kv_heads=8, dim=128, dtype="bfloat16", lens=32),
        # two short caches cut to their budget: latency
        dict(name="evict_small", op="evict", reqs=2, rows=601, keep=257, sink=4, recent=32,
             kv_heads=4, dim=64, dtype="float16", lens=41),
        # eight prompts cut to a quarter
        dict(name="evict_prompts", op="evict", reqs=8, rows=8192, keep=2048, sink=4, recent=128,
             kv_heads=8, dim=128, dtype="bfloat16", lens=42),
        # a serving batch of long caches, one key head each on a long range
        dict(name="evict_long_caches", op="evict", reqs=24, rows=40000, keep=4095, sink=16,
             recent=512, kv_heads=8, dim=128, dtype="bfloat16", lens=43),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prefix", "mass", "evict"])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([g for g in (1, 2, 3, 4, 5, 8, 16) if kv * g <= 64])
    c = dict(op=op, heads=heads, kv_heads=kv, dim=rng.choice([64, 128]),
             dtype=rng.choice(["bfloat16", "float16"]), lens=rng.randrange(1 << 30))
    if op == "prompt":
        c.update(reqs=rng.randint(1, 12), tokens=_log(rng, 24, 10000),
                 cached=rng.choice([0, _log(rng, 8, 1500)]), idle=rng.random() < 0.3)
    elif op == "prefix":
        c.update(reqs=_log(rng, 3, 200), prefix=_log(rng, 500, 24000), rest=_log(rng, 20, 2000))
        c["groups"] = rng.randint(1, 3)
    elif op == "mass":
        c.update(reqs=_log(rng, 1, 48), queries=rng.choice([1, _log(rng, 2, 150)]),
                 rows=_log(rng, 300, 8000), fresh=rng.random() < 0.5)
    else:
        rows = _log(rng, 300, 30000)
        keep = _log(rng, 64, rows)
        sink = rng.randint(0, 16)
        c.update(reqs=_log(rng, 1, 24), rows=rows, keep=keep, sink=sink,
                 recent=rng.randint(0, min(300, keep - sink)))
        del c["heads"]
    return c


def _dtype(case):
    return {"bfloat16": torch.bfloat16, "float16": torch.float16}[case["dtype"]]


def _ragged(rng, n, lo, hi):
    """n lengths, log-uniform in [lo, hi]; the first is hi."""
    return [hi if i == 0 else _log(rng, lo, hi) for i in range(n)]


def _lens(case):
    """Lengths of a case's requests: new tokens, and rows of the cache."""
    rng = random.Random(case["lens"])
    r = case["reqs"]
    if case["op"] == "prompt":
        w = [rng.uniform(0.3, 1.0) ** 3 for _ in range(r)]
        new = [max(1, int(case["tokens"] * x / sum(w))) for x in w]
        new[0] = max(1, case["tokens"] - sum(new[1:]))
        if case["idle"] and r > 1:
            new[r // 2] = 0
        old = [rng.randint(case["cached"] // 4, case["cached"]) for _ in range(r)]
        return new, [a + b for a, b in zip(new, old)]
    if case["op"] == "prefix":
        return [1] * r, _ragged(rng, r, max(1, case["rest"] // 16), case["rest"])
    if case["op"] == "mass":
        rows = _ragged(rng, r, max(1, case["rows"] // 8), case["rows"])
        return [min(case["queries"], n) for n in rows], rows
    return [0] * r, _ragged(rng, r, max(1, case["rows"] // 4), case["rows"])


def _groups(case):
    """First request of each group of requests that share a prefix, and the
    prefixes' lengths."""
    g = min(case["groups"], case["reqs"])
    first = [i * case["reqs"] // g for i in range(g + 1)]
    return first, [case["prefix"] // (i + 1) for i in range(g)]


def _pairs(new, rows):
    """Visible (query, key) pairs: query i of n sees the keys up to m - n + i."""
    return sum(sum(max(0, m - n + i + 1) for i in (0, n - 1)) * n / 2 if n else 0
               for n, m in zip(new, rows))


def work(case):
    new, rows = _lens(case)
    d, kv = case["dim"], case["kv_heads"]
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in rows)
        b = kv * (4 * sum(rows) + 4 * case["reqs"] * case["keep"] + kept * 2 * (2 * 2 * d + 4))
        return {"bytes": b, "flops": kv * sum(rows)}
    h, nq = case["heads"], sum(new)
    b = nq * h * d * 2
    pairs = _pairs(new, rows)
    if case["op"] == "mass":
        b += nq * h * 4 + sum(rows) * kv * (2 * d + 4 + (0 if case["fresh"] else 4))
        return {"bytes": b, "flops": 2 * d * h * pairs}
    b += nq * h * (2 * d + 4) + sum(rows) * kv * 4 * d
    if case["op"] == "prefix":
        first, length = _groups(case)
        b += sum(length) * kv * 4 * d
        pairs += sum((first[i + 1] - first[i]) * length[i] for i in range(len(length)))
    return {"bytes": b, "flops": 4 * d * h * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _starts(lens, gap=3):
    """First rows of runs of the given lengths in a pool, a few unused rows
    between them; and the pool's rows."""
    at, out = gap, []
    for n in lens:
        out.append(at)
        at += n + gap
    return out, at


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt, d, kv = _dtype(case), case["dim"], case["kv_heads"]
    new, rows = _lens(case)
    prefix = _groups(case)[1] if case["op"] == "prefix" else []
    start, pool = _starts(rows + prefix)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)   # noqa: E731
    i64 = lambda v: torch.tensor(v, dtype=torch.int64, device=DEV)   # noqa: E731
    normal = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=dt)   # noqa: E731
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = dict(case=case, new=new, rows=rows, start=start[:len(rows)], cu=cu,
             k=normal(pool, kv, d), d_err=torch.zeros(1, dtype=torch.int32, device=DEV))
    s["batch"] = dict(num_q=cu[-1], num_req=len(rows), cu_q=i32(cu), kv_start=i64(s["start"]),
                      kv_len=i64(rows))
    if case["op"] != "mass":
        s["v"] = normal(pool, kv, d)
    if case["op"] == "evict":
        m = torch.exp(1.5 * torch.randn((kv, pool), generator=g, device=DEV))
        m = torch.where(m < 2.0, (m * 16).round() / 16, m)      # ties, and zeros
        s["mass"] = m
        s["dst_start"] = start = [i * case["keep"] for i in range(len(rows))]
        s["dst_start_t"] = i64(start)
        n = case["keep"] * len(rows)
        s["dst"] = [torch.zeros((n, kv, d), dtype=dt, device=DEV) for _ in range(2)]
        s["dst"].append(torch.zeros((kv, n), dtype=torch.float32, device=DEV))
        return s
    s["q"] = normal(cu[-1], case["heads"], d)
    s["scale"] = d ** -0.5
    if case["op"] == "prefix":
        first, length = _groups(case)
        s["first"], s["length"] = first, length
        s["prefix_start"] = start[len(rows):]
        s["group"] = dict(num_groups=len(length), cu_group=i32(first),
                          prefix_start=i64(s["prefix_start"]), prefix_len=i64(length),
                          max_prefix=max(length))
    if case["op"] == "mass":
        # logits of unit variance: the log of a row's sum is near ln(keys) + 1/2
        n_vis = torch.cat([torch.arange(m - n + 1, m + 1) for n, m in zip(new, rows)])
        s["lse"] = (torch.log(n_vis.double()).to(DEV)[:, None] + 0.5
                    + 0.1 * torch.randn((cu[-1], case["heads"]), generator=g, device=DEV)).float()
        s["old"] = None
        if not case["fresh"]:
            s["old"] = torch.exp(torch.randn((kv, pool), generator=g, device=DEV))
        s["mass"] = torch.zeros((kv, pool), dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# plain forms, in 32 bits
# ---------------------------------------------------------------------------

def _heads_first(x, groups=1):
    """[n, H, D] -> float32 [H / groups, n * groups, D], token-major."""
    n, h, d = x.shape
    x = x.float().reshape(n, h // groups, groups, d).transpose(0, 1)
    return x.reshape(h // groups, n * groups, d)


def _parts(q, k, v, scale, last):
    """Softmax parts of query rows q [Hkv, m, D] over keys k, v [Hkv, n, D]:
    row maxima, sums and unnormalised products.  Row i sees the keys <= last[i]."""
    s = torch.matmul(q, k.transpose(1, 2)) * scale
    s = s.masked_fill(torch.arange(k.shape[1], device=DEV)[None, :] > last[:, None], -math.inf)
    m = s.amax(2, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    return m, p.sum(2, keepdim=True), torch.matmul(p, v)


def _finish(m, l, o, q, out, lse):
    """Normalise and store the rows of query tokens q[...] = [n, H, D]."""
    n, h, d = q.shape
    kv = o.shape[0]
    o = torch.where(l > 0, o / l.clamp_min(1e-30), 0.0)
    out.copy_(o.reshape(kv, n, h // kv, d).transpose(0, 1).reshape(n, h, d))
    r = torch.where(l > 0, m + torch.log(l), -math.inf)
    lse.copy_(r.reshape(kv, n, h // kv).transpose(0, 1).reshape(n, h))


def _plain_prompt(s):
    q, out, lse = s["q"], torch.empty_like(s["q"]), s["q"].new_empty(s["q"].shape[:2],
                                                                     dtype=torch.float32)
    kv = s["k"].shape[1]
    grp = q.shape[1] // kv
    for r, (n, m) in enumerate(zip(s["new"], s["rows"])):
        if not n:
            continue
        k, v = (_heads_first(s[x][s["start"][r]:s["start"][r] + m]) for x in "kv")
        step = max(1, CHUNK // (q.shape[1] * max(m, 1)))
        for a in range(0, n, step):
            b = min(n, a + step)
            rows = slice(s["cu"][r] + a, s["cu"][r] + b)
            last = (m - n + torch.arange(a, b, device=DEV)).repeat_interleave(grp)
            seen = m - n + b                                 # keys that any row of these sees
            if seen <= 0:
                out[rows], lse[rows] = 0, -math.inf
                continue
            _finish(*_parts(_heads_first(q[rows], grp), k[:, :seen], v[:, :seen], s["scale"],
                            last), q[rows], out[rows], lse[rows])
    return out, lse


def _plain_prefix(s):
    q, out, lse = s["q"], torch.empty_like(s["q"]), s["q"].new_empty(s["q"].shape[:2],
                                                                     dtype=torch.float32)
    kv = s["k"].shape[1]
    grp = q.shape[1] // kv
    longest = max(s["rows"])
    at = torch.arange(longest, device=DEV)
    for g, length in enumerate(s["length"]):
        a, b = s["first"][g], s["first"][g + 1]             # one token a request
        p0 = s["prefix_start"][g]
        qh = _heads_first(q[a:b], grp)                       # [Hkv, (b - a) * grp, D]
        k, v = (_heads_first(s[x][p0:p0 + length]) for x in "kv")
        m1, l1, o1 = _parts(qh, k, v, s["scale"], torch.full((qh.shape[1],), length, device=DEV))
        # the requests' own rows, padded to the longest
        n = s["batch"]["kv_len"][a:b]
        rows = s["batch"]["kv_start"][a:b, None] + torch.minimum(at[None, :], n[:, None] - 1)
        k, v = (s[x][rows].float().permute(2, 0, 1, 3) for x in "kv")   # [Hkv, R, longest, D]
        qr = qh.reshape(kv, b - a, grp, -1)
        x = torch.matmul(qr, k.transpose(2, 3)) * s["scale"]
        x = x.masked_fill(at[None, None, None, :] >= n[None, :, None, None], -math.inf)
        m2 = x.amax(3, keepdim=True)
        p = torch.exp(x - m2)
        l2, o2 = p.sum(3, keepdim=True), torch.matmul(p, v)
        m2, l2, o2 = (y.reshape(kv, qh.shape[1], -1) for y in (m2, l2, o2))
        m = torch.maximum(m1, m2)
        w1, w2 = torch.exp(m1 - m), torch.exp(m2 - m)
        _finish(m, w1 * l1 + w2 * l2, w1 * o1 + w2 * o2, q[a:b], out[a:b], lse[a:b])
    return out, lse


def _plain_mass(s):
    kv = s["k"].shape[1]
    grp = s["q"].shape[1] // kv
    for r, (n, m) in enumerate(zip(s["new"], s["rows"])):
        rows = slice(s["cu"][r], s["cu"][r + 1])
        at = slice(s["start"][r], s["start"][r] + m)
        x = torch.matmul(_heads_first(s["q"][rows], grp),
                         _heads_first(s["k"][at]).transpose(1, 2)) * s["scale"]
        x = x - _heads_first(s["lse"][rows][:, :, None], grp)
        last = (m - n + torch.arange(n, device=DEV)).repeat_interleave(grp)
        x = x.masked_fill(torch.arange(m, device=DEV)[None, :] > last[:, None], -math.inf)
        w = torch.exp(x).sum(1)
        s["mass"][:, at] = w if s["old"] is None else s["old"][:, at] + w
    return s["mass"]


def _plain_evict(s):
    c = s["case"]
    keep, longest = c["keep"], max(s["rows"])
    n = s["batch"]["kv_len"]
    at = torch.arange(longest, device=DEV)
    rows = s["batch"]["kv_start"][:, None] + torch.minimum(at[None, :], n[:, None] - 1)
    x = s["mass"][:, rows].transpose(0, 1)                            # [R, Hkv, longest]
    always = (at[None, :] < c["sink"]) | (at[None, :] >= n[:, None] - c["recent"])
    x = torch.where(always[:, None, :], math.inf, x)
    x = torch.where((at[None, :] < n[:, None])[:, None, :], x, -math.inf)
    order = torch.sort(x, dim=2, descending=True, stable=True).indices[:, :, :keep]
    if order.shape[2] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[2]), value=longest)
    order = torch.where(order < n[:, None, None], order, longest)
    idx = torch.sort(order, dim=2).values
    new_len = n.clamp_max(keep)
    held = torch.arange(keep, device=DEV)[None, :] < new_len[:, None]   # [R, keep]
    idx = torch.where(held[:, None, :], idx, -1)
    src = (s["batch"]["kv_start"][:, None, None] + idx).transpose(1, 2)[held]   # [rows kept, Hkv]
    dst = (s["dst_start_t"][:, None] + torch.arange(keep, device=DEV)[None, :])[held]
    h = torch.arange(c["kv_heads"], device=DEV)
    s["dst"][0][dst] = s["k"][src, h]
    s["dst"][1][dst] = s["v"][src, h]
    s["dst"][2][:, dst] = s["mass"][h, src].t()
    return idx.to(torch.int32), new_len, s["dst"]


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------

def _own(s):
    import sparse_attention_prefill_gb300 as S
    op, b = s["case"]["op"], s["batch"]
    if op == "prompt":
        return S.prompt_attn(b, s["q"], s["k"], s["v"], sm_scale=s["scale"], d_err=s["d_err"])
    if op == "prefix":
        return S.prefix_attn(b, s["group"], s["q"], s["k"], s["v"], max_kv=max(s["rows"]),
                             sm_scale=s["scale"], d_err=s["d_err"])
    if op == "mass":
        return S.attn_mass(b, s["q"], s["k"], s["lse"], max_kv=max(s["rows"]),
                           sm_scale=s["scale"], mass_in=s["old"], mass=s["mass"],
                           d_err=s["d_err"])
    c = s["case"]
    idx, new_len = S.evict_select(b["kv_start"], b["kv_len"], s["mass"], c["keep"],
                                  sink=c["sink"], recent=c["recent"], d_err=s["d_err"])
    k, v, m = s["dst"]
    S.evict_rows(idx, new_len, b["kv_start"], s["dst_start_t"],
                 [(s["k"], k), (s["v"], v), (s["mass"].t(), m.t())], d_err=s["d_err"])
    return idx, new_len, s["dst"]


def run(state):
    if own:
        return _own(state)
    return {"prompt": _plain_prompt, "prefix": _plain_prefix, "mass": _plain_mass,
            "evict": _plain_evict}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _softmax_rows(q, ks, vs, scale, seen):
    """Attention of one head's query rows q [n, D] over the concatenated key
    sets; seen[j] is the mask of set j, [n, keys]."""
    x = torch.cat([(q @ k.T * scale).where(m, torch.tensor(-math.inf, dtype=q.dtype, device=DEV))
                   for k, m in zip(ks, seen)], 1)
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - torch.where(lse.isinf(), 0.0, lse)[:, None])
    return p @ torch.cat(vs), lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "evict":
        return _exact_evict(s)
    q, k = s["q"].double(), s["k"].double()
    h, kv = q.shape[1], k.shape[1]
    if op == "mass":
        mass = torch.zeros((kv, k.shape[0]), dtype=torch.float64, device=DEV)
        for r, (n, m) in enumerate(zip(s["new"], s["rows"])):
            a, p = s["cu"][r], s["start"][r]
            see = (torch.arange(m, device=DEV)[None, :]
                   <= torch.arange(m - n, m, device=DEV)[:, None])
            for i in range(h):
                w = torch.exp(q[a:a + n, i] @ k[p:p + m, i * kv // h].T * s["scale"]
                              - s["lse"][a:a + n, i].double()[:, None])
                mass[i * kv // h, p:p + m] += (w * see).sum(0)
            if s["old"] is not None:
                mass[:, p:p + m] += s["old"][:, p:p + m].double()
        return mass
    v = s["v"].double()
    out, lse = torch.empty_like(q), q.new_empty(q.shape[:2])
    if op == "prompt":
        for r, (n, m) in enumerate(zip(s["new"], s["rows"])):
            a0, p = s["cu"][r], s["start"][r]
            step = max(1, CHUNK // 4 // max(m, 1))
            for a in range(0, n, step):
                b = min(n, a + step)
                top = max(0, m - n + b)
                see = (torch.arange(top, device=DEV)[None, :]
                       <= torch.arange(m - n + a, m - n + b, device=DEV)[:, None])
                for i in range(h):
                    j = i * kv // h
                    out[a0 + a:a0 + b, i], lse[a0 + a:a0 + b, i] = _softmax_rows(
                        q[a0 + a:a0 + b, i], [k[p:p + top, j]], [v[p:p + top, j]], s["scale"],
                        [see])
        return out, lse
    for g, length in enumerate(s["length"]):
        a, b, p = s["first"][g], s["first"][g + 1], s["prefix_start"][g]
        # each request's rows of the union: the prefix, then its own
        for i in range(h):
            j = i * kv // h
            x = q[a:b, i] @ k[p:p + length, j].T * s["scale"]
            l1 = torch.logsumexp(x, 1)
            o1 = torch.exp(x - l1[:, None]) @ v[p:p + length, j]
            out[a:b, i], lse[a:b, i] = o1, l1
    for r, m in enumerate(s["rows"]):
        p = s["start"][r]
        x = torch.einsum("jgd,mjd->jgm", q[r].view(kv, h // kv, -1), k[p:p + m]) * s["scale"]
        l2 = torch.logsumexp(x, 2)
        o2 = torch.einsum("jgm,mjd->jgd", torch.exp(x - l2[..., None]), v[p:p + m])
        l1 = lse[r].clone()
        l2, o2 = l2.reshape(h), o2.reshape(h, -1)
        l = torch.logaddexp(l1, l2)
        out[r] = torch.exp(l1 - l)[:, None] * out[r] + torch.exp(l2 - l)[:, None] * o2
        lse[r] = l
    return out, lse


def _exact_evict(s):
    c = s["case"]
    idx = torch.full((len(s["rows"]), c["kv_heads"], c["keep"]), -1, dtype=torch.int64)
    mass = s["mass"].double().cpu()
    for r, n in enumerate(s["rows"]):
        x = mass[:, s["start"][r]:s["start"][r] + n].clone()
        for a in range(c["kv_heads"]):
            kept = torch.zeros(n, dtype=torch.bool)
            kept[:c["sink"]] = True
            kept[max(0, n - c["recent"]):] = True
            room = min(n, c["keep"]) - int(kept.sum())
            if n <= c["keep"]:
                kept[:] = True
            elif room > 0:
                y = torch.where(kept, -1.0, x[a])
                edge = torch.topk(y, room).values[-1]
                kept |= y > edge
                ties = torch.nonzero(y == edge)[:, 0]
                kept[ties[:min(n, c["keep"]) - int(kept.sum())]] = True
            ids = torch.nonzero(kept)[:, 0]
            idx[r, a, :ids.numel()] = ids
    dst = [torch.zeros_like(x) for x in s["dst"]]
    for r, n in enumerate(s["rows"]):
        m = min(n, c["keep"])
        for a in range(c["kv_heads"]):
            src = s["start"][r] + idx[r, a, :m].to(DEV)
            at = slice(s["dst_start"][r], s["dst_start"][r] + m)
            dst[0][at, a], dst[1][at, a] = s["k"][src, a], s["v"][src, a]
            dst[2][a, at] = s["mass"][a, src]
    new_len = torch.tensor([min(n, c["keep"]) for n in s["rows"]], device=DEV)
    return idx.to(DEV), new_len, [x.double() for x in dst]
