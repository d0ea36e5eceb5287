"""Refusals of the calls on 8-bit pages that the host can see (no GPU needed): nothing
is launched, a status comes back."""
import ctypes as C
import math

import pytest
import torch

import sparse_attention_prefill_gb300 as S
from sparse_attention_prefill_gb300 import build

FAKE = 1 << 20           # never read: each case is refused before a launch
BIG = 1 << 34            # where the other arrays of a call are
INV, UNS = S.ERR_INVALID_ARG, S.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return S.load(build.build())


def _packed(**kw):
    d = dict(num_q=10, num_req=2, cu_q=BIG, kv_start=None, kv_len=BIG + 64)
    d.update(kw)
    return S.CPacked(*[d[k] for k in ("num_q", "num_req", "cu_q", "kv_start", "kv_len")])


def _rope(**kw):
    d = dict(freq=BIG + 4096, pos=None, rot=64, interleaved=0, amplitude=1.0)
    d.update(kw)
    return S.CRope(d["freq"], d["pos"], d["rot"], d["interleaved"], d["amplitude"], 0)


def _pages(**kw):
    # 9 pages of 16 rows, 2 heads of 128: 4096 bytes to a page and side
    d = dict(num_pages=9, page=16, k=2 * BIG, v=2 * BIG + (1 << 20), k_stride=4096,
             v_stride=4096, k_scale=3 * BIG, v_scale=3 * BIG + 4096, table=3 * BIG + 8192,
             table_ld=4)
    d.update(kw)
    return S.CPages(*[d[k] for k in ("num_pages", "page", "k", "v", "k_stride", "v_stride",
                                     "k_scale", "v_scale", "table", "table_ld")])


def _rotate(lib, b=None, h=8, dim=128, dt=S.DT_BF16, x=FAKE, ldx=1024, rope=None, out=4 * BIG,
            ldo=1024, err=None):
    b, rope = b or _packed(), rope or _rope()
    return lib.csa2_rotate(C.byref(b), h, dim, dt, x, ldx, C.byref(rope), 0, out, ldo, err, None)


@pytest.mark.parametrize("kw,status", [
    (dict(b=_packed(num_q=-1)), INV), (dict(b=_packed(num_req=-1)), INV),
    (dict(b=_packed(num_q=0)), S.OK), (dict(b=_packed(num_req=0)), S.OK),
    (dict(b=_packed(cu_q=None)), INV), (dict(b=_packed(kv_len=None)), INV),
    (dict(b=_packed(cu_q=BIG + 2)), UNS), (dict(b=_packed(kv_len=BIG + 4)), UNS),
    (dict(h=0), INV), (dict(h=65536, ldx=1 << 23, ldo=1 << 23), UNS), (dict(dim=96), UNS),
    (dict(dt=3), UNS), (dict(x=None), INV), (dict(out=None), INV), (dict(x=FAKE + 8), UNS),
    (dict(out=4 * BIG + 2), UNS), (dict(ldx=1000), INV), (dict(ldx=1028), UNS),
    (dict(ldo=512), INV), (dict(err=2), UNS),
    (dict(rope=_rope(freq=None)), INV), (dict(rope=_rope(freq=BIG + 4)), UNS),
    (dict(rope=_rope(rot=0)), UNS), (dict(rope=_rope(rot=24)), UNS),
    (dict(rope=_rope(rot=144)), UNS), (dict(rope=_rope(amplitude=math.nan)), INV),
    (dict(rope=_rope(amplitude=math.inf)), INV), (dict(rope=_rope(pos=BIG + 4)), UNS),
    # with positions the batch's arrays are not looked at
    (dict(rope=_rope(pos=BIG), b=_packed(num_q=0, cu_q=None, kv_len=None)), S.OK),
    # overlaps: another row distance, a shifted start, rows between each other's (fine:
    # refused for the next reason), the batch, the frequencies, the positions
    (dict(out=FAKE, ldo=2048), INV), (dict(out=FAKE + 2048), INV), (dict(out=FAKE + 16), INV),
    (dict(out=FAKE + 2048, ldx=2048, ldo=2048, err=2), UNS),
    (dict(out=BIG), INV), (dict(out=BIG + 64), INV), (dict(out=BIG + 4096), INV),
    (dict(out=4 * BIG, rope=_rope(pos=4 * BIG + 2048)), INV),
])
def test_rotate_refusals(lib, kw, status):
    assert _rotate(lib, **kw) == status


def _append(lib, b=None, kv=2, dim=128, dt=S.DT_BF16, k=FAKE, ldk=256, v=FAKE + (1 << 16),
            ldv=256, rope=None, cache=None, err=None):
    b, cache = b or _packed(), cache or _pages()
    return lib.csa2_page_append(C.byref(b), kv, dim, dt, k, ldk, v, ldv,
                                None if rope is None else C.byref(rope), C.byref(cache), err, None)


CACHE = [
    (dict(cache=_pages(num_pages=-1)), INV), (dict(cache=_pages(page=48)), UNS),
    (dict(cache=_pages(page=8)), UNS), (dict(cache=_pages(page=256)), UNS),
    (dict(cache=_pages(k=None)), INV), (dict(cache=_pages(v=None)), INV),
    (dict(cache=_pages(k_scale=None)), INV), (dict(cache=_pages(v_scale=None)), INV),
    (dict(cache=_pages(table=None)), INV), (dict(cache=_pages(table_ld=-1)), INV),
    (dict(cache=_pages(table_ld=1 << 28)), UNS), (dict(cache=_pages(k_stride=2048)), INV),
    (dict(cache=_pages(v_stride=4104)), UNS), (dict(cache=_pages(k=2 * BIG + 8)), UNS),
    (dict(cache=_pages(k_scale=3 * BIG + 2)), UNS), (dict(cache=_pages(table=3 * BIG + 2)), UNS),
    (dict(b=_packed(num_q=-1)), INV), (dict(b=_packed(cu_q=None)), INV),
    (dict(b=_packed(kv_len=None)), INV), (dict(b=_packed(kv_len=BIG + 4)), UNS),
    (dict(b=_packed(num_q=0)), S.OK), (dict(b=_packed(num_req=0)), S.OK), (dict(err=2), UNS),
    (dict(dt=4), UNS),
]


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(kv=0), INV), (dict(kv=1025), UNS), (dict(dim=80), UNS), (dict(k=None), INV),
    (dict(v=None), INV), (dict(k=FAKE + 2), UNS), (dict(ldk=128), INV), (dict(ldv=260), UNS),
    (dict(rope=_rope(rot=20)), UNS), (dict(rope=_rope(freq=None)), INV),
    (dict(rope=_rope(rot=192)), UNS),
    # what is written against what is read
    (dict(k=2 * BIG), INV), (dict(v=2 * BIG + (1 << 20)), INV), (dict(k=3 * BIG), INV),
    (dict(cache=_pages(table=3 * BIG)), INV), (dict(cache=_pages(k=BIG)), INV),
    (dict(rope=_rope(freq=3 * BIG + 4096)), INV), (dict(rope=_rope(pos=2 * BIG)), INV),
    # and against itself: sides page by page in one array are fine (refused for the flag)
    (dict(cache=_pages(v_scale=3 * BIG + 16)), INV), (dict(cache=_pages(k_scale=2 * BIG)), INV),
    (dict(cache=_pages(v=2 * BIG)), INV), (dict(cache=_pages(v=2 * BIG + 4096)), INV),
    (dict(cache=_pages(v=2 * BIG + 4096, k_stride=8192, v_stride=12288)), INV),
    (dict(cache=_pages(v=2 * BIG + 2048, k_stride=8192, v_stride=8192)), INV),
    (dict(cache=_pages(v=2 * BIG + 4096, k_stride=8192, v_stride=8192), err=2), UNS),
])
def test_append_refusals(lib, kw, status):
    assert _append(lib, **kw) == status


def _attn(lib, b=None, h=8, kv=2, dim=128, dt=S.DT_BF16, q=FAKE, ldq=1024, cache=None, max_kv=64,
          scale=0.1, out=4 * BIG, lse=None, ws=None, nbytes=0, err=None):
    b, cache = b or _packed(), cache or _pages()
    return lib.csa2_page_attn(C.byref(b), h, kv, dim, dt, q, ldq, C.byref(cache), max_kv, scale,
                              out, lse, ws, nbytes, err, None)


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(h=0), INV), (dict(kv=0), INV), (dict(h=9), INV), (dict(dim=96), UNS),
    (dict(h=258, ldq=258 * 128), UNS), (dict(scale=0.0), INV), (dict(scale=math.nan), INV),
    (dict(scale=math.inf), INV), (dict(max_kv=-1), INV), (dict(nbytes=-1), INV),
    (dict(nbytes=256), INV), (dict(ws=5 * BIG + 16, nbytes=4096), UNS), (dict(q=None), INV),
    (dict(q=FAKE + 4), UNS), (dict(ldq=1020), INV), (dict(ldq=1028), UNS), (dict(out=None), INV),
    (dict(out=4 * BIG + 8), UNS), (dict(lse=5 * BIG + 2), UNS),
    (dict(out=FAKE + 2048), INV), (dict(out=FAKE, ldq=2048), INV), (dict(lse=FAKE), INV),
    (dict(out=2 * BIG), INV), (dict(out=2 * BIG + (1 << 20) + 4096), INV), (dict(lse=3 * BIG), INV),
    (dict(out=3 * BIG + 8192), INV), (dict(out=BIG), INV), (dict(lse=4 * BIG + 16), INV),
    (dict(ws=4 * BIG, nbytes=1 << 30, max_kv=1 << 20), INV),
    (dict(ws=FAKE, nbytes=1 << 30, max_kv=1 << 20), INV),
])
def test_attn_refusals(lib, kw, status):
    assert _attn(lib, **kw) == status


def test_null_structs(lib):
    b, c, r = _packed(), _pages(), _rope()
    assert lib.csa2_rotate(None, 8, 128, 1, FAKE, 1024, C.byref(r), 0, BIG, 1024, None, None) == INV
    assert lib.csa2_rotate(C.byref(b), 8, 128, 1, FAKE, 1024, None, 0, BIG, 1024, None, None) == INV
    assert lib.csa2_page_append(None, 2, 128, 1, FAKE, 256, FAKE, 256, None, C.byref(c), None,
                                None) == INV
    assert lib.csa2_page_append(C.byref(b), 2, 128, 1, FAKE, 256, FAKE, 256, None, None, None,
                                None) == INV
    assert lib.csa2_page_attn(None, 8, 2, 128, 1, FAKE, 1024, C.byref(c), 1, 0.1, BIG, None, None, 0,
                              None, None) == INV
    assert lib.csa2_page_attn(C.byref(b), 8, 2, 128, 1, FAKE, 1024, None, 1, 0.1, BIG, None, None, 0,
                              None, None) == INV


def test_workspace(lib):
    # single tokens: two parts to a CTA, whatever the batch
    one = S.csa2_page_attn_workspace(4, 4, 64, 8, 128, 100000)
    assert one == S.csa2_page_attn_workspace(700, 700, 64, 8, 128, 1 << 40) > 0
    # a few longer extends: split; many items: not
    assert S.csa2_page_attn_workspace(40, 1, 64, 8, 128, 100000) >= 2 * 40 * 64 * 129 * 4
    assert S.csa2_page_attn_workspace(20000, 1, 32, 4, 128, 20000) == 0
    assert S.csa2_page_attn_workspace(0, 0, 8, 2, 64, 0) == 0
    for bad in ((-1, 1, 8, 2, 64, 1), (1, -1, 8, 2, 64, 1), (1, 1, 8, 3, 64, 1),
                (1, 1, 8, 2, 80, 1), (1, 1, 8, 2, 64, -1)):
        with pytest.raises(S.Csa2Error):
            S.csa2_page_attn_workspace(*bad)


def _tensors():
    b = dict(num_q=2, num_req=1, cu_q=torch.tensor([0, 2], dtype=torch.int32),
             kv_len=torch.tensor([2]))
    c = dict(k=torch.zeros((3, 2, 16, 64), dtype=torch.uint8),
             v=torch.zeros((3, 2, 16, 64), dtype=torch.uint8), k_scale=torch.ones(3, 2),
             v_scale=torch.ones(3, 2), table=torch.zeros((1, 2), dtype=torch.int32))
    return b, c


def test_host_tensors_are_refused():
    b, c = _tensors()
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    rope = S.rope_freqs(64, device="cpu")
    for call in (lambda: S.rotate(b, x, rope), lambda: S.page_append(b, x, x, c, rope=rope),
                 lambda: S.page_attn(b, x, c, 2)):
        with pytest.raises(S.Csa2Error, match="device tensors"):
            call()


@pytest.mark.parametrize("change,match", [
    (dict(k=torch.zeros((3, 2, 16, 64))), "codes"),
    (dict(v=torch.zeros((3, 2, 32, 64), dtype=torch.uint8)), "expected"),
    (dict(k=torch.zeros((3, 16, 2, 64), dtype=torch.uint8)), "expected"),
    (dict(k=torch.zeros((3, 2, 64, 16), dtype=torch.uint8).transpose(2, 3)), "contiguous"),
    (dict(table=torch.zeros((0, 2), dtype=torch.int32)), "table"),
    (dict(table=torch.zeros((1, 2), dtype=torch.int64)), "table"),
    (dict(table=torch.zeros((2, 1), dtype=torch.int32).t()), None),
    (dict(k_scale=torch.ones(5)), "k_scale"),
    (dict(v_scale=torch.ones((2, 3))), "v_scale"),
    (dict(v_scale=torch.ones((3, 2), dtype=torch.float64)), "v_scale"),
])
def test_cache_tensors(change, match):
    """Shapes, types and strides of a cache, without a device: -1 is the host's number."""
    _, c = _tensors()
    c.update(change)
    if match is None:
        S._cache_arg(c, 1, 2, 64, -1)
    else:
        with pytest.raises(S.Csa2Error, match=match):
            S._cache_arg(c, 1, 2, 64, -1)


def test_cache_views():
    """Codes as float8, K and V page by page in one array, tables with room to spare."""
    _, c = _tensors()
    both = torch.zeros((3, 2, 2, 16, 64), dtype=torch.uint8)
    c.update(k=both[:, 0], v=both[:, 1].view(torch.float8_e4m3fn),
             table=torch.zeros((5, 7), dtype=torch.int32))
    a = S._cache_arg(c, 3, 2, 64, -1)
    assert (a.num_pages, a.page, a.k_stride, a.v_stride, a.table_ld) == (3, 16, 4096, 4096, 7)
    assert a.v - a.k == 2048
    with pytest.raises(S.Csa2Error, match="contiguous"):
        S._cache_arg(dict(c, table=c["table"][:, :4]), 3, 2, 64, -1)


def test_rope_freqs():
    """Scaled frequencies from their definitions."""
    f = S.rope_freqs(32, base=1000.0, device="cpu")
    assert f["amplitude"] == 1.0 and f["freq"].dtype == torch.float64
    for i in range(16):
        assert abs(float(f["freq"][i]) / 1000.0 ** (-i / 16) - 1) < 1e-14
    lin = S.rope_freqs(32, base=1000.0, scaling="linear", factor=4, device="cpu")
    assert torch.equal(lin["freq"], f["freq"] / 4)
    base = S.rope_freqs(32, base=1000.0, scaling="base", factor=4, device="cpu")["freq"]
    assert float(base[0]) == 1 and abs(float(base[-1]) * 4 / float(f["freq"][-1]) - 1) < 1e-12
    ramp = S.rope_freqs(32, base=1000.0, scaling="ramp", factor=4, original=512, low=1, high=8,
                        device="cpu")
    assert abs(ramp["amplitude"] - (0.1 * math.log(4) + 1)) < 1e-15
    for a, b in zip(f["freq"].tolist(), ramp["freq"].tolist()):
        turns = 512 * a / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1) / 7))
        assert abs(b - a * (keep + (1 - keep) / 4)) <= 1e-15 * a
    for bad in (dict(rot=24), dict(rot=0), dict(rot=32, scaling="cubic"), dict(rot=32, factor=0.5),
                dict(rot=32, scaling="ramp"), dict(rot=32, base=-1.0)):
        with pytest.raises(S.Csa2Error):
            S.rope_freqs(device="cpu", **bad)
