"""Refusals of the dense-cache calls that the host can see (no GPU needed):
nothing is launched, a status comes back."""
import ctypes as C

import pytest
import torch

import sparse_attention_prefill_gb300 as S
from sparse_attention_prefill_gb300 import build

FAKE = 1 << 20           # never read: each case is refused before a launch
INV, UNS = S.ERR_INVALID_ARG, S.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return S.load(build.build())


def _packed(**kw):
    d = dict(num_q=10, num_req=2, cu_q=FAKE, kv_start=FAKE, kv_len=FAKE)
    d.update(kw)
    return S.CPacked(*[d[k] for k in ("num_q", "num_req", "cu_q", "kv_start", "kv_len")])


def _prompt(lib, b=None, h=8, kv=2, dim=128, dt=S.DT_BF16, q=FAKE, ldq=1024, k=FAKE, ldk=256,
            v=FAKE, ldv=256, rows=100, scale=0.1, out=FAKE):
    b = b or _packed()
    return lib.csa2_prompt_attn(C.byref(b), h, kv, dim, dt, q, ldq, k, ldk, v, ldv, rows, scale,
                                out, None, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(b=_packed(num_q=-1)), INV), (dict(b=_packed(num_req=-1)), INV),
    (dict(b=_packed(cu_q=None)), INV), (dict(b=_packed(kv_start=None)), INV),
    (dict(b=_packed(kv_len=None)), INV), (dict(b=_packed(num_q=0)), S.OK),
    (dict(b=_packed(num_req=0)), S.OK), (dict(h=0), INV), (dict(kv=0), INV), (dict(h=9), INV),
    (dict(dim=96, ldq=768), UNS), (dict(dt=3), UNS), (dict(scale=0.0), INV),
    (dict(scale=-1.0), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(out=None), INV),
    (dict(q=FAKE + 2), UNS), (dict(k=FAKE + 8), UNS), (dict(out=FAKE + 4), UNS),
    (dict(ldq=1020), INV), (dict(ldq=1028), UNS), (dict(ldk=0), INV), (dict(ldv=260), UNS),
    (dict(rows=-1), INV), (dict(rows=1 << 31), UNS), (dict(h=258, kv=2, ldq=258 * 128), UNS),
    (dict(h=2048, kv=2048, ldq=1 << 18, ldk=1 << 18, ldv=1 << 18), UNS),
])
def test_prompt_refusals(lib, kw, status):
    assert _prompt(lib, **kw) == status


def _prefix(lib, g=None, ws=FAKE, nbytes=1 << 40, max_kv=100, **kw):
    d = dict(b=_packed(), h=8, kv=2, dim=128, dt=S.DT_F16, q=FAKE, out=FAKE, scale=0.1)
    d.update(kw)
    return lib.csa2_prefix_attn(C.byref(d["b"]), None if g is None else C.byref(g), d["h"],
                                d["kv"], d["dim"], d["dt"], d["q"], 1024, FAKE, 256, FAKE, 256,
                                100, max_kv, d["scale"], d["out"], None, ws, nbytes, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=S.CPrefixGroups(-1, 0, FAKE, FAKE, FAKE, 10)), INV),
    (dict(g=S.CPrefixGroups(1, 0, None, FAKE, FAKE, 10)), INV),
    (dict(g=S.CPrefixGroups(1, 0, FAKE, None, FAKE, 10)), INV),
    (dict(g=S.CPrefixGroups(1, 0, FAKE, FAKE, None, 10)), INV),
    (dict(g=S.CPrefixGroups(1, 0, FAKE, FAKE, FAKE, -1)), INV),
    (dict(ws=None), INV), (dict(nbytes=16), INV), (dict(ws=FAKE + 16), UNS), (dict(max_kv=-1), INV),
    (dict(q=None), INV), (dict(out=FAKE + 2), UNS), (dict(dim=32), UNS), (dict(scale=0.0), INV),
    (dict(b=_packed(num_q=0)), S.OK),
])
def test_prefix_refusals(lib, kw, status):
    assert _prefix(lib, **kw) == status


def test_prefix_workspace(lib):
    need = S.csa2_prefix_attn_workspace(64, 64, 1, 64, 8, 128, 8192, 700)
    # at least one part each for the prefix and the requests' own rows
    assert need >= 2 * 64 * 64 * 129 * 4
    assert S.csa2_prefix_attn_workspace(0, 0, 0, 8, 2, 64, 0, 0) >= 0
    for bad in ((-1, 1, 1, 8, 2, 64, 1, 1), (1, 1, 1, 8, 3, 64, 1, 1), (1, 1, 1, 8, 2, 80, 1, 1),
                (1, 1, 1, 8, 2, 64, -1, 1), (1, 1, 1, 8, 2, 64, 1, -1)):
        with pytest.raises(S.Csa2Error):
            S.csa2_prefix_attn_workspace(*bad)


def _mass(lib, b=None, h=8, kv=2, dim=128, q=FAKE, k=FAKE, rows=100, lse=FAKE, max_kv=100,
          scale=0.1, mass=FAKE):
    b = b or _packed()
    return lib.csa2_attn_mass(C.byref(b), h, kv, dim, S.DT_BF16, q, 1024, k, 256, rows, lse,
                              max_kv, scale, None, mass, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(lse=None), INV), (dict(mass=None), INV),
    (dict(max_kv=-1), INV), (dict(rows=0), S.OK), (dict(b=_packed(num_req=0)), S.OK),
    (dict(b=_packed(num_req=8193)), UNS), (dict(mass=FAKE + 2), UNS), (dict(h=7), INV),
    (dict(dim=256), UNS), (dict(b=_packed(num_q=0, cu_q=None)), INV), (dict(k=FAKE + 4), UNS),
])
def test_mass_refusals(lib, kw, status):
    assert _mass(lib, **kw) == status


def _sel(lib, r=2, h=2, start=FAKE, lens=FAKE, mass=FAKE, rows=100, keep=10, sink=1, recent=2,
         idx=FAKE, new=FAKE):
    return lib.csa2_evict_select(r, h, start, lens, mass, rows, keep, sink, recent, idx, new,
                                 None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(r=-1), INV), (dict(r=0), S.OK), (dict(h=0), INV), (dict(keep=0), INV),
    (dict(sink=-1), INV), (dict(recent=-1), INV), (dict(sink=6, recent=5), INV),
    (dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), INV), (dict(mass=None), INV),
    (dict(start=None), INV), (dict(lens=None), INV), (dict(idx=None), INV), (dict(new=None), INV),
    (dict(rows=-1), INV), (dict(rows=1 << 31), UNS), (dict(mass=FAKE + 1), UNS),
])
def test_select_refusals(lib, kw, status):
    assert _sel(lib, **kw) == status


def _rows(lib, r=2, h=2, idx=FAKE, keep=4, new=FAKE, s0=FAKE, d0=FAKE, n=1, **buf):
    d = dict(src=FAKE, dst=2 * FAKE, src_rows=10, dst_rows=10, src_row_stride=64,
             src_head_stride=32, dst_row_stride=64, dst_head_stride=32, elem_bytes=32)
    d.update(buf)
    one = S.CEvictBuf(*[d[k] for k, _ in S.CEvictBuf._fields_])
    arr = (S.CEvictBuf * 16)(*[one] * 16)
    return lib.csa2_evict_rows(r, h, idx, keep, new, s0, d0, n, arr, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(r=-1), INV), (dict(r=0), S.OK), (dict(n=0), S.OK), (dict(n=-1), INV), (dict(n=9), UNS),
    (dict(h=0), INV), (dict(keep=0), INV), (dict(idx=None), INV), (dict(new=None), INV),
    (dict(s0=None), INV), (dict(d0=None), INV), (dict(src=None), INV), (dict(dst=None), INV),
    (dict(src_rows=-1), INV), (dict(dst_row_stride=-64), INV), (dict(elem_bytes=30), UNS),
    (dict(src=FAKE + 2), UNS), (dict(src_head_stride=33), UNS), (dict(elem_bytes=1 << 25), UNS),
])
def test_rows_refusals(lib, kw, status):
    assert _rows(lib, **kw) == status


def test_binding_refuses_host_tensors_and_wrong_types(lib):
    z = torch.zeros
    b = dict(num_q=4, num_req=1, cu_q=z(2, dtype=torch.int32), kv_start=z(1, dtype=torch.int64),
             kv_len=z(1, dtype=torch.int64))
    q, k = z((4, 4, 64), dtype=torch.bfloat16), z((9, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: S.prompt_attn(b, q, k, k), lambda: S.prefix_attn(b, None, q, k, k, 9),
                 lambda: S.attn_mass(b, q, k, z((4, 4)), 9),
                 lambda: S.evict_select(b["kv_start"], b["kv_len"], z((2, 9)), 4),
                 lambda: S.evict_rows(z((1, 2, 4), dtype=torch.int32), b["kv_len"],
                                      b["kv_start"], b["kv_start"], [(k, k)]),
                 lambda: S.prompt_attn(dict(b, cu_q=z(2)), q, k, k),
                 lambda: S.prompt_attn(dict(b, kv_len=z(0, dtype=torch.int64)), q, k, k)):
        with pytest.raises(S.Csa2Error):
            call()
