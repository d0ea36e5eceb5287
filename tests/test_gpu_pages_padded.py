"""Batches on 8-bit pages that are padded with requests without query rows, as a captured
graph's are: nothing of these is looked at, whichever way the call goes."""
import pytest
import torch

import sparse_attention_prefill_gb300 as S
from tests import page_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
HF = torch.float16
LENGTHS = (-5, 1 << 40, 0, 77, -(1 << 62))

# new rows, cache rows, heads, kv heads: single tokens, wide groups, short and long extends
KINDS = [([1] * 40, 8, 1), ([1] * 40, 40, 1), ([3] * 40, 8, 2), ([90] * 40, 4, 2)]


@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("share", [True, False])
def test_requests_without_rows_are_not_judged(kind, share):
    """Seventy of them among forty others, so that whoever looks for a request's neighbours
    comes by: the others get their results, and there is no flag."""
    new, heads, kv = KINDS[kind]
    rows = [n + (37 * i) % 500 for i, n in enumerate(new)]
    dim, page = 64, 16
    c = R.make_cache(rows, kv, dim, page, seed=kind)
    at = [i * 11 // 4 for i in range(len(new))]           # where the others are among 110
    count = 110
    n2, m2 = [0] * count, [LENGTHS[i % len(LENGTHS)] for i in range(count)]
    table = torch.full((count, c["table"].shape[1]), -3, dtype=torch.int32, device=DEV)
    for i, r in enumerate(at):
        n2[r], m2[r] = new[i], rows[i]
        table[r] = c["table"][i]
    b, cu = R.batch(n2, m2, DEV)
    q = torch.randn((b["num_q"], heads, dim), device=DEV).to(HF)
    ws = None if share else torch.empty(0, dtype=torch.uint8, device=DEV)
    d = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = S.page_attn(b, q, dict(c, table=table), max_kv=600, workspace=ws, d_err=d)
    assert int(d.item()) == 0
    for i, r in enumerate(at):
        lo, hi = cu[r], cu[r + 1]
        ref = R.attend(q[lo:hi], R.held(c, i, rows[i], "k"), R.held(c, i, rows[i], "v"),
                       dim ** -0.5, rows[i] - new[i] + torch.arange(new[i], device=DEV))
        R.check_attention(out[lo:hi], lse[lo:hi], ref, HF, rows[i], float(c["v_scale"].max()))
    # the other calls of a step, too
    k = torch.randn((b["num_q"], kv, dim), device=DEV).to(HF)
    S.rotate(b, q, S.rope_freqs(dim), d_err=d)
    S.page_append(b, k, k, dict(c, table=table), rope=S.rope_freqs(dim), d_err=d)
    assert int(d.item()) == 0
    # one with rows is
    bad = dict(b, kv_len=b["kv_len"].clone())
    bad["kv_len"][at[7]] = 1 << 40
    S.page_attn(bad, q, dict(c, table=table), max_kv=600, workspace=ws, d_err=d)
    assert int(d.item()) == S.DERR_RANGE_ROW
