"""Refusals of the dense-cache calls that concern several arguments at once
(no GPU needed: every call here is refused before a launch)."""
import pytest

import sparse_attention_prefill_gb300 as S
from sparse_attention_prefill_gb300 import build

AT = 1 << 30             # addresses far apart; never read
INV = S.ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    return S.load(build.build())


# 3 requests, 2 heads, 100 rows, 10 kept: kv_start, kv_len and new_len are 24
# bytes, mass is 800, idx 240
@pytest.mark.parametrize("kw", [
    dict(new=2 * AT + 8), dict(new=2 * AT - 8), dict(new=AT), dict(new=AT + 16), dict(new=3 * AT),
    dict(new=3 * AT + 792), dict(idx=AT), dict(idx=AT - 236), dict(idx=2 * AT + 20),
    dict(idx=3 * AT + 796), dict(idx=5 * AT + 20), dict(idx=5 * AT - 236), dict(idx=2 * AT, new=2 * AT)])
def test_select_outputs_that_overlap_are_refused(lib, kw):
    d = dict(idx=4 * AT, new=5 * AT)
    d.update(kw)
    assert lib.csa2_evict_select(3, 2, AT, 2 * AT, 3 * AT, 100, 10, 1, 2, d["idx"], d["new"], None,
                                 None) == INV
