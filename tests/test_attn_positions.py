"""The attention kernels look up to some thousand keys ahead of a context's end in 32 bits: tables
that could hold contexts within 2^16 of 2^31 positions are refused (CPU: nothing is launched)."""
import pytest

from gated_delta_rule_44_gb300 import binding as B
from test_attn8_refusals import cache8
from test_attn8_refusals import call as call8
from test_attn_refusals import cache, call, paged_args, prepare_args

MOST = 2 ** 31 - 2 ** 16


@pytest.mark.parametrize("make", [paged_args, prepare_args])
@pytest.mark.parametrize("page", [16, 48, 1 << 20])
def test_tables_near_2_31(make, page):
    # An empty table: the check behind this one.
    for pages in (MOST // page, MOST // page + 1, (2 ** 31 - 1) // page):
        refused = pages * page > MOST
        rc, msg = call(make(c=cache(2, 64, page=page, max_pages=pages, block_table=None)))
        assert (rc == B.GDN_ERR_UNSUPPORTED and "32 bits" in msg) if refused else msg == "block_table is NULL"
        rc, msg = call8(make, cache8(page=page, max_pages=pages, block_table=None))
        assert (rc == B.GDN_ERR_UNSUPPORTED and "32 bits" in msg) if refused else msg == "block_table is NULL"


def test_workspace_of_tables_near_2_31():
    L = B.lib()
    sizes = (4, 2, 4, 2, 64, 1, B.GDN_DTYPE_F32)
    assert L.gdn_attn8_paged_workspace_bytes(*sizes, MOST // 64 + 1, 64) == 0
    sizes = (1, 1, 64, 1, 64, 1, B.GDN_DTYPE_F32)      # widened: as large as the table
    assert L.gdn_attn8_paged_workspace_bytes(*sizes, MOST // 64, 64) >= MOST * 2 * 64 * 4
