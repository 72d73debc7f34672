"""Row tiles of a call are counted rounded up: a grid that HIP would not launch
is refused before it is tried."""
import pytest

import exact_lloyd_means_amd as fk
from test_kv4_checks import attn, cache, call


@pytest.mark.parametrize("T,B", [(64 * 33 + 1, (1 << 20) - 34), (64 * 40, (1 << 20) - 40)])
def test_as_many_workgroups_as_a_grid_has(T, B):
    # 16 heads x 2^20 tiles of 64 rows: 2^24 workgroups of 256 threads
    a = attn(B=B, T=T, Hq=16, max_q=T, max_pages=1, q_token=16 * 256, q_head=256)
    assert call(c=cache(heads=16, dim=256), a=a) == fk.FK_EUNSUPPORTED
    assert b"2^24" in fk.lib.fk_last_error()
