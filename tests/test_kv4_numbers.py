"""Numbers that fk_kv4_attention's arguments cannot hold are ValueErrors, like
everything else that the binding refuses."""
import pytest

import exact_lloyd_means_amd as fk
from test_kv4_checks import good


@pytest.mark.parametrize("kw", [dict(max_q=1 << 31), dict(max_q=1.5), dict(max_q=None), dict(window=1 << 31),
                                dict(window=0.5), dict(scale="1")])
def test_numbers_out_of_range(kw):
    t = good()
    with pytest.raises(ValueError, match="max_q, window or scale"):
        fk.fk_kv4_attention(t["q"], t["cu"], t["seq"], t["table"], t["codebook"], t["codes"], t["scales"], t["out"],
                            **{"max_q": 2, **kw})
