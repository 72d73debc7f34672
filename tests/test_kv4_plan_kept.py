"""What fk_kv_plan_kept refuses, on the CPU: what fk_kv_plan refuses, and a
misaligned kept_lens."""
import pytest
import torch

import exact_lloyd_means_amd as fk
from test_kv4_checks import FAKE, PLAN


def call(kept=FAKE, **kw):
    a = {**PLAN, **kw}
    ws = [a.pop("ws"), a.pop("ws_bytes")]
    return fk.lib.fk_kv_plan_kept(*a.values(), kept, *ws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(kept=FAKE + 2), fk.FK_EINVAL), (dict(B=0), fk.FK_EINVAL), (dict(page_size=31), fk.FK_EUNSUPPORTED),
    (dict(ctx=None), fk.FK_EINVAL), (dict(status=None), fk.FK_EINVAL), (dict(ws=None), fk.FK_EWORKSPACE),
    (dict(ws_bytes=8), fk.FK_EWORKSPACE)])
def test_arguments(kw, status):
    assert call(**kw) == status


def test_binding():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    args = [i(3), i(3), 32, i(9), i(1), i(3, 4), i(3), i(4), i(7), i(7), i(1), i(4)]
    with pytest.raises(ValueError, match="kept_lens must have shape"):
        fk.fk_kv_plan(*args, kept_lens=i(4))
    with pytest.raises(ValueError, match="on the GPU"):
        fk.fk_kv_plan(*args, kept_lens=i(3))
