"""Row numbers of KV4Cache.fork and release in integers of few bits, on the CPU:
they name the same rows as in 64 bits where the table has more rows than the
type has numbers."""
import pytest
import torch

import exact_lloyd_means_amd as fk


@pytest.mark.parametrize("R", [4, 100, 200, 256, 300, 40000])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.int8, torch.int16, torch.int32, torch.int64])
def test_rows(monkeypatch, R, dtype):
    cache = fk.KV4Cache(8, 32, 1, 64, torch.zeros(2, 1, 16).half(), R, 32, device="cpu")
    calls = []

    def take(rows, sources, keep):
        calls.append((rows, sources))
        return torch.empty(len(rows), 3, dtype=torch.int32)
    monkeypatch.setattr(cache, "_fork", take)
    ends = torch.iinfo(dtype)
    given = [x for x in (0, 3, 100, 127, 128, 255, -1, -4, -100, -128, 32767, -32768, 2 ** 31 - 1) if ends.min <= x <= ends.max]
    want = [x if 0 <= x < R else x + R if -R <= x < 0 else R for x in given]      # R: none
    rows = torch.tensor(given, dtype=dtype)
    cache.release(rows)
    cache.fork(rows, rows)
    for x in (calls[0][0], *calls[1]):
        assert x.dtype is torch.int32 and x.tolist() == want
