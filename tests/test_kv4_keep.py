"""What KV4Cache.fork and release keep of a row, as the kernels get it: lengths
that 32 bits do not hold are all of a row, on the CPU."""
import pytest
import torch

import exact_lloyd_means_amd as fk

MOST = 2 ** 31 - 1


def cache(monkeypatch):
    c, calls = fk.KV4Cache(8, 32, 1, 64, torch.zeros(2, 1, 16).half(), 4, 64, device="cpu"), []

    def take(rows, sources, keep):
        calls.append(keep)
        return torch.empty(len(rows), 3, dtype=torch.int32)
    monkeypatch.setattr(c, "_fork", take)
    return c, calls


@pytest.mark.parametrize("dtype,given,want", [
    (torch.int64, [2 ** 31, 2 ** 40], [MOST, MOST]), (torch.int64, [2 ** 63 - 1, MOST], [MOST, MOST]),
    (torch.int64, [2 ** 32, 2 ** 32 + 5], [MOST, MOST]), (torch.int64, [-2 ** 63, -1], [0, 0]), (torch.int64, [-2 ** 40, 70], [0, 70]),
    (torch.int32, [MOST, -2 ** 31], [MOST, 0]), (torch.int32, [MOST - 1, 3], [MOST - 1, 3]), (torch.int64, [MOST - 1, 16777217], [MOST - 1, 16777217]),
    (torch.uint8, [200, 0], [200, 0]), (torch.int16, [-5, 32767], [0, 32767]), (torch.float32, [2.0 ** 31, float("inf")], [MOST, MOST])])
def test_a_tensor(monkeypatch, dtype, given, want):
    c, calls = cache(monkeypatch)
    keep = torch.tensor(given, dtype=dtype)
    c.fork([0, 1], [2, 3], keep=keep)
    c.release([0, 1], keep=keep)
    for got in calls:
        assert got.dtype is torch.int32 and got.is_contiguous() and got.tolist() == want
    assert len(calls) == 2


@pytest.mark.parametrize("given,want", [(2 ** 31, MOST), (2 ** 63, MOST), (MOST, MOST), (-1, 0), (0, 0), (64, 64)])
def test_a_number(monkeypatch, given, want):
    c, calls = cache(monkeypatch)
    c.fork([0, 1], [2, 3], keep=given)
    c.release([0, 1], keep=given)
    assert [x.tolist() for x in calls] == [[want] * 2] * 2


def test_none(monkeypatch):
    # fork: all of the source; release: nothing
    c, calls = cache(monkeypatch)
    c.fork([0, 1], [2, 3])
    c.release([0, 1])
    assert [x.tolist() for x in calls] == [[MOST] * 2, [0, 0]]


def test_one_for_all_rows(monkeypatch):
    c, calls = cache(monkeypatch)
    c.release([0, 1, 2], keep=torch.tensor([2 ** 35]))
    assert calls[0].tolist() == [MOST] * 3
