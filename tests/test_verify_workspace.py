"""Workspaces of fk_verify, on the CPU: one for the largest step does for all
smaller ones."""
import itertools

import pytest

import exact_lloyd_means_amd as fk

size = fk.lib.fk_verify_workspace_bytes


def pieces(rows, V, greedy):
    """How many pieces a call cuts each row into: by the card's 1024 workgroups of
    1024 to 8192 elements (four waves of one each where it samples), in whole
    16-byte accesses."""
    c = max(min(-(-1024 // rows), -(-V // 1024)), -(-V // 8192)) * (1 if greedy else 4)
    each = -(-(-(-V // c)) // 8) * 8
    return -(-V // each)


@pytest.mark.parametrize("V", [1, 8, 9, 500, 1024, 1025, 32000, 128000, 150001, 1 << 20])
def test_more_requests_need_no_less(V):
    last = 0
    for B in range(1, 2100):
        n = size(B, 4 * B, V)
        assert n >= last, B
        assert n >= max(B * pieces(B, V, False) * 16 + B * 4, 4 * B * pieces(4 * B, V, True) * 8)
        last = n


def test_each_size_alone():
    rng = list(range(1, 40)) + [63, 64, 65, 511, 512, 513, 1023, 1024, 1025, 5000]
    for B, V in itertools.product((1, 7, 64, 1000), (3, 1000, 40000)):
        t = [size(B, T, V) for T in rng]
        assert t == sorted(t)
    for B, T in ((1, 1), (3, 9), (64, 384), (1000, 1000)):
        v = [size(B, T, V) for V in [*range(1, 3000), *range(3000, 200000, 997)]]
        assert v == sorted(v)


def test_not_much_more_than_a_call_takes():
    for B, V in itertools.product((1, 2, 11, 12, 64, 300, 3000), (32000, 128000)):
        takes = max(B * pieces(B, V, False) * 16 + B * 4, B * pieces(B, V, True) * 8)
        # the card's 1024 pieces, once more
        assert size(B, B, V) <= takes + 1024 * 4 * 16
