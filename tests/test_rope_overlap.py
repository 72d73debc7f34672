"""Rows that fk_rope writes share no element, on the CPU: calls that are refused
before anything runs, or for another reason that is checked behind this one."""
import itertools
import struct

import pytest

import exact_lloyd_means_amd as fk

FAKE = 0x10000
ROPE, ROWS = struct.Struct("@qiiiiifPP"), struct.Struct("@PPqqqqii")
D = 8


def refused(*sets):
    """The message for sets of (y, tokens' stride, heads' stride, heads); the last row
    is broken in a way that is looked at afterwards, so that nothing is launched."""
    T = sets[0][0]
    packed = b"".join(ROWS.pack(FAKE, y, 64, 64, yt, yh, H, i == len(sets) - 1) for i, (_, y, yt, yh, H) in enumerate(sets))
    assert fk.lib.fk_rope(ROPE.pack(T, D, D, fk.FK_F32, 0, 0, 1.0, FAKE, FAKE), len(sets), packed, None) == fk.FK_EINVAL
    return fk.lib.fk_last_error().decode()


def share(T, yt, H, yh):
    seen = set()
    for t, h in itertools.product(range(T), range(H)):
        row = set(range(t * yt + h * yh, t * yt + h * yh + D))
        if seen & row:
            return True
        seen |= row
    return False


def test_strides_of_all_kinds():
    # against the rows laid out one by one: interleaved, in either order, with gaps, sharing a single element
    count = [0, 0]
    for T, H in ((1, 1), (1, 4), (4, 1), (2, 2), (3, 2), (2, 5), (4, 3), (7, 6)):
        for yt, yh in itertools.product([0, 1, 7, 8, 9, 15, 16, 17, 20, 24, 25, 31, 32, 33, 40, 48, 56, 63, 64, 72], repeat=2):
            message = refused((T, 2 * FAKE, yt, yh, H))
            want = share(T, yt, H, yh)
            assert ("overlap" in message) == want, (T, yt, H, yh, message)
            assert want or "reserved" in message
            count[want] += 1
    assert min(count) > 500


@pytest.mark.parametrize("T,yt,H,yh,overlap", [
    (2, D, 2, D, True),                                # (0, 1) and (1, 0) are one row
    (1 << 24, 40 * D, 40, D, False), (1 << 24, D, 40, D << 24, False), (1 << 24, D, 40, (D << 24) - 1, True),
    (1 << 24, 65536 * D - 1, 65536, D, True),
    (1 << 24, 2 ** 62, 65536, 2 ** 63 - 1, True),      # four tokens are 2^64, two heads 2^64 - 2
    (2, 2 ** 62, 65536, 2 ** 63 - 1, False), (3, 2 ** 63 - 1, 65536, 2 ** 63 - 1, True)])
def test_the_largest(T, yt, H, yh, overlap):
    assert ("overlap" in refused((T, 2 * FAKE, yt, yh, H))) == overlap


def test_two_sets():
    assert "same rows" in refused((4, 2 * FAKE, 16, 8, 2), (4, 2 * FAKE, 16, 8, 2))
    assert "overlap" in refused((4, 2 * FAKE, 8, 8, 2), (4, 3 * FAKE, 16, 8, 2))
    # queries and keys of one projection lie between each other
    assert "reserved" in refused((4, 2 * FAKE, 32, 8, 2), (4, 2 * FAKE + 64, 32, 8, 2))
