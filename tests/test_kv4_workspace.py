"""Size of the attention's workspace, on the CPU: two places of partial sums
(head_dim + 2 fp32 numbers a row) for every wave that runs, and no more."""
import struct

import pytest

import exact_lloyd_means_amd as fk

CACHE = struct.Struct("@PPPqiiii")


def size(B, T, Hq, H, D, max_q):
    c = CACHE.pack(0, 0, 0, 1000, 64, H, D, fk.FK_BF16)
    return fk.lib.fk_kv4_attn_workspace_bytes(c, B, T, Hq, max_q)


# heads x row tiles, rows of a tile, and waves of a workgroup: eight where the
# tile is one block of 16 rows of at most 128 dimensions, else four
@pytest.mark.parametrize("B,T,Hq,H,D,max_q,tiles,rows,waves", [
    (64, 64, 32, 8, 128, 1, 8, 4, 8), (64, 64, 32, 8, 64, 1, 8, 4, 8),
    (64, 64, 32, 8, 256, 1, 8, 4, 4),                 # 256 dimensions
    (64, 64, 64, 2, 128, 1, 2, 32, 4),                # two blocks of rows
    (1, 512, 32, 8, 128, 512, 8 * 43, 48, 4), (64, 575, 32, 8, 128, 512, 8 * 43, 48, 4),
    (16, 80, 16, 1, 256, 5, 5, 16, 4)])
def test_partial_sums_of_the_waves_that_run(B, T, Hq, H, D, max_q, tiles, rows, waves):
    # workgroups of a tile: the fewest rounds of 512 of which 88 % are full, else the fullest of eight
    full = [(r * 512 // tiles) * tiles / (r * 512) for r in range(1, 9)]
    r = next((i for i, f in enumerate(full) if f >= 0.88), full.index(max(full))) + 1
    parts = tiles * (r * 512 // tiles) * waves * 2 * rows
    prefix = 4 * (tiles // H) * (B + 1)
    got = size(B, T, Hq, H, D, max_q)
    assert 0 <= got - parts * (D + 2) * 4 - prefix < 3 * 256


def test_a_prompt_of_one_request():
    assert size(1, 512, 32, 8, 128, 512) < 280 << 20      # 32 / 8 heads of 128
