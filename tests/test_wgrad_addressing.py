"""Host-side model of the weight gradient kernel's tile walk and global-to-LDS loads (wgrad.hip), checked without a GPU.

- Every tile of an expert belongs to exactly one workgroup, each XCD (workgroup i runs on XCD i % 8) has one contiguous
  range of the walk, and the ranges differ by at most one tile.
- Of the loads that pass the hardware's check (on the VGPR offset alone) every one lies inside the operand, inside a row
  that exists, and at the expert's own blocks; every chunk of every row that exists is loaded once a block.
- Scale groups: each block's scales lie where they are read, in bounds.
"""
import itertools

import pytest

CONFIGS = {"large": (256, 8, 128), "whole128": (128, 4, 128), "half128": (128, 4, 64), "whole64": (64, 4, 128), "half64": (64, 4, 64)}      # tile, waves, depth of a step
WALK = 4


@pytest.mark.parametrize("tiles_n", [1, 2, 3, 4, 5, 7, 8, 9, 16])
@pytest.mark.parametrize("tiles_k", [1, 2, 3, 7, 28])
def test_walk(tiles_n, tiles_k):
    tiles = tiles_n * tiles_k
    share = tiles if tiles < 8 else (tiles + 7) // 8 * 8
    seen, by_xcd = [], {}
    for wg in range(share):
        i = wg
        if share >= 8:
            x, per, rest = wg & 7, tiles >> 3, tiles & 7
            if (wg >> 3) >= per + (x < rest):
                continue
            i = x * per + min(x, rest) + (wg >> 3)
            by_xcd.setdefault(x, []).append(i)
        high, inside = divmod(i, WALK * tiles_k)
        height = min(tiles_n - high * WALK, WALK)
        seen.append((high * WALK + inside % height, inside // height))
    assert sorted(seen) == sorted(itertools.product(range(tiles_n), range(tiles_k)))
    for ids in by_xcd.values():
        assert ids == list(range(ids[0], ids[0] + len(ids)))
    if by_xcd:
        assert max(map(len, by_xcd.values())) - min(map(len, by_xcd.values())) <= 1 or len(by_xcd) < 8


def swizzle(row, deep):
    return (row & 7) ^ ((row >> 3) & 1) if deep == 128 else (row >> 2) & 3


@pytest.mark.parametrize("deep", [128, 64])
def test_swizzle_repeats_and_spreads(deep):
    """16 consecutive rows' chunks at one logical place fill the 16 different 16-byte groups of the 64 banks, and the pattern repeats every 16 rows, which is what lets one offset serve every row group."""
    chunks = deep // 16
    for q in range(chunks):
        groups = [((r * deep + ((q ^ swizzle(r, deep)) << 4)) // 16) % 16 for r in range(16)]
        assert sorted(groups) == list(range(16))
    assert all(swizzle(r, deep) == swizzle(r + 16, deep) for r in range(64))


@pytest.mark.parametrize("cfg", sorted(CONFIGS))
@pytest.mark.parametrize("rows", [16, 48, 112, 128, 144, 240, 256])
@pytest.mark.parametrize("first,depth,columns,pitch", [(0, 1, 128, 128), (0, 5, 640, 640), (3, 2, 640, 656), (4, 1, 640, 640), (2, 3, 896, 1024)])
def test_loads_of_codes(cfg, rows, first, depth, columns, pitch):
    height, waves, deep = CONFIGS[cfg]
    rows, per = min(rows, height), 1024 // deep
    end = (rows - 1) * pitch + columns                     # bytes of the operand from this tile's first row on
    got = {}
    for v, wave, lane, h in itertools.product(range(height // per // waves), range(waves), range(64), range(depth * 128 // deep)):
        skip, records = per * v * waves, rows * pitch - first * 128
        lrow = per * wave + lane // (deep // 16)
        voff = lrow * pitch + (((lane & (deep // 16 - 1)) ^ swizzle(lrow, deep)) << 4) + skip * pitch
        if voff >= records:
            assert skip + lrow >= rows
            continue
        assert voff + 16 <= records
        address = first * 128 + voff + h * deep
        assert 0 <= address and address + 16 <= end
        row, column = divmod(address, pitch)
        assert row == skip + lrow < rows
        assert first * 128 + h * deep <= column < first * 128 + (h + 1) * deep
        lds = (v * waves + wave) * 1024 + lane * 16          # where the hardware puts it
        assert lds // deep == row and (lds % deep) // 16 == ((column % deep) // 16) ^ swizzle(row, deep)
        got.setdefault((h, row), set()).add(column)
    assert set(got) == set(itertools.product(range(depth * 128 // deep), range(rows)))
    assert all(len(c) == deep // 16 for c in got.values())


@pytest.mark.parametrize("cfg", sorted(CONFIGS))
@pytest.mark.parametrize("rows", [16, 112, 128, 240])
@pytest.mark.parametrize("first,depth,blocks", [(0, 1, 1), (0, 9, 9), (3, 2, 5), (4, 5, 12)])
def test_loads_of_scales(cfg, rows, first, depth, blocks):
    height, waves, _ = CONFIGS[cfg]
    rows = min(rows, height)
    held = {}
    for q, u, wave, lane in itertools.product(range(-(-depth // 4)), range(height // 16 // waves), range(waves), range(64)):
        records = rows * blocks * 4 - first * 4
        voff = ((16 * wave + (lane >> 2)) * blocks + (lane & 3)) * 4 + q * 16 + 16 * u * waves * blocks * 4
        place = (16 * (u * waves + wave) + (lane >> 2), 4 * q + (lane & 3))
        if voff >= records:
            held[place] = None
            continue
        index = (first * 4 + voff) // 4
        assert 0 <= index < rows * blocks
        held[place] = divmod(index, blocks)
    for row, kb in itertools.product(range(rows), range(depth)):
        assert held[row, kb] == (row, first + kb)


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("depth", range(1, 20))
def test_schedule(depth, parts):
    """Steps in order, `parts` a block: a stage or scale group is filled only after the barrier that follows its last read, and
    is complete at a barrier before its first."""
    steps = depth * parts
    stage, group = {0: (0, True)}, {0: (0, True)}            # buffer -> (content, complete); the first barrier waits for these
    if steps > 1:
        stage[1] = (1, False)
    last_read = {}                                           # group -> step in whose second half its last scales are read
    for h in range(steps):
        s = h & 1
        assert stage[s] == (h, True)
        assert group[(h // parts >> 2) & 1] == (h // parts >> 2, True)
        if h + 1 < steps:
            stage = {k: (c, True) for k, (c, _) in stage.items()}      # the wait for all loads, then the barrier
            group = {k: (c, True) for k, (c, _) in group.items()}
            if h + 2 < steps:
                stage[s] = (h + 2, False)
                if (h + 2) % (4 * parts) == 0:
                    q = (h + 2) // (4 * parts)
                    assert last_read.get(q - 2, -1) < h       # a whole barrier lies between
                    group[q & 1] = (q, False)
            assert stage[s ^ 1] == (h + 1, True)              # its first slice is read here
            if parts == 1 or s == 1:
                q = (h + 1) // parts >> 2
                assert group[q & 1] == (q, True)
                last_read[q] = h
