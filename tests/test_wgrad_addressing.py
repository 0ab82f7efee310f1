"""Host-side model of the weight gradient kernel's tile walk and global-to-LDS loads (wgrad.hip), checked without a GPU.

- Every tile of an expert belongs to exactly one workgroup, each XCD (workgroup i runs on XCD i % 8) has one contiguous
  range of the walk, and the ranges differ by at most one tile.
- Of the loads that pass the hardware's check (on the VGPR offset alone) every one lies inside the operand, inside a row
  that exists, and at the expert's own blocks; every chunk of every row that exists is loaded once a block.
- Scale groups: each block's scales lie where they are read, in bounds.
"""
import itertools

import pytest

LARGE, SMALL = (256, 256, 8), (128, 128, 4)      # BM, BN, waves
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


def swz(row):
    return (row & 7) ^ ((row >> 3) & 1)


@pytest.mark.parametrize("height,waves", [(LARGE[0], LARGE[2]), (SMALL[0], SMALL[2])])
@pytest.mark.parametrize("rows", [16, 48, 112, 128, 144, 240, 256])
@pytest.mark.parametrize("first,depth,columns,pitch", [(0, 1, 128, 128), (0, 5, 640, 640), (3, 2, 640, 656), (4, 1, 640, 640), (2, 3, 896, 1024)])
def test_loads_of_codes(height, waves, rows, first, depth, columns, pitch):
    rows = min(rows, height)
    end = (rows - 1) * pitch + columns                     # bytes of the operand from this tile's first row on
    got = {}
    for v, wave, lane, kb in itertools.product(range(height // 8 // waves), range(waves), range(64), range(depth)):
        skip = 8 * v * waves
        records = max((rows - skip) * pitch - first * 128, 0) if rows > skip else 0
        lrow = 8 * wave + (lane >> 3)
        voff = lrow * pitch + (((lane & 7) ^ swz(lrow)) << 4)
        if voff + 16 > records:
            assert skip + lrow >= rows or voff >= records, "a chunk of a row that exists is cut"
            if voff >= records:
                continue
        address = skip * pitch + first * 128 + voff + kb * 128
        assert 0 <= address and address + 16 <= end
        row, column = divmod(address, pitch)
        assert row == skip + lrow < rows
        assert (first + kb) * 128 <= column < (first + kb + 1) * 128
        lds = (v * waves + wave) * 1024 + lane * 16          # where the hardware puts it
        assert lds // 128 == row and (lds % 128) // 16 == ((column % 128) // 16) ^ swz(row)
        got.setdefault((kb, row), set()).add(column)
    assert set(got) == set(itertools.product(range(depth), range(rows)))
    assert all(len(c) == 8 for c in got.values())


@pytest.mark.parametrize("height,waves", [(LARGE[0], LARGE[2]), (SMALL[0], SMALL[2])])
@pytest.mark.parametrize("rows", [16, 112, 128, 240])
@pytest.mark.parametrize("first,depth,blocks", [(0, 1, 1), (0, 9, 9), (3, 2, 5), (4, 5, 12)])
def test_loads_of_scales(height, waves, rows, first, depth, blocks):
    rows = min(rows, height)
    held = {}
    for q, u, wave, lane in itertools.product(range(-(-depth // 4)), range(height // 16 // waves), range(waves), range(64)):
        skip = 16 * u * waves
        records = max((rows - skip) * blocks * 4 - first * 4, 0) if rows > skip else 0
        voff = ((16 * wave + (lane >> 2)) * blocks + (lane & 3)) * 4 + q * 16
        place = (16 * (u * waves + wave) + (lane >> 2), 4 * q + (lane & 3))
        if voff >= records:
            held[place] = None
            continue
        index = (skip * blocks * 4 + first * 4 + voff) // 4
        assert 0 <= index < rows * blocks
        held[place] = divmod(index, blocks)
    for row, kb in itertools.product(range(rows), range(depth)):
        assert held[row, kb] == (row, first + kb)


@pytest.mark.parametrize("depth", range(1, 30))
def test_schedule(depth):
    """Steps in order: a stage or scale group is filled only after the barrier that follows its last read, and is complete at a
    barrier before its first."""
    stage, group = {}, {}                                    # what is visible or on its way: buffer -> (content, complete)
    group[0], stage[0] = (0, True), (0, True)                # the first barrier waits for these
    if depth > 1:
        stage[1] = (1, False)
    for kb in range(depth):
        s = kb & 1
        assert stage[s] == (kb, True)
        assert group[(kb >> 2) & 1] == (kb >> 2, True)
        if kb + 1 < depth:
            stage = {k: (c, True) for k, (c, _) in stage.items()}      # the wait for all loads, then the barrier
            group = {k: (c, True) for k, (c, _) in group.items()}
            if kb + 2 < depth:
                stage[s] = (kb + 2, False)
                if (kb + 2) % 4 == 0:
                    q = (kb + 2) >> 2
                    assert group.get(q & 1, (q - 2, True))[0] <= q - 2 and (kb + 1) >> 2 != q - 2
                    group[q & 1] = (q, False)
            assert stage[s ^ 1] == (kb + 1, True)             # its first slice and scales are read here
            assert group[((kb + 1) >> 2) & 1] == ((kb + 1) >> 2, True)
