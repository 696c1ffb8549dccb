"""Host model of the gated linear scan's buffer accesses: which elements of a tensor [T][D] (token stride s1) a
workgroup of 64 channels reads or writes, tile by tile, and that nothing else is touched.

A tile's rows are addressed from its first element: the lane's offset and the row's are added and an access
behind the descriptor's range is dropped, as `Place`, `Rows::load` and `store_row` of the kernels do. Offsets are
formed in 32 bits.
"""
import numpy as np
import pytest

TILE, COLS, WAVES, ELEMS, NOWHERE, WRAP = 128, 64, 8, 16, 0x80000000, 2**32


def accesses(T, D, s1, eb, V, k, c0):
    """(tokens, channels) inside the range of tile k, and whether any piece straddles its end; a single
    token's rows are taken to be 64 elements apart."""
    pitch = (s1 if T > 1 else COLS) * eb
    last = min(T - k * TILE, TILE) - 1
    limit = last * pitch + min(D - c0, COLS) * eb
    assert pitch < WRAP and 0 < limit < 2**31
    lanes, L = COLS // V, ELEMS // V
    groups = 64 // lanes
    got, torn = [], False
    for wave in range(WAVES):
        for lane in range(64):
            run, ch = wave * groups + lane // lanes, lane % lanes * V
            ok = c0 + ch < D
            off = run * L * pitch + ch * eb if ok else NOWHERE
            assert not ok or off < 2**31
            for j in range(L):
                at = off + j * pitch
                assert at < WRAP
                if at < limit:
                    torn |= at + V * eb > limit
                    got.append((run * L + j, ch, at))
    return got, torn, last


@pytest.mark.parametrize("eb", [1, 2, 4])
@pytest.mark.parametrize("V", [1, 2])
@pytest.mark.parametrize("T", [1, 5, 127, 128, 129, 300])
@pytest.mark.parametrize("D,pad", [(1, 0), (2, 0), (63, 0), (64, 0), (66, 2), (130, 0), (200, 1000)])
def test_rows_that_do_not_exist_are_dropped(T, D, pad, V, eb):
    """Outputs (rows apart): every element once, nothing else."""
    if D % V:
        pytest.skip("two channels per lane need an even width")
    s1 = D + pad
    seen = np.zeros((T, D), dtype=int)
    for k in range(-(-T // TILE)):
        for c0 in range(0, D, COLS):
            got, torn, last = accesses(T, D, s1, eb, V, k, c0)
            assert not torn
            for row, ch, at in got:
                assert row <= last and at == (row * s1 + ch) * eb
                seen[k * TILE + row, c0 + ch:c0 + ch + V] += 1
    assert (seen == 1).all()


@pytest.mark.parametrize("s1", [0, 1, 7, 40])
@pytest.mark.parametrize("T", [2, 129, 200])
def test_overlapping_inputs_stay_inside(T, s1):
    """Inputs may repeat or overlap rows: what a row behind the last reads in the range is the tensor's own memory."""
    D, eb = 64, 2
    for k in range(-(-T // TILE)):
        got, torn, last = accesses(T, D, s1, eb, 1, k, 0)
        assert not torn
        assert {r for r, _, _ in got} >= set(range(last + 1))
        assert max(at for _, _, at in got) + eb <= (last * s1 + D) * eb


def test_farthest_rows_do_not_wrap():
    """Token strides just below the limit of 2^22 elements, float32."""
    got, torn, last = accesses(TILE, COLS, 2**22 - 2, 4, 2, 0, 0)
    assert not torn and last == TILE - 1 and len(got) == TILE * COLS // 2


@pytest.mark.parametrize("eb", [1, 2, 4])
@pytest.mark.parametrize("V", [1, 2])
def test_a_single_token_of_the_widest_rows(V, eb):
    """2^24 channels: with the width as stride the offsets of float32 rows from the 64th on would come round to the first."""
    for c0 in (0, 2**24 - COLS):
        got, torn, _ = accesses(1, 2**24, 0, eb, V, 0, c0)
        assert not torn and sorted(at for _, _, at in got) == [i * eb for i in range(0, COLS, V)]


def test_a_planted_mistake_is_seen():
    """A range of one row more lets the row behind the last through."""
    got, _, last = accesses(5, 64, 64, 2, 1, 0, 0)
    limit = (last + 1) * 128 + 128
    assert any(run * 128 + ch * 2 < limit for run in range(last + 1, TILE) for ch in range(64))
    assert all(row <= last for row, _, _ in got)
