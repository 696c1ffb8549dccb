"""Host model of the gated delta rule's buffer accesses (rows of q, k, v, o, dO and of the
gradients, a chunk of 64 tokens at a time): which elements of a row that exists are touched, and
that nothing else is.

A chunk's rows are addressed from its first element by 32-bit byte offsets; a descriptor's range
drops what lies behind it. With 16-byte rows ("vec") the range alone tells rows that exist from
those that do not; without, every element is masked.
"""
import numpy as np
import pytest

CHUNK, NOWHERE, WRAP = 64, 0x80000000, 2**32


def stored_stride(T, s1, width):
    """The token stride that the entry points keep: with one token it has no meaning."""
    return s1 if T > 1 else width


def accepted(T, s1):
    return 0 <= s1 and (T <= 1 or s1 < 2**22)


def is_vec(T, s1, width, eb):
    """Rows that do not overlap, of 16-byte pieces one behind the other (other strides aligned)."""
    return (T <= 1 or s1 >= width) and width % 8 == 0 and (T <= 1 or s1 * eb % 16 == 0)


def touched(offsets, size, limit):
    """The offsets (bytes, as the kernel computes them modulo 2^32) of which a byte is in range."""
    o = np.asarray(offsets, dtype=np.uint64) % WRAP
    return o[o < limit], o[(o < limit) & (o + np.uint64(size) > limit)]


def check_rows(T, s1, width, pad, eb, vec, piece, keep=stored_stride):
    """Every chunk of a tensor [T][width] with token stride s1: `piece` elements per access (8: tiles of
    q, k and dO; 1: v, o and the gradients), columns up to `pad`."""
    s1 = keep(T, s1, width)
    pitch = s1 * eb % WRAP
    for t0 in range(0, T, CHUNK):
        rows = min(CHUNK, T - t0)
        limit = ((rows - 1) * s1 + width) * eb if vec else NOWHERE
        assert limit <= NOWHERE, "32-bit range"
        row, col = np.meshgrid(np.arange(CHUNK, dtype=np.int64), np.arange(0, pad, piece, dtype=np.int64), indexing="ij")
        off = (row * pitch + col * eb) % WRAP
        real = (row < rows) & (col < width)
        if vec:
            off = np.where(col < width, off, NOWHERE + row * pitch % WRAP)
            size = 16 if piece > 1 else eb
            offs = [off + 16 * i for i in range(max(1, piece * eb // 16))]
        else:  # element by element
            offs = [np.where((row < rows) & (col + i < width), off + i * eb, NOWHERE) for i in range(piece)]
            size = eb
        # the bytes that are touched, and what the rows that exist have there, without 32-bit arithmetic
        exact = row * s1 * eb + col * eb
        seen, want = [], []
        for i, o in enumerate(offs):
            hit, partial = touched(o, size, limit)
            assert partial.size == 0, "an access across the end of the range"
            seen.append(hit)
            want.append((exact + i * size)[real & (col + (i if size == eb else 0) < width)])
        seen, want = np.sort(np.concatenate(seen)), np.sort(np.concatenate(want))
        assert np.array_equal(seen, want), (T, s1, width, "rows that do not exist are touched, or existing ones are not")


WIDTHS = [(8, 64), (37, 64), (64, 64), (96, 128), (128, 128)]


@pytest.mark.parametrize("eb", [2, 4])
@pytest.mark.parametrize("width,pad", WIDTHS)
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 130])
def test_rows_of_a_chunk(T, width, pad, eb):
    strides = [width, width + 8, width + 3, 4 * width, 2**22 - 8, 2**22 - 1]
    if T == 1:  # any stride: channels first, an expanded row, a slice of a far larger tensor
        strides += [0, 1, 7, 8, 2**22, 2**26, 2**27 + 8, 2**30, 2**31, 2**40]
    else:
        strides += [0, 1, width - 1]  # inputs may overlap
    for s1 in strides:
        if not accepted(T, s1):
            continue
        vec = is_vec(T, s1, width, eb)
        check_rows(T, s1, width, pad, eb, vec, 8)
        check_rows(T, s1, width, pad, eb, T <= 1 or s1 >= width, 1)  # v, o, gradients: rows apart, of any width
        check_rows(T, s1, width, pad, eb, False, 8)


@pytest.mark.parametrize("s1", [0, 1, 8, 2**26, 2**30])
def test_a_kept_stride_of_one_token_is_seen(s1):
    """Kept as given, rows 1 .. 63 of a single token land on row 0."""
    with pytest.raises(AssertionError, match="do not exist"):
        check_rows(1, s1, 64, 64, 2, is_vec(1, s1, 64, 2), 1, keep=lambda T, s, w: s)


@pytest.mark.parametrize("threads", [256, 512])
@pytest.mark.parametrize("DK", [64, 128])
def test_tiles_are_covered_once(DK, threads):
    """The threads' pieces of a [64][DK] tile, and of 64 rows of 32 value columns (dO)."""
    per, step = CHUNK * DK // 8 // threads, threads // (DK // 8)
    pieces = [(t // (DK // 8) + i * step, t % (DK // 8) * 8) for t in range(threads) for i in range(per)]
    assert sorted(pieces) == [(r, c) for r in range(CHUNK) for c in range(0, DK, 8)]
    rows = [(t >> 2, (t & 3) * 8) for t in range(threads) if t < 4 * CHUNK]
    assert sorted(rows) == [(r, c) for r in range(CHUNK) for c in range(0, 32, 8)]
    column = [16 * (e >> 2) + (e & 3) + 4 * q for e in range(16) for q in range(4)]
    assert sorted(column) == list(range(CHUNK))
