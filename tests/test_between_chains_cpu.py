"""The longest chain of additions behind a row's or head's sum in each kernel of the block boundary
and of rotary positions, against the chain(H) = H / 256 + 40 that the 64-bit references' bounds count
(CPU; the layouts are restated from the kernels' own constants)."""
import math

import pytest

from _between64 import chain

WIDTHS = sorted({1, 2, 3, 7, 8, 31, 64, 100, 255, 256, 257, 1000, 1024, 2050, 4096, 4097, 6144, 8191,
                 8192, 12288, 16384, 32768, 65536, 131072, 262144, 1 << 20})


def up(a, b):
    return -(-a // b)


def vectors(size):
    return [v for v in (16, 8, 4, 2) if v >= size]


@pytest.mark.parametrize("size", [4, 2])
def test_staged_rows(size):
    """32 bytes to a thread, added in pairs of sums, then a warp's five levels, the warps in fours and
    two levels more, and the ranks of a cluster."""
    for h in WIDTHS:
        for cluster in (1, 2, 4, 8, 16):
            threads = up(up(h * size, 16 * cluster), 2)
            if threads > 1024:
                continue
            own = 32 // size // 2 + 1
            longest = own + 5 + up(up(threads, 32), 4) + 2 + (cluster if cluster > 1 else 0)
            assert longest <= chain(h), (h, cluster)


@pytest.mark.parametrize("size", [4, 2])
def test_rows_in_registers(size):
    """Four or eight vectors of less than 16 bytes to a thread, the warps one after the other."""
    for h in WIDTHS:
        for v in vectors(size):
            if v == 16 or h * size % v:
                continue
            for each in (4, 8):
                threads = up(up(h * size // v, each), 32) * 32
                if threads > 1024 or (each == 8 and threads < 416):
                    continue        # eight only where four need more than 768 threads
                assert each * (v // size) + 5 + threads // 32 <= chain(h), (h, v, each)


@pytest.mark.parametrize("size", [4, 2])
def test_rows_read_for_each_sum(size):
    """256 threads, a sum for each vector added to the thread's, then eight warps."""
    for h in WIDTHS:
        for v in vectors(size):
            if h * size % v == 0:
                assert v // size + up(h * size // v, 256) + 5 + 8 <= chain(h), (h, v)


@pytest.mark.parametrize("size", [4, 2])
def test_heads(size):
    """Two vectors to a lane, added in pairs of sums; or a warp's lanes with every 32nd pair."""
    for dim in (2, 16, 64, 80, 96, 128, 192, 256, 512, 1024):
        for v in vectors(size):
            if v // size <= dim:
                assert max(1, v // size) + 1 + int(math.log2(32)) <= chain(dim)
        assert 2 * up(dim // 2, 32) + 5 <= chain(dim)
