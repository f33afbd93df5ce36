"""Which kernel, tile and end of the contraction the sizes of the GPU tests
reach: the library's choice (int8_tiles.h), built for the host."""
import ctypes
import os
import subprocess

import pytest

import test_gpu_int8
import test_gpu_int8_tails

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("tiles") / "int8_tiles_emul.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-I{ROOT}/bit_nf4_quantized_18_amd/csrc",
                    os.path.join(ROOT, "tests", "native", "int8_tiles_emul.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.int8_choice.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_void_p]
    return lib


def _choice(lib, m, n, k):
    out = (ctypes.c_int64 * 4)()
    lib.int8_choice(m, n, -(-k // 64) * 64, out)
    return tuple(out)


def _tiles(lib):
    tiles, out = [], (ctypes.c_int64 * 4)()
    while lib.int8_tile(len(tiles), out):
        tiles.append(tuple(out))
    return tiles


def _turn(parts):
    """Units of 128 codes after which a ring of so many parts (two a unit) is in the same place again."""
    return parts if parts % 2 else parts // 2


def _ends(lib, size):
    """{(tile, a whole turn of the ring is run, units behind the last whole turn)} of a size's launches."""
    decode, one, cols, two = _choice(lib, *size)
    if decode:
        return {"decode"}
    ends = set()
    for i in {one, two} - {-1}:
        _, _, groups, parts = _tiles(lib)[i]
        turns = -(-(-(-size[2] // 64) * 64) // (128 * groups))
        ends.add((i, turns >= _turn(parts), turns % _turn(parts)))
    return ends


def test_sizes_reach_every_tile_and_end(lib):
    reached = set().union(*(_ends(lib, s) for s in test_gpu_int8.LINEAR + test_gpu_int8.TILES +
                            test_gpu_int8_tails.TAILS))
    tiles = _tiles(lib)
    names = {f"{t[0]}x{t[1]}": i for i, t in enumerate(tiles)}
    every = {"decode"} | {(i, whole, tail) for i, t in enumerate(tiles) for tail in range(_turn(t[3]))
                          for whole in (True, False) if whole or tail}
    # Ends that no size has. 64 x 128 takes one unit in 3.34 us a round, 64 x 64 in 1.62
    # with at most two rounds for one. 32 x 64 starts 0.8 us later than 64 x 64 and gains
    # 0.08 us a unit, so it has more than 10 units, 5 for each of its groups: a whole turn.
    never = {(names["64x128"], False, 1)} | {(names["32x64"], False, tail) for tail in (1, 2, 3)}
    assert every - reached == never


def test_two_launches(lib):
    """The size of the GPU test of two launches, and the last round of tiles that the split avoids."""
    size = (1000, 53248 + 77, 1856)
    decode, one, cols, two = _choice(lib, *size)
    assert not decode and one == 0 and 0 < cols < size[1] and cols % 256 == 0 and two > 0
    assert _choice(lib, 1000, 16384, 1856)[2] == 0  # whole rounds: one launch


def test_choice_edges(lib):
    assert _choice(lib, 16, 8191, 64)[0] == 1
    assert _choice(lib, 16, 8192, 64)[0] == 0 and _choice(lib, 17, 8191, 64)[0] == 0
    # the largest product that a launch takes
    assert _choice(lib, (1 << 31) - 256, 255, 64)[1] >= 0 and _choice(lib, (1 << 31) - 1, 1 << 22, 64)[1] == -1
