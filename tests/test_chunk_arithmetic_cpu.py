"""The arithmetic by which the chunk attention kernel cuts requests into tiles of rows, key blocks and shares
(csrc/lq_chunk.h, the same source that the kernel is built from), compiled for the host and walked through.  No GPU."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_quantized_dequant_gb300", "csrc")

SOURCE = r"""
#include <vector>
#include "lq_chunk.h"
using namespace lq;

static bool sees(long long p, long long j, int window, int sinks) { return j <= p && (window <= 0 || j > p - window || j < sinks); }

// Every tile's blocks against what its rows see.  0, or the number of the first thing that is wrong.
extern "C" int check_tiles(int len, int fresh, int group, int window, int sinks, int tile_rows) {
    const int tiles = chunk_tiles(fresh, group, tile_rows), kbs = (len + kChunkKeys - 1) / kChunkKeys;
    if ((long long)tiles * tile_rows < (long long)fresh * group || (long long)(tiles - 1) * tile_rows >= (long long)fresh * group) return 1;
    for (int rt = 0; rt < tiles; ++rt) {
        const ChunkTile t(len, fresh, group, window, sinks, tile_rows, rt);
        if (t.blocks < 1) return 2;
        std::vector<int> visits(kbs + 1, 0);
        int last = -1;
        for (int i = 0; i < t.blocks; ++i) {
            const int kb = t.block(i);
            if (kb <= last) return 3;                        // in order, each once
            last = kb;
            if (kb < kbs) visits[kb] = 1;
            else if (t.p1 >= 0) return 4;
        }
        for (int kb = 0; kb < kbs; ++kb) {
            bool any = false, all = true;
            for (int r = rt * tile_rows; r < (rt + 1) * tile_rows && r < fresh * group; ++r)
                for (int k = 0; k < kChunkKeys; ++k) {
                    const bool s = sees((long long)len - fresh + r / group, (long long)kb * kChunkKeys + k, window, sinks);
                    any |= s, all &= s;
                }
            if (any && !visits[kb]) return 5;
            if (visits[kb] && t.whole(kb, window, sinks) && !all) return 6;
            if (visits[kb] && !any && t.p1 >= 0 && t.blocks > 2) return 7;    // (nothing is visited for nothing)
        }
    }
    return 0;
}

// n places shared out: every place is its party's, parties' shares follow one another.
extern "C" int check_shares(long long n, int c) {
    const WideShares s(n, c);
    if (s.first(0) != 0 || s.first(c) != n) return 1;
    for (int k = 0; k < c; ++k) {
        const int64_t a = s.first(k), b = s.first(k + 1);
        if (b < a || b - a > n / c + 1) return 2;
        if (b > a && (s.of(a) != k || s.of(b - 1) != k)) return 3;
    }
    return 0;
}

// Ends of the range: nothing wraps.
extern "C" int check_ends() {
    const int most = 0x7fffff00;
    const ChunkTile a(most, 1, 1, 0, 0, 128, 0), b(most, 1, 1, most, most, 128, 0), c(0, most, 1, 1, most, 128, most / 128 - 1);
    if (a.p0 != most - 1 || a.blocks != most / 128 || a.block(a.blocks - 1) != most / 128 - 1) return 1;
    if (b.lowest != 0 || b.sunk != 0 || b.blocks != most / 128) return 2;
    if (c.p1 != -1 || c.blocks != 1 || c.block(0) != 0) return 3;
    const ChunkTile d(most, 1, 1, 1, most, 128, 0);
    if (d.lowest != most - 1 || d.sunk != most / 128 - 1 || d.gap != 0 || d.blocks != most / 128) return 4;
    if (!a.whole(0, 0, 0) || !b.whole(0, most, most) || d.whole(most / 128 - 1, 1, most) == false) return 5;
    return 0;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("chunk")
    (d / "walk.cpp").write_text(SOURCE)
    subprocess.run([cc, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "walk.cpp"), "-o", str(d / "walk.so")], check=True)
    L = ctypes.CDLL(str(d / "walk.so"))
    L.check_shares.argtypes = [ctypes.c_longlong, ctypes.c_int]
    return L


@pytest.mark.parametrize("tile_rows", [128, 256])
def test_tiles_visit_what_their_rows_see(lib, tile_rows):
    g = random.Random(tile_rows)
    for _ in range(600):
        fresh, group = g.choice([1, 2, 7, 65, 128, 300]), g.choice([1, 2, 3, 8, 40, 130])
        length = max(0, fresh + g.choice([-5, 0, 0, 1, 60, 128, 700, 1500]))
        window, sinks = g.choice([0, 1, 2, 63, 128, 129, 400, 5000]), g.choice([0, 1, 4, 128, 129, 300, 5000])
        assert lib.check_tiles(length, fresh, group, window, sinks if window else 0, tile_rows) == 0, (length, fresh, group, window, sinks)


def test_shares(lib):
    for n in (0, 1, 5, 151, 152, 153, 10007, 2 ** 33 + 7):
        for c in (1, 2, 76, 152):
            assert lib.check_shares(n, c) == 0, (n, c)


def test_ends_of_the_range(lib):
    assert lib.check_ends() == 0
