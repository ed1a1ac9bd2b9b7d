"""The arithmetic by which the attention kernels share work out to their blocks (csrc/lq_share.h, the same source that
the kernels are built from), compiled for the host and walked through.  No GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_quantized_dequant_gb300", "csrc")

SOURCE = r"""
#include <map>
#include <set>
#include <utility>
#include <vector>
#include "lq_share.h"
using namespace lq;

// Walks the prefix kernel's blocks, then the joins of all units.  0, or the number of the first thing that is wrong.
extern "C" int walk_prefix(int units, int each, int sms) {
    const int total = units * (each + kPreUnitCost), blocks = sms < total ? sms : total;
    const int slots = prefix_slots(each, total, blocks);
    const Shares s(total, blocks);
    std::map<std::pair<int, int>, std::pair<int, int>> wrote;      // (block, slot) -> unit, key blocks
    long long keys = 0;
    for (int c = 0; c < blocks; ++c) {
        const int g0 = prefix_block_at(each, s.first(c)), g1 = prefix_block_at(each, s.first(c + 1));
        if (g0 > g1 || (c == 0 && g0 != 0) || (c == blocks - 1 && g1 != units * each)) return 1;
        for (int done = 0; done < g1 - g0;) {
            const int unit = (g0 + done) / each, end = (unit + 1) * each < g1 ? (unit + 1) * each : g1, nb = end - (g0 + done);
            const int slot = prefix_slot(s, each, c, unit);
            if (slot < 0 || slot >= slots) return 2;
            if (!wrote.insert({{c, slot}, {unit, nb}}).second) return 3;      // a slot taken twice
            done += nb;
            keys += nb;
        }
    }
    if (keys != (long long)units * each) return 4;
    for (int unit = 0; unit < units; ++unit) {
        const int us = prefix_unit_place(each, unit), c0 = s.of(us), c1 = s.of(us + each - 1);
        int got = 0;
        for (int c = c0; c <= c1; ++c) {
            const auto it = wrote.find({c, c == c0 ? prefix_slot(s, each, c, unit) : 0});
            if (it == wrote.end() || it->second.first != unit) return 5;      // another unit's sums
            got += it->second.second;
        }
        if (got != each) return 6;
    }
    return 0;
}

// n things over c parties: consecutive ranges that differ by one at most, and every thing's party.
extern "C" int walk_shares(int n, int c) {
    const Shares s(n, c);
    if (s.first(0) != 0 || s.first(c) != n) return 1;
    for (int k = 0; k < c; ++k) {
        const int a = s.first(k), b = s.first(k + 1), size = b - a;
        if (size != n / c && size != n / c + 1) return 2;
        if (size > 0 && (s.of(a) != k || s.of(b - 1) != k)) return 3;
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def shares(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("shares")
    (d / "walk.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "walk.cpp"), "-o", str(d / "walk.so")], check=True)
    return ctypes.CDLL(str(d / "walk.so"))


@pytest.mark.parametrize("sms", [1, 7, 148, 152])
@pytest.mark.parametrize("each", [1, 2, 4, 16, 251])
def test_every_unit_of_the_prefix_kernel_has_slots_of_its_own(shares, sms, each):
    for units in list(range(1, 601)) + [1024, 4097]:
        assert shares.walk_prefix(units, each, sms) == 0, (units, each, sms)


@pytest.mark.parametrize("blocks", [1, 148, 152, 304, 456, 608, 1024])
def test_shares_up_to_the_limit_of_a_call(shares, blocks):
    """A call's places go up to 2^31 - 1 (the host refuses more); blocks are one to four per SM."""
    for n in (1, blocks - 1, blocks, blocks + 1, 39916801, 2 ** 29 + 11, 640000003, 1300000000, 2147483547, 2 ** 31 - 1):
        if n > 0:
            assert shares.walk_shares(n, blocks) == 0, n
