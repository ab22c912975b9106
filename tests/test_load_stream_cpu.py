"""The large FP8 product's stream of loads (csrc/load_stream.h), replayed on the host: no half tile is read from LDS
before its loads have been waited for, and no slot is loaded again before it has been read.

The replay is a C++ program over the header that the kernel takes its counts and its rule from.  Memory operations of a
wave end in the order in which they were begun, so "all but the last n" has the ones before those ended, and nothing
else may be taken as ended.
"""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_diagonal_eigenbasis_amd", "csrc")

REPLAY = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "load_stream.h"
using namespace dobb;

struct Replay {
    std::vector<long> ops;                       // in order: the half that a load is for, -1 for a store or another load
    size_t ended = 0;
    std::vector<long> slot = std::vector<long>(kRing, -1);
    std::vector<bool> read_done = std::vector<bool>(kRing, true);
    long bad = 0;
    void ask(long g) {
        if (!read_done[g % kRing]) ++bad;
        slot[g % kRing] = g;
        read_done[g % kRing] = false;
        for (int k = 0; k < kHalfLoads + (g % 2 ? 0 : kScaleLoads); ++k) ops.push_back(g);
    }
    void wait(int left) {
        if (left > kMostLeft) ++bad;
        if (ops.size() > (size_t)left && ops.size() - left > ended) ended = ops.size() - left;
    }
    void read(long g) {
        if (slot[g % kRing] != g) ++bad;
        for (size_t i = ended; i < ops.size(); ++i)
            if (ops[i] == g) { ++bad; break; }
        read_done[g % kRing] = true;
    }
    void store(int n) { for (int k = 0; k < n; ++k) ops.push_back(-1); }
};

// tiles: bit t of `whole` says whether tile t's stores are counted; else it leaves `few` stores.  groups: loads of a
// bias come before each part of the stores and are waited for, with all that is before them.
long replay(int H, bool fp32, int tiles, unsigned whole, int few, bool bias) {
    Replay r;
    StreamWaits waits;
    const int left = stream_left(fp32);
    for (long g = 0; g < kRing; ++g) r.ask(g);
    r.wait(kStartLeft);
    r.read(0);
    long g = 0;
    for (int t = 0; t < tiles; ++t) {
        for (int h = 0; h < H; ++h, ++g) {
            r.wait(waits.next() ? left : kBehind);
            r.read(g + 1);
            r.ask(g + kRing);
        }
        const bool counted = whole >> t & 1;
        const int stores = counted ? stream_stores(fp32) : few, groups = fp32 ? 4 : 2;
        for (int k = 0; k < groups; ++k) {
            if (bias) {
                r.store(16);                     // (loads, that is)
                r.wait(0);
            }
            r.store(stores / groups);
        }
        waits.stored(counted);
    }
    return r.bad;
}

int main() {
    long cases = 0;
    for (int H : {2, 4, 6, 8, 26, 100})
        for (int fp32 = 0; fp32 < 2; ++fp32)
            for (int few : {0, 4, 64, 256})
                for (int bias = 0; bias < 2; ++bias)
                    for (unsigned whole = 0; whole < 32; ++whole) {
                        ++cases;
                        if (const long bad = replay(H, fp32, 5, whole, few, bias)) {
                            std::printf("%d halves, fp32 %d, whole tiles %#x, %d stores of others, bias %d: %ld read or loaded too early\n", H,
                                        fp32, whole, few, bias, bad);
                            return 1;
                        }
                    }
    std::printf("%ld cases\n", cases);
    return 0;
}
"""


def _replay(tmp_path, source):
    cxx = shutil.which(os.environ.get("CXX", "g++")) or shutil.which("clang++")
    if not cxx:
        pytest.skip("no host compiler")
    src, exe = str(tmp_path / "replay.cpp"), str(tmp_path / "replay")
    with open(src, "w") as f:
        f.write(source)
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-I", CSRC, src, "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True)


def test_every_half_is_waited_for(tmp_path):
    r = _replay(tmp_path, REPLAY)
    assert r.returncode == 0, r.stdout
    assert r.stdout == f"{6 * 2 * 4 * 2 * 32} cases\n"


@pytest.mark.parametrize("old,new", [("kBehind)", "kBehind + 1)"), ("kStartLeft)", "kStartLeft + 1)"), ("waits.next() ? left", "true ? left"),
                                     ("stream_left(fp32)", "stream_left(fp32) + (fp32 ? 0 : 1)")])
def test_the_replay_sees_a_wait_that_leaves_too_much(tmp_path, old, new):
    assert REPLAY.count(old) == 1
    assert _replay(tmp_path, REPLAY.replace(old, new)).returncode == 1


def test_the_kernel_takes_its_waits_from_the_header():
    text = open(os.path.join(CSRC, "k_fp8_matmul.hip")).read()
    waits = re.findall(r"wait_all_but<([^>]*)>\(([^;]*)\);", text)
    assert waits == [("kStartLeft", ""), ("kBehind, kLeft", "waits.next()"), ("kBehind, kLeft", "waits.next()")]
    assert "kLeft = stream_left(EXACT)" in text and len(re.findall(r"waits\.stored\(", text)) == 2
