"""What the cache reads when it looks an accepted path over, whatever the path holds (CPU only).

The function that decides whether a stream's path may be kept is taken from the kernel's source and compiled for the CPU with
tables that record every read outside of them.  Each lane runs on its own: a lane reads before it can know what the others found.
"""
import itertools
import os
import re
import subprocess

import pytest

import mxfp4_moe_expert_gb300 as pkg

PACKAGE = os.path.dirname(os.path.abspath(pkg.__file__))
CSRC, INCLUDE = os.path.join(PACKAGE, "csrc"), os.path.join(os.path.dirname(PACKAGE), "include")

HARNESS = r"""
#include <cstdint>
#include <cstdio>
#include "moe_mxfp4.h"
#define __device__
#define __forceinline__ inline
static long long outside = 0;
struct Checked {
    const int* p;
    int n;
    int operator[](int64_t i) const {
        if (i >= 0 && i < n) return p[i];
        ++outside;
        return 0;
    }
};
struct CacheView {
    struct { int M, P; } L;
    int page_shift;
    Checked lengths, helds, pages, counts;
    Checked length() const { return lengths; }
    Checked held() const { return helds; }
    Checked table(int) const { return pages; }
    Checked refcount() const { return counts; }
};
inline int __all_sync(unsigned, int x) { return x; }
%s
// Lines of: length, block, accepted, and the path.  Answers: what the stream keeps (-1: left alone), reads outside.
int main() {
    const int held = 3, pages[3] = {2, 0, 1}, counts[3] = {1, 1, 1};
    int length, block, accepted, path[64];
    while (std::scanf("%%d %%d %%d", &length, &block, &accepted) == 3) {
        for (int i = 0; i < block; ++i)
            if (std::scanf("%%d", path + i) != 1) return 1;
        CacheView c = {{4, 3}, 4, {&length, 1}, {&held, 1}, {pages, held}, {counts, 3}};
        moe_mxfp4_commit_args a = {};
        a.accepted_dev = &accepted;
        a.path_dev = path;
        a.streams = 1;
        a.block = block;
        outside = 0;
        int keeps = accepted;
        for (int lane = 0; lane < 32; ++lane) {
            bool bad;
            const int n = path_count(c, a, 0, lane, &bad);
            if (n < 0) keeps = n;
            if (accepted >= 0 && bad != (n < 0)) return 2;
        }
        std::printf("%%d %%lld\n", keeps, outside);
    }
}
"""


def function_text(source, name):
    """The definition of `name`, from the beginning of its line to the brace that closes it."""
    at = re.search(rf"^[^\n]*\b{name}\([^;{{]*\{{", source, re.M)
    end, depth = at.end(), 1
    while depth:
        depth += {"{": 1, "}": -1}.get(source[end], 0)
        end += 1
    return source[at.start():end]


@pytest.fixture(scope="module")
def look(tmp_path_factory):
    where = tmp_path_factory.mktemp("paths")
    with open(os.path.join(CSRC, "cache_pages.cu")) as f:
        text = HARNESS % function_text(f.read(), "path_count")
    (where / "look.cpp").write_text(text)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-I", INCLUDE, "-o", str(where / "look"), str(where / "look.cpp")], check=True)

    def run(cases):
        lines = "".join(" ".join(map(str, (length, len(path), n, *path))) + "\n" for length, n, path in cases)
        out = subprocess.run([str(where / "look")], input=lines, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


VALUES = [-(1 << 31), -(1 << 30), -40, -21, -6, -5, -3, -1, 0, 1, 2, 3, 4, 20, (1 << 31) - 1]


@pytest.mark.parametrize("length", [0, 1, 15, 20, 43, 44, 45, 48])
def test_no_path_is_looked_up_outside_the_pages_that_are_held(look, length):
    room = 48                                            # three pages of 16
    cases = [(length, n, (*path, 7)) for path in itertools.product(VALUES, repeat=3) for n in (1, 2, 3)]
    for (_, n, path), (keeps, outside) in zip(cases, look(cases)):
        took = path[:n]
        good = (all(0 <= p < 4 and length + p < room for p in took) and all(a < b for a, b in zip(took, took[1:]))
                and length + n <= room)
        assert outside == 0, (n, path)
        assert keeps == (n if good else -1), (n, path)


def test_counts_that_no_block_has(look):
    cases = [(20, n, (0, 1, 2, 3)) for n in (-1, 0, 4, 5, 29, 1 << 30)]
    assert look(cases) == [(-1, 0), (0, 0), (4, 0), (-1, 0), (-1, 0), (-1, 0)]
