"""The walk over packed requests, taken on the host over every small table of lengths.  The convolution's: whatever the
table holds, no row outside the packed tensor or before the request's own is read, every row of a tile is gone over
once, and sound tables give each row to its request.  The recurrence's: rows of no request get zeros."""
import os
import subprocess

import pytest

from kda_gated_delta_gb300 import build

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "kda_walk.cuh"

static long tables = 0, foreign = 0;
static std::vector<int32_t> cu;
static void fail(const char* what, int T, int tile, int W)
{
    printf("%s: W %d, %d rows, tiles of %d, table", what, W, T, tile);
    for (int32_t c : cu) printf(" %d", c);
    printf("\n");
    exit(1);
}

// What a thread of the convolution does with its tile, row numbers in the place of accesses.
template <int W>
static void walk(int T, int tile)
{
    const int n = (int)cu.size() - 1;
    bool sound = cu[0] == 0 && cu[n] == T;
    for (int b = 0; b < n; ++b) sound = sound && cu[b] <= cu[b + 1];
    std::vector<int> owner(T, -1), seen(T, 0), starts(n, 0);
    if (sound)
        for (int b = 0; b < n; ++b)
            for (int t = cu[b]; t < cu[b + 1]; ++t) owner[t] = b;
    for (int k = 0; k * tile < T; ++k) {
        const int64_t t0 = kda::conv_tile_edge<W>(cu.data(), n, T, (int64_t)k * tile), t1 = kda::conv_tile_edge<W>(cu.data(), n, T, (int64_t)(k + 1) * tile);
        if (t0 < 0 || t1 > T) fail("tile outside the rows", T, tile, W);
        if (t0 >= t1) continue;
        int32_t b = kda::layer_owner(cu.data(), n, t0);
        int64_t t = t0;
        while (t < t1) {
            const kda::Stretch s = kda::conv_stretch<W>(cu.data(), n, T, t, b);
            if (s.last <= t) fail("no way on", T, tile, W);
            if (s.own) {
                if (b < 0 || b >= n) fail("slot of no request", T, tile, W);
                if (t == s.first) {
                    ++starts[b];
                    for (int i = 0; i < W - 1; ++i) {               // the new state
                        const int64_t row = s.last - (W - 1) + i;
                        if (row >= s.first && (row < 0 || row >= T)) fail("row of the new state outside", T, tile, W);
                    }
                } else {
                    for (int i = 0; i < W - 1; ++i) {               // the window
                        const int64_t row = t - (W - 1) + i;
                        if (row < 0 || row >= T || row < s.first) fail("row of the window outside", T, tile, W);
                    }
                }
                if (s.last > T) fail("rows behind the last", T, tile, W);
            } else {
                ++foreign;
            }
            if (sound && (!s.own || b != owner[t])) fail("a sound table's row given to another", T, tile, W);
            for (; t < s.last && t < t1; ++t) ++seen[t];
        }
    }
    if (sound) {
        for (int t = 0; t < T; ++t)
            if (seen[t] != 1) fail("a row not gone over once", T, tile, W);
        for (int b = 0; b < n; ++b)
            if (starts[b] != (cu[b + 1] > cu[b])) fail("a state not replaced once", T, tile, W);
    }
}

// The rows that the recurrence gives zeros to: in a table that does not decrease, all that no request owns, and no others.
static void unowned(int T)
{
    const int n = (int)cu.size() - 1;
    int64_t lo, hi, first, last;
    kda::unowned_rows(cu.data(), n, T, lo, hi);
    if (lo < 0 || hi < lo || hi > T) fail("zeros outside the rows", T, 0, 0);
    std::vector<char> owned(T, 0);
    for (int b = 0; b < n; ++b) {
        if (cu[b] > cu[b + 1]) return;
        if (kda::layer_rows(cu.data(), b, T, first, last))
            for (int64_t t = first; t < last; ++t) owned[t] = 1;
    }
    for (int t = 0; t < T; ++t)
        if (owned[t] == (t < lo || t >= hi)) fail("zeros in a request's rows, or none in nobody's", T, 0, 0);
}

static void all(size_t at, int lo, int hi, int T)
{
    if (at < cu.size()) {
        for (int v = lo; v <= hi; ++v) {
            cu[at] = v;
            all(at + 1, lo, hi, T);
        }
        return;
    }
    ++tables;
    unowned(T);
    for (int tile : {4, 12}) {
        walk<2>(T, tile);
        walk<3>(T, tile);
        walk<4>(T, tile);
    }
}

int main()
{
    for (int T : {1, 2, 3, 5, 9, 14})
        for (int n = 1; n <= 3; ++n) {
            cu.assign(n + 1, 0);
            all(0, -2, T + 2, T);
        }
    for (int T : {4, 9}) {
        cu.assign(5, 0);
        all(0, 0, T, T);
    }
    printf("tables %ld foreign %ld\n", tables, foreign);
    return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("walk")
    src, exe = d / "walk.cpp", d / "walk"
    src.write_text(SOURCE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", build.CSRC, "-I", cuda, str(src), "-o", str(exe)], check=True)
    return str(exe)


def test_every_small_table(program):
    r = subprocess.run([program], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    tables, foreign = (int(w) for w in r.stdout.split()[1::2])
    assert tables > 100000 and foreign > 0
