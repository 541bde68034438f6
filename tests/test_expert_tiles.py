"""Which tile a workgroup of the expert products takes, run on the host from
the kernels' own header (csrc/groups.hpp): 64 contexts stand for a wave's lanes
and meet at every lane shift, lane read and ballot.

Valid offsets: the workgroups that the host launches take every row of every
group, in every column tile, exactly once.  Offsets that break the rules, also so far that
the tiles they count do not fit 32 bits: no tile leaves the rows or the columns."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "communication_gemm_amd", "csrc")

WAVE = r"""
#include <ucontext.h>
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <functional>
#include <vector>
#include "experts.hpp"

static ucontext_t lanes[64], host;
static int lane_now;
static long long slot[64], seen[64];
static struct { unsigned x; } lane_id[64];
#define threadIdx lane_id[lane_now]

// Every lane gives v; all go on once each has.
static long long* meet(long long v)
{
    const int me = lane_now;
    slot[me] = v;
    swapcontext(&lanes[me], &host);
    return seen;
}
static int update_dpp(int old, int v, int ctrl, int rows)
{
    const int me = lane_now, row = me / 16;
    const long long* all = meet(v);
    int from = -1;
    if (ctrl > 0x110 && ctrl < 0x120) { if (me % 16 >= ctrl - 0x110) from = me - (ctrl - 0x110); }
    else if (ctrl == 0x142) { if (row > 0) from = row * 16 - 1; }
    else if (ctrl == 0x143) { if (row > 1) from = 31; }
    else abort();
    return (rows >> row & 1) && from >= 0 ? (int)all[from] : old;
}
static int readlane(int v, int lane) { return (int)meet(v)[lane]; }
static unsigned long long ballot(bool b)
{
    const long long* all = meet(b);
    unsigned long long m = 0;
    for (int l = 0; l < 64; ++l) m |= (unsigned long long)(all[l] != 0) << l;
    return m;
}
#define __builtin_amdgcn_update_dpp(o, v, c, r, b, z) update_dpp(o, v, c, r)
#define __builtin_amdgcn_readlane(v, l) readlane(v, l)
#define __builtin_amdgcn_ballot_w64(b) ballot(b)
using std::max;
#include "groups_host.hpp"
using namespace agg;

static std::function<void()>* body;
static void enter() { (*body)(); }
static void wave(std::function<void()> f)     // f as a whole wave runs it
{
    static std::vector<char> stacks(64 << 16);
    body = &f;
    static bool done[64];
    for (int l = 0; l < 64; ++l) {
        lane_id[l].x = l;
        done[l] = false;
        getcontext(&lanes[l]);
        lanes[l].uc_stack.ss_sp = &stacks[(size_t)l << 16];
        lanes[l].uc_stack.ss_size = 1 << 16;
        lanes[l].uc_link = &host;
        makecontext(&lanes[l], enter, 0);
        slot[l] = 0;
    }
    static long long mark = 0x7fffffffffffffffll;
    for (bool any = true; any;) {
        any = false;
        for (int l = 0; l < 64; ++l) {
            if (done[l]) continue;
            slot[l] = mark;
            lane_now = l;
            swapcontext(&host, &lanes[l]);
            if (slot[l] == mark) done[l] = true; else any = true;
        }
        std::copy(slot, slot + 64, seen);
    }
}

struct Got { TileRef t; bool half; };

int main(int argc, char** argv)
{
    // variant rows columns first_block blocks offsets...
    const int variant = atoi(argv[1]);
    ProductArgs a{};
    a.rows = atoll(argv[2]);
    a.J = atoi(argv[3]);
    a.cus = 256;
    const unsigned b0 = (unsigned)atoll(argv[4]), nb = (unsigned)atoll(argv[5]);
    std::vector<int32_t> off;
    for (int i = 6; i < argc; ++i) off.push_back(atoi(argv[i]));
    a.offsets = off.data();
    a.groups = (int)off.size() - 1;
    std::vector<Got> got;
    wave([&] {
        auto note = [&](const TileRef& t, bool half) { if (lane_now == 0) got.push_back({t, half}); };
        if (variant == 0) {
            HalfTiles h;
            h.init(a, (a.J + 255) / 256, a.cus);
            if (lane_now == 0) printf("positions %u\n", h.positions());
            for (unsigned b = b0; b < b0 + nb; ++b) {
                const uint32_t p = round_position(b, h.positions(), a.cus);
                if (p >= h.positions()) continue;
                TileRef t;
                bool half;
                if (h.tile(a, (a.J + 255) / 256, p, half, t)) note(t, half);
            }
        } else {
            for (unsigned b = b0; b < b0 + nb; ++b) {
                TileRef t;
                const bool ok = variant == 64 ? find_tile<64, 4>(a, b, (a.J + 63) / 64, t)
                                              : find_tile<16, 1>(a, b, (a.J + 15) / 16, t);
                if (ok) note(t, false);
            }
        }
    });
    for (const Got& g : got)
        printf("%d %lld %d %d %d\n", g.t.group, (long long)g.t.row0, g.t.rows, g.t.j, (int)g.half);
}
"""

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ needed")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("tiles")
    header = open(os.path.join(CSRC, "groups.hpp")).read()
    assert '#include "device.hpp"' in header
    (at / "groups_host.hpp").write_text(header.replace('#include "device.hpp"', ""))
    (at / "tiles.cpp").write_text(WAVE)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-D__HIP_PLATFORM_AMD__", f"-I{rocm}/include",
                    f"-I{CSRC}", f"-I{at}", str(at / "tiles.cpp"), "-o", str(at / "tiles")], check=True)

    def run(variant, rows, N, first, blocks, offsets):
        out = subprocess.run([str(at / "tiles"), *map(str, (variant, rows, N, first, blocks, *offsets))],
                             check=True, capture_output=True, text=True, timeout=120).stdout
        lines = out.split("\n")[:-1]
        positions = int(lines.pop(0).split()[1]) if variant == 0 else None
        return positions, [tuple(map(int, line.split())) for line in lines]
    return run


def launched(variant, rows, N, groups):
    """Workgroups of csrc/launch.hpp's grid_of and csrc/experts.hip's launch_large."""
    bi, bj = (256, 256) if variant == 0 else (variant, variant)
    tiles = (rows // bi + min(groups, rows)) * -(-N // bj)
    if variant == 0:
        tiles += min(tiles, 128)
    return -(-tiles // 8) * 8


def starts(counts, first=0):
    at = [first]
    for c in counts:
        at.append(at[-1] + c)
    return at


CASES = [
    (0, [700, 300, 129, 1, 100, 0, 128], 4360),          # cut tiles
    (0, [1500, 1025, 1100, 300, 129], 4360),             # two rounds, the second cut
    (0, [3000, 3328, 70], 4360),
    (0, [600], 8200),
    (0, [60] * 30 + [0] + [61] * 35 + [0, 300, 257, 1, 128], 520),
    (0, [0, 0, 0], 520),
    (64, [20, 64, 1, 0, 7, 33, 16, 65], 328),
    (64, [3, 0, 64, 65, 17] * 14, 200),
    (16, [1, 16, 17, 0, 3], 72),
]


@pytest.mark.parametrize("variant,counts,N", CASES)
@pytest.mark.parametrize("first", [0, 5])
def test_every_row_and_column_tile_once(program, variant, counts, N, first):
    rows = first + sum(counts) + 2 * first
    off = starts(counts, first)
    bi, bj = (256, 256) if variant == 0 else (variant, variant)
    positions, got = program(variant, rows, N, 0, launched(variant, rows, N, len(counts)), off)
    want = {}
    for e, c in enumerate(counts):
        for j in range(-(-N // bj)):
            for r in range(off[e], off[e] + c):
                want[r, j] = e
    taken = {}
    for e, row0, n, j, half in got:
        assert 1 <= n <= (bi // 2 if half else bi)
        for r in range(row0, row0 + n):
            assert (r, j) not in taken
            taken[r, j] = e
    assert taken == want
    assert positions is None or positions == len(got)


@pytest.mark.parametrize("variant", [0, 64, 16])
@pytest.mark.parametrize("off", [[-5, 10, 20], [0, 300, 10 ** 6], [0, 700, 4], [700, 0, 700, 0, 700, 3],
                                 [2 ** 31 - 1, -2 ** 31, 7, 2 ** 31 - 1], [900, 800, 700, 600]])
def test_broken_offsets_stay_inside(program, variant, off):
    rows, N = 700, 520
    _, got = program(variant, rows, N, 0, launched(variant, rows, N, len(off) - 1), off)
    for e, row0, n, j, half in got:
        assert 0 <= e < len(off) - 1 and 0 <= row0 and 1 <= n and row0 + n <= rows
        assert 0 <= j < -(-N // (variant or 256))


@pytest.mark.parametrize("columns,tiles", [(768, (2 ** 32 + 2) // 3), (1280, (2 ** 32 + 4) // 5),
                                           (2816, (2 ** 33 + 6) // 11), (256 * 23, (2 ** 32 + 91) // 23)])
def test_broken_offsets_that_count_past_32_bits_stay_inside(program, columns, tiles):
    """Groups that all hold (almost) every row: tiles x columns is a little
    more than a multiple of 2^32."""
    per = 1 << 20
    off = [0]
    while tiles:
        n = min(tiles, per)
        off += [256 * n, 0]
        tiles -= n
    nj = columns // 256
    _, got = program(0, 256 * per, columns, 0, 16 * nj, off)
    for e, row0, n, j, half in got:
        assert 0 <= row0 and 1 <= n and row0 + n <= 256 * per and 0 <= j < nj
