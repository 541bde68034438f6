// groups.hpp -- which tile of which group a workgroup computes.
//
// The rows of each group are only known on the device (offsets), so the
// host launches the most workgroups any offsets can need and each finds its
// own tile: one wave-wide scan over the groups' tile counts.
#pragma once

#include "device.hpp"
#include "experts.hpp"

namespace agg {

namespace {

constexpr int kXcds = 8;

struct TileRef {
    int group;
    int64_t row0;      // first row of the tile
    int rows;          // rows of the tile that exist (the tile's height at most)
    int j;             // column tile
};

// Rows [lo, hi) of group e, kept inside [0, rows) whatever the offsets hold.
__device__ __forceinline__ void group_rows(const ProductArgs& a, int e, int& lo, int& hi)
{
    const int all = a.rows;
    if (!a.offsets) { lo = 0; hi = all; return; }
    const int b = a.offsets[e], t = a.offsets[e + 1];
    lo = b < 0 ? 0 : b > all ? all : b;
    hi = t < lo ? lo : t > all ? all : t;
}

// Everything below runs before a workgroup's first load, so it is kept
// short: lane shifts and lane reads instead of LDS shuffles, 32-bit
// positions (a launch has fewer than 2^32 threads): about 0.7 us a workgroup
// less than with shuffles and 64-bit divisions (one 1024-column call of five
// rows, fp8: 10.4 against 11.2 us).

// Sum over lanes 0 .. lane: within rows of 16 lanes, then across them.
__device__ __forceinline__ uint32_t wave_inclusive_sum(uint32_t v)
{
    int x = (int)v;
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);   // row_shr:1
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);   // row_shr:2
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);   // row_shr:4
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);   // row_shr:8
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // row_bcast:15
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);   // row_bcast:31
    return (uint32_t)x;
}

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane)
{
    return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// Position of workgroup `block` among `total`: XCD x (workgroups are dealt
// to the XCDs in turn) takes the x-th stretch of positions, so the tiles an
// L2 serves at one time are neighbours.  `total` or more: none.
__device__ __forceinline__ uint32_t xcd_position(uint32_t block, uint32_t total)
{
    const uint32_t per = total / kXcds, more = total % kXcds;
    const uint32_t x = block % kXcds, seq = block / kXcds;
    if (seq >= per + (x < more)) return total;
    return x * per + (x < more ? x : more) + seq;
}

// The same where tiles differ in cost: within each round of `round`
// workgroups (those that run at a time), so that every XCD gets its part of
// every round, the last one's too: `total` counts the tiles there are, not
// the workgroups launched (8191 rows of 16 experts, 2.6 rounds: 152 against
// 156 us; fp8, 3001 rows of 32 experts: 56 against 57; 16384 rows of 8, 4.3
// rounds, the other way: 451 against 447).
__device__ __forceinline__ uint32_t round_position(uint32_t block, uint32_t total, uint32_t round)
{
    const uint32_t in = block % round, round0 = block - in;
    if (round0 >= total) return total;
    const uint32_t left = total - round0;
    return left < round ? round0 + xcd_position(in, left) : round0 + in % kXcds * (round / kXcds) + in / kXcds;
}

// This lane's group of the 64 from c on: its rows, and its row tiles.
struct LaneGroup {
    int lo, hi;
    uint32_t n, sum;     // row tiles, and those of lanes 0 .. lane
};

template <int BI>
__device__ __forceinline__ LaneGroup lane_group(const ProductArgs& a, int c)
{
    const int e = c + (int)(threadIdx.x & 63);
    LaneGroup g{0, 0, 0, 0};
    if (e < a.groups) group_rows(a, e, g.lo, g.hi);
    g.n = (uint32_t)(g.hi - g.lo + BI - 1) / BI;
    g.sum = wave_inclusive_sum(g.n);
    return g;
}

// The tile of workgroup `block`: row tiles of BI rows, nj column tiles.
// Positions walk blocks of kPanel row tiles column by column.  Every wave
// computes the same answer.  False: nothing is left for this workgroup.
template <int BI, int kPanel>
__device__ __forceinline__ bool find_tile(const ProductArgs& a, uint32_t block, uint32_t nj, TileRef& t)
{
    const LaneGroup first = lane_group<BI>(a, 0);
    uint32_t total = lane_value(first.sum, 63);
    for (int c = 64; c < a.groups; c += 64) total += lane_value(lane_group<BI>(a, c).sum, 63);
    const uint32_t p = xcd_position(block, total * nj);
    if (p >= total * nj) return false;
    const uint32_t panel = p / (kPanel * nj), in = p - panel * kPanel * nj;
    const uint32_t left = total - panel * kPanel, high = left < kPanel ? left : kPanel;
    t.j = (int)(in / high);
    uint32_t m = panel * kPanel + in % high;      // row tile, over all groups
    for (int c = 0; c < a.groups; c += 64) {
        const LaneGroup g = c ? lane_group<BI>(a, c) : first;
        const uint64_t hit = __builtin_amdgcn_ballot_w64(g.sum > m);
        if (hit) {
            const int at = __builtin_ctzll(hit);
            m -= lane_value(g.sum - g.n, at);
            const int row0 = __builtin_amdgcn_readlane(g.lo, at) + (int)m * BI;
            const int have = __builtin_amdgcn_readlane(g.hi, at) - row0;
            t.group = c + at;
            t.row0 = row0;
            t.rows = have < BI ? have : BI;
            return true;
        }
        m -= lane_value(g.sum, 63);
    }
    return false;
}

// The tiles of the large kernel, `grid` of which run at a time: whole tiles
// of 256 rows, and half tiles of 128.  A group's last rows make a whole tile
// if they are more than 128, a half one otherwise.  The whole tiles come
// first; those that do not fill a last round of the grid are cut into half
// tiles where that ends sooner (a half tile takes 0.55 of a whole one's time).
struct HalfTiles {
    static constexpr int kBI = 256;

    struct Count {
        int lo, hi;
        uint32_t whole, half, whole_sum, half_sum;
    };

    Count first;                   // of the first 64 groups
    uint32_t wholes, cut, halves;  // positions: whole tiles, cut tiles' halves, half tiles

    __device__ __forceinline__ static Count count(const ProductArgs& a, int c)
    {
        const int e = c + (int)(threadIdx.x & 63);
        Count g{0, 0, 0, 0, 0, 0};
        if (e < a.groups) group_rows(a, e, g.lo, g.hi);
        const uint32_t rows = (uint32_t)(g.hi - g.lo), rest = rows % kBI;
        g.whole = rows / kBI + (rest > kBI / 2);
        g.half = rest > 0 && rest <= kBI / 2;
        g.whole_sum = wave_inclusive_sum(g.whole);
        g.half_sum = wave_inclusive_sum(g.half);
        return g;
    }

    __device__ __forceinline__ void init(const ProductArgs& a, uint32_t nj, uint32_t grid)
    {
        first = count(a, 0);
        uint32_t nw = lane_value(first.whole_sum, 63), nh = lane_value(first.half_sum, 63);
        for (int c = 64; c < a.groups; c += 64) {
            const Count g = count(a, c);
            nw += lane_value(g.whole_sum, 63);
            nh += lane_value(g.half_sum, 63);
        }
        // Offsets that overlap can count more tiles than 32 bits hold (others
        // fit one launch): positions that wrapped would name columns that are
        // not there.
        if (((uint64_t)nw + nh) * nj >> 30) nw = nh = 0;
        wholes = nw * nj;
        halves = nh * nj;
        const uint32_t left = wholes % grid;
        // in twentieths of a whole tile's time; workgroups without one of the
        // last whole tiles take the half ones meanwhile
        const uint32_t uncut = max(left ? 20u : 0u, 11 * ((halves + grid - left - 1) / (grid - left)));
        const bool split = left <= grid / 2 && 11 * ((halves + 2 * left + grid - 1) / grid) < uncut;
        cut = split ? 2 * left : 0;
        wholes -= cut / 2;
    }

    __device__ __forceinline__ uint32_t positions() const { return wholes + cut + halves; }

    // Row tile m (counted over all groups) of one kind.
    __device__ __forceinline__ bool rows_of(const ProductArgs& a, bool is_half, uint32_t m, TileRef& t) const
    {
        for (int c = 0; c < a.groups; c += 64) {
            const Count g = c ? count(a, c) : first;
            const uint32_t n = is_half ? g.half : g.whole, sum = is_half ? g.half_sum : g.whole_sum;
            const uint64_t hit = __builtin_amdgcn_ballot_w64(sum > m);
            if (hit) {
                const int at = __builtin_ctzll(hit);
                m -= lane_value(sum - n, at);
                const int lo = __builtin_amdgcn_readlane(g.lo, at), hi = __builtin_amdgcn_readlane(g.hi, at);
                // the half tile is the group's last
                const int row0 = lo + (is_half ? (hi - lo) / kBI : (int)m) * kBI;
                t.group = c + at;
                t.row0 = row0;
                t.rows = hi - row0 < kBI ? hi - row0 : kBI;
                return true;
            }
            m -= lane_value(sum, 63);
        }
        return false;
    }

    // The tile of position p (`is_half`: it has at most 128 rows); false if
    // there is none.
    __device__ __forceinline__ bool tile(const ProductArgs& a, uint32_t nj, uint32_t p, bool& is_half,
                                         TileRef& t) const
    {
        constexpr uint32_t kPanel = 4;
        is_half = p >= wholes;
        const bool of_half = p >= wholes + cut;
        const uint32_t q = of_half ? p - wholes - cut : is_half ? wholes + (p - wholes) / 2 : p;
        const uint32_t tiles = (of_half ? halves : wholes + cut / 2) / nj;
        const uint32_t panel = q / (kPanel * nj), in = q - panel * kPanel * nj;
        const uint32_t left = tiles - panel * kPanel, high = left < kPanel ? left : kPanel;
        t.j = (int)(in / high);
        if (!rows_of(a, of_half, panel * kPanel + in % high, t)) return false;
        if (is_half && !of_half) {
            const int second = (int)((p - wholes) & 1);
            t.row0 += second * (kBI / 2);
            t.rows = second ? t.rows - kBI / 2 : kBI / 2;   // a whole tile has more than 128
        }
        return true;
    }
};

}  // namespace

}  // namespace agg
