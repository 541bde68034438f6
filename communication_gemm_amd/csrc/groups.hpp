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
__device__ __forceinline__ void group_rows(const ProductArgs& a, int e, int64_t& lo, int64_t& hi)
{
    if (!a.offsets) { lo = 0; hi = a.rows; return; }
    int64_t b = a.offsets[e], t = a.offsets[e + 1];
    lo = b < 0 ? 0 : b > a.rows ? a.rows : b;
    hi = t < lo ? lo : t > a.rows ? a.rows : t;
}

__device__ __forceinline__ uint32_t wave_inclusive_sum(uint32_t v, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// Position of workgroup `block` among `total`: XCD x (workgroups are dealt
// to the XCDs in turn) takes the x-th stretch of positions, so the tiles an
// L2 serves at one time are neighbours.  Past the end: -1.
__device__ __forceinline__ int64_t xcd_position(uint32_t block, int64_t total)
{
    const int64_t per = total / kXcds, more = total % kXcds;
    const int64_t x = block % kXcds, seq = block / kXcds;
    if (seq >= per + (x < more)) return -1;
    return x * per + (x < more ? x : more) + seq;
}

// The tile of workgroup `block`: row tiles of BI rows, nj column tiles.
// Positions walk blocks of kPanel row tiles column by column.  Every wave
// computes the same answer.  False: nothing is left for this workgroup.
template <int BI, int kPanel>
__device__ __forceinline__ bool find_tile(const ProductArgs& a, uint32_t block, int nj, TileRef& t)
{
    const int lane = threadIdx.x & 63;
    uint32_t first = 0;      // tiles of the groups of lanes 0 .. lane, first 64 groups
    uint32_t own = 0;
    int64_t total = 0;
    for (int c = 0; c < a.groups; c += 64) {
        uint32_t n = 0;
        if (c + lane < a.groups) {
            int64_t lo, hi;
            group_rows(a, c + lane, lo, hi);
            n = (uint32_t)((hi - lo + BI - 1) / BI);
        }
        const uint32_t s = wave_inclusive_sum(n, lane);
        if (c == 0) { first = s; own = n; }
        total += (uint32_t)__shfl((int)s, 63);
    }
    total = uniform(total);
    const int64_t p = xcd_position(block, total * nj);
    if (p < 0) return false;
    const int64_t panel = p / ((int64_t)kPanel * nj);
    const int64_t left = total - panel * kPanel;
    const int high = left < kPanel ? (int)left : kPanel;
    const int in = (int)(p - panel * kPanel * nj);
    t.j = in / high;
    int64_t m = panel * kPanel + in % high;      // row tile, over all groups
    for (int c = 0; c < a.groups; c += 64) {
        uint32_t n = own, s = first;
        if (c > 0) {
            n = 0;
            if (c + lane < a.groups) {
                int64_t lo, hi;
                group_rows(a, c + lane, lo, hi);
                n = (uint32_t)((hi - lo + BI - 1) / BI);
            }
            s = wave_inclusive_sum(n, lane);
        }
        const uint64_t hit = __builtin_amdgcn_ballot_w64((int64_t)s > m);
        if (hit) {
            const int at = __builtin_ctzll(hit);
            m -= (uint32_t)__shfl((int)(s - n), at);
            t.group = c + at;
            int64_t lo, hi;
            group_rows(a, t.group, lo, hi);
            t.row0 = uniform(lo + m * BI);
            const int64_t have = hi - t.row0;
            t.rows = uniform((int)(have < BI ? have : BI));
            t.group = uniform(t.group);
            return true;
        }
        m -= (uint32_t)__shfl((int)s, 63);
    }
    return false;
}

// Position of this workgroup where tiles differ in cost: as xcd_position,
// but within each round of `round` workgroups (those that run at a time),
// so that every XCD gets its part of every round.
__device__ __forceinline__ uint32_t round_position(uint32_t round)
{
    const uint32_t in = blockIdx.x % round, round0 = blockIdx.x - in;
    const uint32_t left = gridDim.x - round0, wide = left < round ? left : round;
    return round0 + in % kXcds * (wide / kXcds) + in / kXcds;
}

// The group of the k-th most rows (ties: the lower index first), so that the
// longest reductions start first and none of them ends the call alone; the
// k-th group as it stands where there are more than a wave's lanes.
__device__ __forceinline__ int by_rows(const ProductArgs& a, int k)
{
    if (a.groups > 64) return k;
    const int lane = threadIdx.x & 63;
    int64_t lo, hi;
    int rows = -1;
    if (lane < a.groups) {
        group_rows(a, lane, lo, hi);
        rows = (int)(hi - lo);
    }
    int rank = 0;
    for (int e = 0; e < a.groups; ++e) {
        const int other = __builtin_amdgcn_readlane(rows, e);
        rank += other > rows || (other == rows && e < lane);
    }
    return uniform((int)__builtin_ctzll(__builtin_amdgcn_ballot_w64(lane < a.groups && rank == k)));
}

// The tiles of the large kernel, `grid` of which run at a time: whole tiles of 256
// rows, and half tiles of 128.  A group's last rows make a whole tile if
// they are more than 128, a half one otherwise.  The whole tiles come
// first; those that do not fill a last round of the grid are cut into half
// tiles where that ends sooner (a half tile takes 0.55 of a whole one's time).
struct HalfTiles {
    static constexpr int kBI = 256;
    uint32_t wholes, cut, halves;   // positions: whole tiles, cut tiles' halves, half tiles

    __device__ __forceinline__ static void count(const ProductArgs& a, int e, uint32_t& w, uint32_t& h)
    {
        w = h = 0;
        if (e >= a.groups) return;
        int64_t lo, hi;
        group_rows(a, e, lo, hi);
        const int64_t rows = hi - lo, rest = rows % kBI;
        w = (uint32_t)(rows / kBI + (rest > kBI / 2));
        h = rest > 0 && rest <= kBI / 2;
    }

    __device__ __forceinline__ void init(const ProductArgs& a, uint32_t nj, uint32_t grid)
    {
        const int lane = threadIdx.x & 63;
        uint32_t nw = 0, nh = 0;
        for (int c = 0; c < a.groups; c += 64) {
            uint32_t w, h;
            count(a, c + lane, w, h);
            nw += (uint32_t)__shfl((int)wave_inclusive_sum(w, lane), 63);
            nh += (uint32_t)__shfl((int)wave_inclusive_sum(h, lane), 63);
        }
        wholes = uniform(nw) * nj;
        halves = uniform(nh) * nj;
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
        const int lane = threadIdx.x & 63;
        for (int c = 0; c < a.groups; c += 64) {
            uint32_t w, h;      // counted anew: kept, they would cost the main loop registers
            count(a, c + lane, w, h);
            const uint32_t n = is_half ? h : w, s = wave_inclusive_sum(n, lane);
            const uint64_t hit = __builtin_amdgcn_ballot_w64(s > m);
            if (hit) {
                const int at = __builtin_ctzll(hit);
                m -= (uint32_t)__shfl((int)(s - n), at);
                t.group = uniform(c + at);
                int64_t lo, hi;
                group_rows(a, t.group, lo, hi);
                // the half tile is the group's last
                t.row0 = uniform(lo + (is_half ? (hi - lo) / kBI : (int64_t)m) * kBI);
                t.rows = uniform((int)(hi - t.row0 < kBI ? hi - t.row0 : kBI));
                return true;
            }
            m -= (uint32_t)__shfl((int)s, 63);
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
        const uint32_t panel = q / (kPanel * nj);
        const uint32_t left = tiles - panel * kPanel;
        const uint32_t high = left < kPanel ? left : kPanel;
        const uint32_t in = q - panel * kPanel * nj;
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
