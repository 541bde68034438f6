// mx.hpp -- the matrix instruction and the tile engine of the microscaled
// 4-bit products.
#pragma once

#include <type_traits>
#include <utility>

#include "device.hpp"
#include "layers.hpp"
#include "mfma.hpp"
#include "tile.hpp"

namespace agg {

namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));

// E2M1 codes with an E8M0 scale for each 32 of r.  16 x 16 blocks: 128 r an
// instruction, lane l holds the 32 values (16 bytes) number l / 16 of row l %
// 16; 32 x 32 blocks: 64 r, number l / 32 of row l % 32.  A lane's values are one
// scale block, whose scale is byte kB of the lane's scale operand.  As in
// mfma.hpp the first operand is Q, so a lane's accumulators are four neighbouring
// columns (32 x 32: 8 q + 4 (l / 32) .., q = 0 .. 3) of one output row.
// Operands are moved as rows of 16-bit units of four values.  can(t): outputs of
// type t.  Products of two E2M1 values are multiples of 1/4 below 64, which the
// instruction adds without loss in a block; blocks whose scales differ are joined
// exactly where the result fits float32 (1 and 2^-22 in any two blocks, whole
// blocks 2^8 apart), so float32 outputs need no other form, as E4M3's do.
struct MX4 {
    static constexpr int kElt = 2, kStep = 32, kFrag = 1;
    static constexpr bool can(int t) { return t == kTypeF16 || t == kTypeBF16 || t == kTypeF32; }
    struct Frag { uint4 v[1]; };

    __device__ __forceinline__ static intx8 wide(const uint4& v)
    {
        return {(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
    }

    template <int kQB, int kPB>
    __device__ __forceinline__ static floatx4 mma(const Frag& q, const Frag& p, floatx4 c, uint32_t qs,
                                                  uint32_t ps)
    {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(q.v[0]), wide(p.v[0]), c, 4, 4, kQB,
                                                                (int)qs, kPB, (int)ps);
    }

    template <int kB>
    __device__ __forceinline__ static floatx16 mma32(const Frag& q, const Frag& p, floatx16 c, uint32_t qs,
                                                     uint32_t ps)
    {
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(q.v[0]), wide(p.v[0]), c, 4, 4, kB, (int)qs,
                                                               kB, (int)ps);
    }
};

// The E8M0 codes of `left` blocks of a dword, 0 behind them (their codes are 0
// too, but NaN times 0 is NaN).
__device__ __forceinline__ uint32_t first_scales(uint32_t v, int left)
{
    const uint32_t mask = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << 8 * left) - 1u;
    return v & mask;
}

// Where a tile's scales lie.
struct MxScales {
    const uint8_t* pe;    // the tile's first row
    const uint8_t* qe;
    int64_t ldpe, ldqe;
    int kb;               // scales of a row
};

// Rows of scales lie on dwords, or (kShift) anywhere: then a row's are read as
// the dwords they lie in, each joined with the next and shifted by the row's
// place in its first.  Only dwords that hold a scale of a tile's rows are read, so
// nothing is read across a page's end.  Rows on dwords / off them, us: 33 x 7168
// x 4096 7.6 / 8.0; 512 x 4096 x 4096 11.6 / 12.6; 8192 rows 72.5 / 74.8; 3000 rows
// of 32 experts, 2048 x 2816, 24 / 25 to 26 (equal groups).

// How far behind a dword's start p lies.
template <bool kShift>
__device__ __forceinline__ uint32_t skip_of(const uint8_t* p)
{
    return kShift ? (uint32_t)reinterpret_cast<uintptr_t>(p) & 3 : 0;
}

// The scales of `rows` rows from p on, from the dword p lies in.
template <bool kShift>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t scale_rsrc(const uint8_t* p, int64_t rows, int64_t ld, int kb)
{
    const uint32_t skip = skip_of<kShift>(p);
    return scalar_rsrc(p - skip, ((rows - 1) * ld + kb + skip + 3) & ~(int64_t)3);
}

// The four bytes from byte `skip` of lo on.
template <bool kShift>
__device__ __forceinline__ uint32_t shifted(uint32_t lo, uint32_t hi, uint32_t skip)
{
    return kShift ? __builtin_amdgcn_alignbyte(hi, lo, skip) : lo;
}

// Tile (see tile.hpp) with scales, in blocks of 32 x 32: half the operand
// registers of 16 x 16 blocks.  A slice is 256 r, four steps of 64.
//
// Scales: a slice is eight bytes of a row, and a step takes byte 2 step + h in
// the lanes of half h.  A lane fetches what kBatch / 2 slices need of its row,
// those of half 1 the later ones, a batch ahead; even and odd bytes are
// selected into two dwords, and one exchange of lane halves makes them the
// operands of a slice and of the one kBatch / 2 later, whose bytes the four
// steps take in turn.
template <int BI, int BJ, int WI, int WJ, int NS, bool kShift>
struct MxTile : Tile<MX4, BI, BJ, WI, WJ, NS, false, false> {
    typedef Tile<MX4, BI, BJ, WI, WJ, NS, false, false> Base;
    typedef typename Base::Src Src;
    typedef typename Base::Lane Lane;
    typedef typename Base::Window Window;
    typedef typename Base::P P;
    typedef typename Base::Q Q;
    static constexpr int kWI = BI / WI, kWJ = BJ / WJ;       // a wave's part
    static constexpr int kTI = kWI / 32, kTJ = kWJ / 32, kX = kTI + kTJ;
    static constexpr int kR = Base::kR, kSteps = 4;
    static constexpr int kBatch = 4;     // slices whose scales are fetched at a time
    static_assert(kTI >= 1 && kTJ >= 1 && kTI * 32 == kWI && kTJ * 32 == kWJ, "blocks of 32");
    // matrix instructions from one load to the next
    static constexpr int kQEvery = kTI * kTJ * (kSteps - 1) >= 2 * Base::kQLoads ? 2 : 1;
    static constexpr int kPEvery = kTI * kTJ >= 2 * Base::kPLoads ? 2 : 1;

    typedef floatx16 Acc[kTI][kTJ];

    struct Frags {
        MX4::Frag p[kTI], q[kTJ];
    };

    typedef MxScales Scales;

    static constexpr int kFetches = kShift ? 2 * kX : kX;     // loads of a batch

    // Scales of a batch: as fetched, and as the slices' operands.
    struct Fetched { uint32_t v[kX][kBatch + kShift]; };
    struct Batch { uint32_t v[kX][kBatch]; };

    struct ScaleLane {
        __amdgpu_buffer_rsrc_t rp, rq;
        uint32_t at[kX];
        uint32_t p_skip, q_skip;     // the same in rows 32 apart
    };

    __device__ __forceinline__ static ScaleLane scale_lane(const Src& s, const Scales& sc, int lane, int wave)
    {
        const int wi = wave / WJ * kWI, wj = wave % WJ * kWJ, cols = s.cols < BJ ? s.cols : BJ;
        const uint32_t p0 = skip_of<kShift>(sc.pe), q0 = skip_of<kShift>(sc.qe);
        ScaleLane c{scale_rsrc<kShift>(sc.pe, s.rows, sc.ldpe, sc.kb),
                    scale_rsrc<kShift>(sc.qe, cols, sc.ldqe, sc.kb), {}, 0, 0};
#pragma unroll
        for (int u = 0; u < kX; ++u) {
            const uint32_t at = u < kTI ? (uint32_t)((wi + 32 * u + (lane & 31)) * sc.ldpe) + p0
                                        : (uint32_t)((wj + 32 * (u - kTI) + (lane & 31)) * sc.ldqe) + q0;
            c.at[u] = (kShift ? at & ~3u : at) + (uint32_t)(lane >> 5) * (4 * kBatch);
            if (kShift && u == 0) c.p_skip = at & 3;
            if (kShift && u == kTI) c.q_skip = at & 3;
        }
        return c;
    }

    __device__ __forceinline__ static Fetched fetch(const ScaleLane& c, int t0)
    {
        static_assert(kBatch == 4, "16 bytes");
        Fetched b;
#pragma unroll
        for (int u = 0; u < kX; ++u) {
            const uint32_t off = c.at[u] + (uint32_t)t0 * 8u;
            const auto x = __builtin_amdgcn_raw_buffer_load_b128(u < kTI ? c.rp : c.rq, off, 0, 0);
            b.v[u][0] = x[0]; b.v[u][1] = x[1]; b.v[u][2] = x[2]; b.v[u][3] = x[3];
            if constexpr (kShift) b.v[u][4] = __builtin_amdgcn_raw_buffer_load_b32(u < kTI ? c.rp : c.rq, off + 16, 0, 0);
        }
        return b;
    }

    // The operands of slices t0 .. t0 + kBatch - 1.
    __device__ __forceinline__ static Batch operands(const Fetched& b, const ScaleLane& c, int t0, int kb)
    {
        const bool ends = 8 * (t0 + kBatch) > kb;
        const int first = 8 * t0 + ((int)(threadIdx.x & 63) >> 5) * (4 * kBatch);   // this lane's first block
        Batch o;
#pragma unroll
        for (int u = 0; u < kX; ++u)
#pragma unroll
            for (int s = 0; s < kBatch / 2; ++s) {
                const uint32_t skip = u < kTI ? c.p_skip : c.q_skip;
                uint32_t d0 = shifted<kShift>(b.v[u][2 * s], b.v[u][2 * s + 1], skip);
                uint32_t d1 = shifted<kShift>(b.v[u][2 * s + 1], b.v[u][2 * s + 1 + kShift], skip);
                if (ends) {
                    d0 = first_scales(d0, kb - first - 8 * s);
                    d1 = first_scales(d1, kb - first - 8 * s - 4);
                }
                const auto x = __builtin_amdgcn_permlane32_swap(__builtin_amdgcn_perm(d1, d0, 0x06040200u),
                                                                __builtin_amdgcn_perm(d1, d0, 0x07050301u),
                                                                false, false);
                o.v[u][s] = x[0];
                o.v[u][s + kBatch / 2] = x[1];
            }
        return o;
    }

    // Where lane reads its 16 bytes of step 0 in a part's LDS rows; step s is at
    // that xor 32 s (pieces 2 s + h, swizzled as Operand places them).
    __device__ __forceinline__ static uint32_t read_at(int lane, int w0)
    {
        const int row = w0 + (lane & 31);
        return (uint32_t)(row * 128 + (((lane >> 5) ^ P::swizzle(row)) << 4));
    }

    __device__ __forceinline__ static MX4::Frag read(const char* part, uint32_t at, int step, int b)
    {
        return {*reinterpret_cast<const uint4*>(part + (at ^ (uint32_t)(32 * step)) + b * 4096)};
    }

    // The matrix instructions of one step, each operand read again (from step
    // `next` of sp, sq) once its last one is issued.  between(n) runs behind
    // instruction n; a fence after each keeps this order.
    template <int kStep, class Between>
    __device__ __forceinline__ static void roll(Frags& f, const Batch& x, int b, const char* sp, const char* sq,
                                                uint32_t pa, uint32_t qa, int next, Acc& acc, Between between)
    {
#pragma unroll
        for (int j = 0; j < kTJ; ++j)
#pragma unroll
            for (int i = 0; i < kTI; ++i) {
                acc[i][j] = MX4::mma32<kStep>(f.q[j], f.p[i], acc[i][j], x.v[kTI + j][b], x.v[i][b]);
                if (j == kTJ - 1) f.p[i] = read(sp, pa, next, i);
                if (i == kTI - 1) f.q[j] = read(sq, qa, next, j);
                between(j * kTI + i);
                __builtin_amdgcn_sched_barrier(0);
            }
    }

    // One slice.  kExtra: loads issued since P(t + 1)'s that are not Q(t + NS)'s.
    template <int kExtra>
    __device__ __attribute__((always_inline)) static void slice(
        const char* __restrict__ cp, const char* __restrict__ cq, const char* __restrict__ np,
        const char* __restrict__ nq, char* __restrict__ lp, char* __restrict__ lq, const Src& s, const Lane& L,
        int wave, int64_t r_load, const Batch& x, int b, uint32_t pa, uint32_t qa, Frags& f, Acc& acc)
    {
        const Window w = Base::window(s, r_load);
        const auto load_q = [&](int n) __attribute__((always_inline)) {
            if (n % kQEvery == 0 && n / kQEvery < Base::kQLoads) Base::load_q(lq, w, L, wave, n / kQEvery);
        };
        constexpr int N = kTI * kTJ;
        roll<0>(f, x, b, cp, cq, pa, qa, 1, acc, [&](int n) __attribute__((always_inline)) { load_q(n); });
        roll<1>(f, x, b, cp, cq, pa, qa, 2, acc, [&](int n) __attribute__((always_inline)) { load_q(N + n); });
        roll<2>(f, x, b, cp, cq, pa, qa, 3, acc, [&](int n) __attribute__((always_inline)) { load_q(2 * N + n); });
        static_assert((Base::kQLoads - 1) * kQEvery < 3 * N, "Q's loads before the barrier");
        wait_vm_lgkm0<Base::kFlying + kExtra>();
        bare_barrier();
        roll<3>(f, x, b, np, nq, pa, qa, 0, acc, [&](int n) __attribute__((always_inline)) {
            if (n % kPEvery == 0 && n / kPEvery < Base::kPLoads) Base::load_p(lp, w, L, wave, n / kPEvery);
        });
        // those that did not fit between
#pragma unroll
        for (int u = (N + kPEvery - 1) / kPEvery; u < Base::kPLoads; ++u) Base::load_p(lp, w, L, wave, u);
        __builtin_amdgcn_sched_barrier(0);
    }

    __device__ __attribute__((always_inline)) static void run(char* ring, const Src& s, const Scales& sc, Acc& acc)
    {
        const int lane = threadIdx.x & 63;
        const int wave = uniform((int)(threadIdx.x >> 6));
        const int wi = wave / WJ * kWI, wj = wave % WJ * kWJ;
        Lane L;
        Base::init_lane(L, s, wave);
        const int nk = (int)((s.r_all + kR - 1) / kR);
        const ScaleLane c = scale_lane(s, sc, lane, wave);
        Fetched nxt = fetch(c, 0);
        Base::prologue(ring, s, L, wave);
        const uint32_t pa = read_at(lane, wi), qa = read_at(lane, wj);
        Frags f;
#pragma unroll
        for (int j = 0; j < kTJ; ++j) f.q[j] = read(ring, qa, 0, j);
#pragma unroll
        for (int i = 0; i < kTI; ++i) f.p[i] = read(ring + Base::kP0, pa, 0, i);
        int p = 0, q = 0;      // t % NS, t % (NS + 1)
        const auto one = [&](int t, const Batch& x, int b, auto extra) __attribute__((always_inline)) {
            const int p1 = p == NS - 1 ? 0 : p + 1, q1 = q == NS ? 0 : q + 1, q2 = q == 0 ? NS : q - 1;
            slice<decltype(extra)::value>(
                ring + Base::kP0 + p * P::kBytes, ring + q * Q::kBytes, ring + Base::kP0 + p1 * P::kBytes,
                ring + q1 * Q::kBytes, ring + Base::kP0 + p * P::kBytes, ring + q2 * Q::kBytes, s, L, wave,
                (int64_t)(t + NS) * kR, x, b, pa, qa, f, acc);
            p = p1;
            q = q1;
        };
        for (int t0 = 0; t0 < nk; t0 += kBatch) {
            const Batch x = operands(nxt, c, t0, sc.kb);
            __builtin_amdgcn_sched_barrier(0);
            nxt = fetch(c, t0 + kBatch);
            __builtin_amdgcn_sched_barrier(0);
            one(t0, x, 0, std::integral_constant<int, kFetches>{});
#pragma unroll
            for (int b = 1; b < kBatch; ++b) {
                if (t0 + b >= nk) break;
                one(t0 + b, x, b, std::integral_constant<int, 0>{});
            }
        }
        wait_vm_lgkm0<0>();
        bare_barrier();
    }

    // As Tile::store, for 32 x 32 blocks: rows [0, rows) x columns [0, cols) of
    // the tile to c through 4 KiB of LDS a wave, 32 rows of 128 bytes (or of 64)
    // at a time; c's rows are whole pieces of 16 bytes, or not.
    template <int kType>
    __device__ __forceinline__ static void store(char* stage, char* c, int64_t ldc, int rows, int cols, bool pieces,
                                                 Acc& acc)
    {
        constexpr int kOut = kType == kTypeF32 ? 4 : 2;
        constexpr int kPJ = kOut == 4 || kTJ == 1 ? 1 : 2;        // column blocks of a part
        typedef Stager<kOut, 2 * kPJ> S;
        static_assert(kTJ % kPJ == 0, "whole parts");
        const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
        const int wi = wave / WJ * kWI, wj = wave % WJ * kWJ;
        char* own = stage + wave * 4096;
        const __amdgpu_buffer_rsrc_t rc = scalar_rsrc(c, ((rows - 1) * ldc + cols) * kOut);
        constexpr int kLanesRow = S::kPieces, kRowsPer = 64 / kLanesRow;
        const uint32_t row_out = (uint32_t)ldc * kOut;
#pragma unroll
        for (int i = 0; i < kTI; ++i)
#pragma unroll
            for (int j0 = 0; j0 < kTJ; j0 += kPJ) {
#pragma unroll
                for (int j = 0; j < kPJ; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = lane & 31, h = lane >> 5;
                        const floatx16& x = acc[i][j0 + j];
                        if constexpr (kOut == 4) {
                            *reinterpret_cast<floatx4*>(own + S::at(row, 2 * e + h)) =
                                floatx4{x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]};
                        } else {
                            const uint32_t lo = to_bits16(x[4 * e], kType) | (uint32_t)to_bits16(x[4 * e + 1], kType) << 16;
                            const uint32_t hi = to_bits16(x[4 * e + 2], kType) | (uint32_t)to_bits16(x[4 * e + 3], kType) << 16;
                            *reinterpret_cast<uint2*>(own + S::at(row, 4 * j + e) + 8 * h) = make_uint2(lo, hi);
                        }
                    }
                Base::staged();      // own part only: no barrier
                const int col = wj + j0 * 32 + lane % kLanesRow * (16 / kOut);
#pragma unroll
                for (int u = 0; u < 32 / kRowsPer; ++u) {
                    const int row = u * kRowsPer + lane / kLanesRow;
                    const uint4 v = *reinterpret_cast<const uint4*>(own + S::at(row, lane % kLanesRow));
                    const int out = wi + i * 32 + row;
                    const uint32_t at = (uint32_t)out * row_out + (uint32_t)col * kOut;
                    if (pieces) {
                        __builtin_amdgcn_raw_buffer_store_b128(
                            (__attribute__((ext_vector_type(4))) unsigned int){v.x, v.y, v.z, v.w}, rc,
                            out < rows && col < cols ? at : kOutOfRange, 0, 0);
                        continue;
                    }
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 16 / kOut; ++e) {
                        const uint32_t off = out < rows && col + e < cols ? at + (uint32_t)e * kOut : kOutOfRange;
                        if constexpr (kOut == 4) __builtin_amdgcn_raw_buffer_store_b32(w[e], rc, off, 0, 0);
                        else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(w[e / 2] >> (16 * (e & 1))), rc, off, 0, 0);
                    }
                }
                Base::staged();      // before the next part is written over it
            }
    }
};

// f(0), f(1), ... f(N - 1) with constants (a byte of a scale operand is part of
// the instruction).
template <class F, int... I>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F f)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F f)
{
    each_of(std::make_integer_sequence<int, N>{}, f);
}

// BI x 256 tiles by eight waves (2 x 4), in blocks of 16 x 16: of operands in
// registers the 16 x 16 instruction multiplies random codes at 6.9 PFLOP/s, the one
// of 32 x 32 blocks at 6.3.  8192 x 4096 x 4096 by MxTile: 86 us; with its blocks and
// scales as here 82; 16384 x 1024 x 4096 66 against 71.
//
// Where its 78 us (67 on the fastest of several cards) go: 1 to 8 rounds of 4096 rows, K 2048,
// 4096 and 8192, N 4096 take 10 us a round and 1.82 us a slice of 256 r.  So two
// rounds' ends, stores and first loads that nothing covers, are 20 us, and 32
// slices 58, where the instruction alone would take 40.  On zeros, which the
// board's power does not slow, it is 9 us a round and 1.45 a slice (the instruction
// alone: 0.94): power is 12 of the 58, the rest of the way to the instruction's rate
// is LDS and waits.
//
// The scales go through LDS: fetched into registers by every wave that needs them,
// scattered rows of 16 to 32 bytes, they took as long in the address units as
// the codes do.  LDS: two stages of P, five halves of Q's stages (128 rows each),
// and the scales of two pairs of slices, 16 bytes a row.  In slice t the first half
// of Q(t + 2) is loaded before the barrier and behind it, when all of slice t has
// been read, its second half and P(t + 2); behind an odd slice the scales of the
// next pair but one, in the place of its own.
//
// A slice's scales reach the registers eight bytes a row, lane group g holding rows
// 16 (4 u + g) + lane % 16: [row block][r block of 32], where an instruction takes [r
// block][row block].  Two exchanges, of lane halves and of neighbouring rows of 16
// lanes, with byte selections before each, transpose the two dwords in six
// instructions; the choice of the row block is left to the matrix instruction's
// byte selectors.
//
// Pieces behind the last slice's end are not pushed out of range: both operands'
// scales of their blocks are 2^-127, and with products of at most 36 what they add
// is below half of the smallest float32.
template <int BI, bool kShift>
struct MxLargeTile : Tile<MX4, BI, 256, 2, 4, 2, false, false> {
    static constexpr int BJ = 256, WI = 2, WJ = 4;
    typedef Tile<MX4, BI, BJ, WI, WJ, 2, false, false> Base;
    typedef typename Base::Src Src;
    typedef typename Base::Window Window;
    typedef typename Base::Frags Frags;
    typedef typename Base::Acc Acc;
    typedef typename Base::P P;
    typedef MxScales Scales;
    static constexpr int kTI = Base::kTI, kTJ = Base::kTJ, kR = Base::kR, kPLoads = Base::kPLoads;
    static constexpr int kXI = kTI / 4, kXJ = kTJ / 4, kX = kXI + kXJ;
    static_assert(kTI % 4 == 0 && kTJ % 4 == 0 && Base::kQLoads == 4, "row blocks in fours, two loads a half");
    static constexpr int kHalf = 128 * 128;                       // bytes of half a stage of Q
    static constexpr int kPair = 512 * 16;                        // and of a pair's scales
    static constexpr int kP0 = 5 * kHalf, kE0 = kP0 + 2 * P::kBytes;
    static constexpr int kLds = kE0 + 2 * kPair;
    static_assert(kLds <= 163840, "LDS");

    struct Raw { uint32_t v[kX][2 + kShift]; };      // scales of a slice as they lie in memory
    struct Ops { uint32_t v[kX][2]; };               // as operands: rows of even and of odd blocks

    struct Where {
        int wave;
        uint32_t p_ld[kPLoads], q_ld[4];    // of Q, loads 0, 1: first half, 2, 3: second
        typename Base::PRead p;
        typename Base::QRead q;
        __amdgpu_buffer_rsrc_t re;          // the scales that this wave loads
        uint32_t e_ld;
        uint32_t e_p, e_q;                  // reads of those that it needs
        uint32_t p_skip, q_skip;            // in rows 64 apart the same
    };

    __device__ static void init(Where& w, const Src& s, const Scales& sc)
    {
        const int lane = threadIdx.x & 63;
        w.wave = uniform((int)(threadIdx.x >> 6));
        const int wi = w.wave / WJ * (BI / WI), wj = w.wave % WJ * (BJ / WJ);
        w.p.init(lane, wi);
        w.q.init(lane, wj & 127);
#pragma unroll
        for (int u = 0; u < kPLoads; ++u) w.p_ld[u] = P::load_offset(w.wave * kPLoads + u, lane, s.ldp, s.rows);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            w.q_ld[u] = Base::Q::load_offset(16 * (u >> 1) + 2 * w.wave + (u & 1), lane, s.ldq, s.cols);
        // 64 rows an instruction: the tile's rows (of 256; those past BI are out of
        // range) by the first four waves, its columns by the others
        const bool rows = w.wave < 4;
        const int cols = s.cols < BJ ? s.cols : BJ;
        w.re = rows ? scale_rsrc<kShift>(sc.pe, s.rows, sc.ldpe, sc.kb) : scale_rsrc<kShift>(sc.qe, cols, sc.ldqe, sc.kb);
        const uint32_t p0 = skip_of<kShift>(sc.pe), q0 = skip_of<kShift>(sc.qe);
        const uint32_t at = (uint32_t)(((w.wave & 3) * 64 + lane) * (rows ? sc.ldpe : sc.ldqe)) + (rows ? p0 : q0);
        w.e_ld = kShift ? at & ~3u : at;
        w.p_skip = ((uint32_t)((wi + lane) * sc.ldpe) + p0) & 3;
        w.q_skip = ((uint32_t)((wj + lane) * sc.ldqe) + q0) & 3;
        w.e_p = (uint32_t)(kE0 + (wi + lane) * 16);
        w.e_q = (uint32_t)(kE0 + (256 + wj + lane) * 16);
    }

    // Pair k: of slices 2 k and 2 k + 1.
    __device__ __forceinline__ static void load_scales(char* ring, const Where& w, int k)
    {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            w.re, (LDS_PTR void*)(ring + kE0 + (k & 1) * kPair + w.wave * 1024), 16, w.e_ld + (uint32_t)k * 16u, 0, 0, 0);
    }

    __device__ __forceinline__ static void read_scales(Raw& e, const char* ring, const Where& w, int t)
    {
        const char* at = ring + (t >> 1 & 1) * kPair + (t & 1) * 8;
#pragma unroll
        for (int u = 0; u < kX; ++u) {
            const uint2 v = *reinterpret_cast<const uint2*>(at + (u < kXI ? w.e_p + u * 1024 : w.e_q + (u - kXI) * 1024));
            e.v[u][0] = v.x;
            e.v[u][1] = v.y;
            // behind a pair's last dword stands the next pair's first
            if constexpr (kShift) {
                const char* nxt = t & 1 ? ring + (~(t >> 1) & 1) * kPair : at + 8;
                e.v[u][2] = *reinterpret_cast<const uint32_t*>(nxt + (u < kXI ? w.e_p + u * 1024 : w.e_q + (u - kXI) * 1024));
            }
        }
    }

    __device__ __forceinline__ static Ops operands(const Raw& e, const Where& w, int t, int kb)
    {
        Ops x;
#pragma unroll
        for (int n = 0; n < kX; ++n) {
            const uint32_t skip = n < kXI ? w.p_skip : w.q_skip;
            const uint32_t d0 = first_scales(shifted<kShift>(e.v[n][0], e.v[n][1], skip), kb - 8 * t);
            const uint32_t d1 = first_scales(shifted<kShift>(e.v[n][1], e.v[n][1 + kShift], skip), kb - 8 * t - 4);
            // bytes 0, 1 and 2, 3 of both; halves: from row blocks g % 2 and g % 2 + 2
            const auto h = __builtin_amdgcn_permlane32_swap(__builtin_amdgcn_perm(d1, d0, 0x05040100u),
                                                            __builtin_amdgcn_perm(d1, d0, 0x07060302u), false, false);
            // first and second byte of each pair
            const uint32_t h0 = h[0], h1 = h[1];
            const auto q = __builtin_amdgcn_permlane16_swap(__builtin_amdgcn_perm(h1, h0, 0x06040200u),
                                                            __builtin_amdgcn_perm(h1, h0, 0x07050301u), false, false);
            x.v[n][0] = q[0];      // row block 0 of steps 0 and 1, row block 2 of both
            x.v[n][1] = q[1];      // 1, 3
        }
        return x;
    }

    // Byte of an operand that holds the scale of row block b, step s.
    static constexpr int byte_of(int b, int s) { return (b & 2) + s; }

    // Load u of Q (of four) into half stage `to`, load u of P into stage `to`.
    __device__ __forceinline__ static void load_q(char* to, const Window& win, const Where& w, int u)
    {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(win.q, (LDS_PTR void*)(to + (2 * w.wave + (u & 1)) * 1024), 16,
                                                 w.q_ld[u], 0, 0, 0);
    }
    __device__ __forceinline__ static void load_p(char* to, const Window& win, const Where& w, int u)
    {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(win.p, (LDS_PTR void*)(to + (w.wave * kPLoads + u) * 1024), 16,
                                                 w.p_ld[u], 0, 0, 0);
    }

    // Slice t, column block by column block of its two steps: Q's blocks are read
    // three ahead, P's behind their last instruction of a step.  The barrier stands
    // where the last block of the slice has been read.  Half stage h0 takes Q(t +
    // 2)'s first half, h1 (Q(t)'s first) its second.
    __device__ __attribute__((always_inline)) static void slice(
        const char* __restrict__ cp, const char* __restrict__ cq, const char* __restrict__ np,
        const char* __restrict__ nq, char* __restrict__ lp, char* __restrict__ h0, char* __restrict__ h1,
        const char* __restrict__ scales, const Src& s, const Where& w, int t, const Ops& x, Raw& e, Frags& f, Acc& acc)
    {
        const Window win = Base::window(s, (int64_t)(t + 2) * kR);
        constexpr int kAhead = kTJ - 1, N = 2 * kTI * kTJ, kLast = N - kTI * kAhead, kLoads = kPLoads + 2;
        static_assert(kLast > 4 && kLast + 2 * kLoads <= N, "loads between the matrix instructions");
        each<N>([&](auto at) __attribute__((always_inline)) {
            constexpr int n = decltype(at)::value, step = n / (kTI * kTJ), c = n / kTI, j = c % kTJ, i = n % kTI;
            if constexpr (n == kLast) {
                wait_vm_lgkm0<2>();
                bare_barrier();
                read_scales(e, scales, w, t + 1);
            }
            if constexpr (i == 0) {
                constexpr int d = c + kAhead;
                f.q[d % kTJ] = d < 2 * kTJ ? w.q.read(cq, d / kTJ, d % kTJ) : w.q.read(nq, 0, d - 2 * kTJ);
            }
            acc[i][j] = MX4::mma<byte_of(j % 4, step), byte_of(i % 4, step)>(
                f.q[j], f.p[i], acc[i][j], x.v[kXI + j / 4][j & 1], x.v[i / 4][i & 1]);
            if constexpr (j == kTJ - 1) f.p[i] = step == 0 ? w.p.read(cp, 1, i) : w.p.read(np, 0, i);
            if constexpr (n == 0 || n == 4) load_q(h0, win, w, n / 4);
            if constexpr (n >= kLast && (n - kLast) % 2 == 0 && (n - kLast) / 2 < kLoads) {
                constexpr int u = (n - kLast) / 2;
                if constexpr (u < 2) load_q(h1, win, w, 2 + u);
                else load_p(lp, win, w, u - 2);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    }

    // The sums are made before this point: sunk behind the branches that follow,
    // they would be made without the loads between them, out of order and out of
    // registers.
    __device__ __forceinline__ static void pin(const Acc& acc)
    {
#pragma unroll
        for (int i = 0; i < kTI; ++i)
#pragma unroll
            for (int j = 0; j < kTJ; ++j) asm volatile("" ::"v"(acc[i][j]));
    }

    __device__ __attribute__((always_inline)) static void run(char* ring, const Src& s, const Scales& sc, Acc& acc)
    {
        Where w;
        init(w, s, sc);
        const int nk = (int)((s.r_all + kR - 1) / kR);
        load_scales(ring, w, 0);
        load_scales(ring, w, 1);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Window win = Base::window(s, (int64_t)k * kR);
#pragma unroll
            for (int u = 0; u < 4; ++u) load_q(ring + (2 * k + (u >> 1)) * kHalf, win, w, u);
#pragma unroll
            for (int u = 0; u < kPLoads; ++u) load_p(ring + kP0 + k * P::kBytes, win, w, u);
        }
        wait_vm_lgkm0<Base::kLoads>();
        bare_barrier();
        const int mine = w.wave % WJ / 2;      // this wave's half of Q
        Raw e;
        read_scales(e, ring, w, 0);
        Frags f;
#pragma unroll
        for (int j = 0; j < kTJ - 1; ++j) f.q[j] = w.q.read(ring + mine * kHalf, 0, j);
#pragma unroll
        for (int i = 0; i < kTI; ++i) f.p[i] = w.p.read(ring + kP0, 0, i);
        const auto half = [](int n) { return n >= 5 ? n - 5 : n; };
        int p = 0, q = 0;                      // t % 2, 2 t % 5
        for (int t = 0; t < nk; ++t) {
            slice(ring + kP0 + p * P::kBytes, ring + half(q + mine) * kHalf, ring + kP0 + (1 - p) * P::kBytes,
                  ring + half(half(q + 2) + mine) * kHalf, ring + kP0 + p * P::kBytes, ring + half(q + 4) * kHalf,
                  ring + q * kHalf, ring, s, w, t, operands(e, w, t, sc.kb), e, f, acc);
            pin(acc);
            p = 1 - p;
            q = half(q + 2);
            // every wave has read this pair's before the barrier above
            if (t & 1) load_scales(ring, w, (t >> 1) + 2);
        }
        // every load has landed and every wave is done reading: the ring may
        // be used for the output
        wait_vm_lgkm0<0>();
        bare_barrier();
    }

    // c's rows: whole pieces of 16 bytes.
    template <int kType>
    __device__ __forceinline__ static void store(char* stage, char* c, int64_t ldc, int rows, int cols, bool, Acc& acc)
    {
        Base::template store<kType, false>(stage, c, ldc, rows, cols, acc);
    }
};

// Small tiles: a step is one matrix instruction, too few to cover an LDS read,
// so a wave reads all four steps of a slice at once, a slice ahead of the matrix
// instructions (64 x 64 tiles, 2048 x 4096 x 4096: 42 us, 50 as above; tiles of
// 128 columns or rows 26 to 28 and 27).  Both operands' rings are NS stages deep; a
// stage is loaded again right behind the barrier at which every wave has read it.
//
// G groups of WI x WJ waves share r, each with a stretch of slices and a ring of
// its own, and the first adds the others' sums in their order: where a round holds
// all tiles, a call takes as long as one tile's slices do, one after the other (64
// x 64 tiles, 256 x 4096 x 4096: G 1 10.5 us, 2 9.3, 4 with two stages 10.3; 33 x
// 7168 x 4096: 14.3, 11.4, 11.8, and 8.8 as 32 x 32 tiles of eight groups).
template <int BI, int BJ, int WI, int WJ, int NS, int G, bool kShift>
struct MxSmallTile : MxTile<BI, BJ, WI, WJ, NS, kShift> {
    typedef MxTile<BI, BJ, WI, WJ, NS, kShift> Base;
    typedef typename Base::Base Loads;
    typedef typename Base::Src Src;
    typedef typename Base::Lane Lane;
    typedef typename Base::Scales Scales;
    typedef typename Base::Batch Batch;
    typedef typename Base::Acc Acc;
    static constexpr int kTI = Base::kTI, kTJ = Base::kTJ, kBatch = Base::kBatch;
    static constexpr int kWaves = Loads::kWaves, kThreads = 64 * kWaves * G;
    static constexpr int kStage = Loads::P::kBytes + Loads::Q::kBytes;
    static constexpr int kLds = G * NS * kStage;
    static constexpr int kSums = kTI * kTJ * 4096;                 // bytes of a wave's sums
    static_assert(kLds <= 163840 && kWaves * 4096 <= kLds && kWaves * kSums * G <= kLds && NS >= 2 && kSums >= 4096,
                  "LDS");

    struct Slice {
        MX4::Frag p[Base::kSteps][kTI], q[Base::kSteps][kTJ];
    };

    __device__ __forceinline__ static void read_all(Slice& f, const char* __restrict__ stage, uint32_t pa, uint32_t qa)
    {
#pragma unroll
        for (int s = 0; s < Base::kSteps; ++s) {
#pragma unroll
            for (int i = 0; i < kTI; ++i) f.p[s][i] = Base::read(stage, pa, s, i);
#pragma unroll
            for (int j = 0; j < kTJ; ++j) f.q[s][j] = Base::read(stage + Loads::P::kBytes, qa, s, j);
        }
    }

    template <int kStep>
    __device__ __forceinline__ static void multiply(const Slice& f, const Batch& x, int b, Acc& acc)
    {
#pragma unroll
        for (int j = 0; j < kTJ; ++j)
#pragma unroll
            for (int i = 0; i < kTI; ++i)
                acc[i][j] = MX4::mma32<kStep>(f.q[kStep][j], f.p[kStep][i], acc[i][j], x.v[kTI + j][b], x.v[i][b]);
    }

    __device__ __forceinline__ static void load(char* __restrict__ stage, const Src& s, const Lane& L, int wave, int t)
    {
        const typename Loads::Window w = Loads::window(s, (int64_t)t * Base::kR);
#pragma unroll
        for (int u = 0; u < Loads::kPLoads; ++u) Loads::load_p(stage, w, L, wave, u);
#pragma unroll
        for (int u = 0; u < Loads::kQLoads; ++u) Loads::load_q(stage + Loads::P::kBytes, w, L, wave, u);
    }

    // Multiplies slice t (in f) while slice t + 1 is read into g; slice t + NS is
    // loaded into slice t's stage, the same memory as `ld`.  kExtra: scale
    // fetches issued since slice t + NS - 1's loads.
    template <int kExtra>
    __device__ __attribute__((always_inline)) static void slice(
        const char* __restrict__ nxt, char* __restrict__ ld, const Src& s, const Lane& L, int wave, int t,
        const Batch& x, int b, uint32_t pa, uint32_t qa, const Slice& f, Slice& g, Acc& acc)
    {
        wait_vm_lgkm0<(NS - 2) * Loads::kLoads + kExtra>();
        bare_barrier();
        read_all(g, nxt, pa, qa);
        load(ld, s, L, wave, t + NS);
        __builtin_amdgcn_sched_barrier(0);
        multiply<0>(f, x, b, acc);
        multiply<1>(f, x, b, acc);
        multiply<2>(f, x, b, acc);
        multiply<3>(f, x, b, acc);
        __builtin_amdgcn_sched_barrier(0);
    }

    __device__ __attribute__((always_inline)) static void run(char* lds, Src s, Scales sc, Acc& acc)
    {
        const int lane = threadIdx.x & 63;
        const int all = uniform((int)(threadIdx.x >> 6)), group = all / kWaves, wave = all % kWaves;
        const int nk = (int)(((s.r_all + Base::kR - 1) / Base::kR + G - 1) / G);     // slices of each group
        const int first = group * nk;
        // what lies behind r_all is out of range, and its scales are 2^-127
        s.p += (int64_t)first * 128;
        s.q += (int64_t)first * 128;
        s.r_all -= (int64_t)first * Base::kR;
        sc.pe += first * 8;
        sc.qe += first * 8;
        sc.kb -= first * 8;
        char* ring = lds + group * (NS * kStage);
        Lane L;
        Loads::init_lane(L, s, wave);
        const typename Base::ScaleLane c = Base::scale_lane(s, sc, lane, wave);
        typename Base::Fetched nxt = Base::fetch(c, 0);
#pragma unroll
        for (int k = 0; k < NS; ++k) load(ring + k * kStage, s, L, wave, k);
        const uint32_t pa = Base::read_at(lane, wave / WJ * Base::kWI), qa = Base::read_at(lane, wave % WJ * Base::kWJ);
        wait_vm_lgkm0<(NS - 1) * Loads::kLoads>();
        bare_barrier();
        Slice f[2];
        read_all(f[0], ring, pa, qa);
        int p = 0;             // t % NS
        for (int t0 = 0; t0 < nk; t0 += kBatch) {
            const Batch x = Base::operands(nxt, c, t0, sc.kb);
            __builtin_amdgcn_sched_barrier(0);
            nxt = Base::fetch(c, t0 + kBatch);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (b && t0 + b >= nk) break;
                const int p1 = p == NS - 1 ? 0 : p + 1;
                char* now = ring + p * kStage;
                if (b == 0) slice<Base::kFetches>(ring + p1 * kStage, now, s, L, wave, t0, x, 0, pa, qa, f[0], f[1], acc);
                else slice<0>(ring + p1 * kStage, now, s, L, wave, t0 + b, x, b, pa, qa, f[b & 1], f[~b & 1], acc);
                p = p1;
            }
        }
        // every load has landed and every wave is done reading: the rings may
        // be used for the sums, and the first group's part of them for the output
        wait_vm_lgkm0<0>();
        bare_barrier();
        if constexpr (G > 1) {
            float* sums = reinterpret_cast<float*>(lds + wave * kSums) + lane;
            if (group)
#pragma unroll
                for (int i = 0; i < kTI; ++i)
#pragma unroll
                    for (int j = 0; j < kTJ; ++j)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            sums[group * (kWaves * kSums / 4) + ((i * kTJ + j) * 16 + e) * 64] = acc[i][j][e];
            wait_vm_lgkm0<63>();
            bare_barrier();
            if (group) return;
#pragma unroll
            for (int g = 1; g < G; ++g)
#pragma unroll
                for (int i = 0; i < kTI; ++i)
#pragma unroll
                    for (int j = 0; j < kTJ; ++j)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            acc[i][j][e] += sums[g * (kWaves * kSums / 4) + ((i * kTJ + j) * 16 + e) * 64];
        }
    }

    // The first group's (see run()).
    template <int kType>
    __device__ __forceinline__ static void store(char* stage, char* c, int64_t ldc, int rows, int cols, bool pieces,
                                                 Acc& acc)
    {
        if (G > 1 && threadIdx.x >= 64 * kWaves) return;
        Base::template store<kType>(stage, c, ldc, rows, cols, pieces, acc);
    }
};

}  // namespace

}  // namespace agg
