// tile.hpp -- the tile engine of the expert products: one BI x BJ output
// tile, D[i, j] = sum_r P[i, r] Q[j, r], by WI x WJ waves.
//
// r is walked in slices of 128 bytes (64 16-bit or 128 fp8 values) through
// LDS rings that direct global-to-LDS loads fill: NS stages of P, NS + 1 of
// Q (256 x 256 with NS = 2: all of the 160 KiB).  Pieces of 16 bytes are
// XOR-swizzled per LDS row, by choosing which piece each lane fetches, so
// that the reads below touch every bank once.
//
// One barrier a slice.  Behind the barrier of slice t slice t + 1 is in and
// every wave is done reading slice t, so
//   P(t + NS) is loaded right behind it, into P(t)'s stage, and
//   Q(t + NS + 1) from the start of slice t + 1 on, into Q(t)'s stage:
// P has almost NS - 1 slices to land and Q almost NS.  The loads go between
// the matrix instructions, a few apart.
//
// What bounds it, and what it measured (one MI355X, 256 x 256 tiles, eight
// waves): a 64-deep slice is 2048 matrix-core cycles a SIMD, 64 KiB loaded
// into LDS and 192 KiB read from it, which at 128 bytes a cycle is as many
// LDS cycles; the three overlap imperfectly, and the board's power holds the
// clock near 1.95 GHz.  8192 x 4096 x 4096 bf16 takes 198 to 201 us (1.37
// PFLOP/s; cards differ by a few percent, and the pairs below are of one card
// each); of 200 us before the output left in parts, 165 were left without the
// loads in the loop and 185 without the LDS reads; the matrix cores are busy 62%
// of a 16384-row call.  Per tile about 8 us are not covered by other work: the
// first slices' latency, the output's stores and the next workgroup's start.
//   Loads issued at once behind the barrier: 222 us; every 2nd / 4th matrix
//     instruction with two stages of each operand: 219 / 213; with three of
//     Q: 193 to 204 by spacing (early is better than even).
//   Four waves of 128 x 128 (accumulators in AGPRs, a third fewer LDS bytes):
//     191 against 198 us where a CU computes one tile, 224 against 204 where
//     it computes two.
//   Operands read three blocks ahead, Q's set doubled (no read waited for
//     right away): 208 against 198 us.
//   Workgroups that stay and walk the tiles, the next tile's first slices
//     loaded ahead of this one's stores: the same within 1% (442 against 443
//     us for 16384 rows of eight experts, 142 for 8191 of 16).
#pragma once

#include "device.hpp"
#include "experts.hpp"
#include "mfma.hpp"

namespace agg {

namespace {

constexpr int kStoreStream = 2;   // non-temporal

// How one operand's tile of B rows (or columns) lies in global memory and
// in LDS.  kStrided false: r runs along memory; LDS holds B rows of 128
// bytes.  kStrided true (16-bit only): r is memory's row index; LDS holds 64
// rows of B values, and transpose reads hand each lane consecutive r.
template <int kElt, int B, bool kStrided>
struct Operand {
    static constexpr int kRow = kStrided ? B * kElt : 128;   // bytes of an LDS row
    static constexpr int kPieces = kRow / 16;
    static constexpr int kBytes = B * 128;
    static constexpr int kR = 128 / kElt;                    // r per slice
    static_assert(!kStrided || kElt == 2, "transpose reads of 16-bit values");

    // Swizzle of an LDS row's pieces.  r along memory: 16 lanes read one piece
    // of 16 rows, whose 128 bytes alternate between the halves of the 64
    // banks.  r-strided: a half-wave reads two pieces of rows 0..3 and 8..11.
    __device__ static int swizzle(int row)
    {
        if constexpr (!kStrided) return (row >> 1) & 7;
        if constexpr (kRow >= 256) return 2 * (row & 3) + 8 * ((row >> 3) & 1);
        return 2 * ((row >> 1) & 1) + 4 * ((row >> 3) & 1);
    }

    // LDS row and piece that lane `lane` of load instruction q fills, and
    // the piece of memory that belongs there.
    __device__ static void place(int q, int lane, int& row, int& piece)
    {
        const int pos = q * 1024 + lane * 16;
        row = pos / kRow;
        piece = ((pos % kRow) >> 4) ^ swizzle(row);
    }

    // Byte offset of that piece from the tile's origin at the slice's first
    // r; r-strided pieces past `width` (values to the matrix's edge) are
    // pushed out of range for the whole tile.
    __device__ static uint32_t load_offset(int q, int lane, int64_t ld, int width)
    {
        int row, piece;
        place(q, lane, row, piece);
        if (kStrided && piece * (16 / kElt) >= width) return kOutOfRange;
        return (uint32_t)(row * ld * kElt + piece * 16);
    }

    // Descriptor of the tile from r = r0 on: it ends with the last valid row
    // (r-contiguous: `edge` rows; r-strided: r_all), so rows past it read as
    // zeros.
    __device__ static __amdgpu_buffer_rsrc_t window(const char* origin, int64_t ld, int64_t r0,
                                                    int64_t r_all, int edge)
    {
        if constexpr (kStrided)
            return scalar_rsrc(origin + r0 * ld * kElt, ((r_all - r0 - 1) * ld + edge) * kElt);
        else
            return scalar_rsrc(origin + r0 * kElt,
                               r0 < r_all ? ((edge - 1) * ld + r_all - r0) * kElt : 0);
    }
};

// Fragment reads of one operand: T::kFrag pieces of 16 bytes a lane.
template <class T, int B, bool kStrided, int kBlocks>
struct Reader {
    typedef Operand<T::kElt, B, kStrided> O;
    // r-contiguous: one offset per piece of a slice that a lane reads (the
    // blocks are 2048 bytes apart); r-strided: one per block.
    uint32_t at[kStrided ? kBlocks : 2];

    __device__ void init(int lane, int w0)
    {
        const int g = lane >> 4, l = lane & 15;
        if constexpr (!kStrided) {
            const int row = w0 + l;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int piece = 4 * u + g;   // fp8: half u of the lane's 32 r (the two
                                               // operands' r agree; pieces 2g + u conflict)
                at[u] = (uint32_t)(row * 128 + ((piece ^ O::swizzle(row)) << 4));
            }
        } else {
            // lane group g reads rows 8g + l / 4 (and 4 on), four columns
            // each, and lane l of the group receives column l
            const int r = 8 * g + (l >> 2);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const int n = w0 + 16 * b + 4 * (l & 3);
                at[b] = (uint32_t)(r * O::kRow + (((n >> 3) ^ O::swizzle(r)) << 4) + (n & 7) * 2);
            }
        }
    }

    __device__ __forceinline__ typename T::Frag read(const char* part, int step, int b) const
    {
        typename T::Frag f;
        if constexpr (!kStrided) {
#pragma unroll
            for (int h = 0; h < T::kFrag; ++h)
                f.v[h] = *reinterpret_cast<const uint4*>(part + at[T::kElt == 2 ? step : h] + b * 2048);
        } else {
            short4_ v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (LDS_PTR short4_*)(part + at[b] + (32 * step + 4 * h) * O::kRow));
            const uint2 lo = __builtin_bit_cast(uint2, v[0]), hi = __builtin_bit_cast(uint2, v[1]);
            f.v[0] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
        return f;
    }
};

// The output tile, staged through LDS so that every store instruction
// writes whole row segments: a lane's four columns are only 8 (16-bit) or
// 16 bytes of a row.  Each wave stages its own block in its own part.
template <int kOut, int kBlocks>   // bytes of an output value, column blocks
struct Stager {
    static constexpr int kPitch = kBlocks * 16 * kOut;
    static constexpr int kPieces = kPitch / 16;
    static constexpr int kShift = kPitch >= 256 ? 0 : kPitch == 128 ? 1 : 2;

    __device__ static uint32_t at(int row, int piece)
    {
        return (uint32_t)(row * kPitch + ((piece ^ ((row >> kShift) & (kPieces - 1))) << 4));
    }
};

template <class T, int BI, int BJ, int WI, int WJ, int NS, bool kPS, bool kQS>
struct Tile {
    typedef T Type;
    static constexpr int kWaves = WI * WJ;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int kTI = BI / (16 * WI), kTJ = BJ / (16 * WJ);
    static constexpr int kR = 128 / T::kElt;
    static constexpr int kSteps = kR / T::kStep;
    typedef Operand<T::kElt, BI, kPS> P;
    typedef Operand<T::kElt, BJ, kQS> Q;
    typedef Reader<T, BI, kPS, kTI> PRead;
    typedef Reader<T, BJ, kQS, kTJ> QRead;
    static constexpr int kPLoads = BI / 8 / kWaves, kQLoads = BJ / 8 / kWaves;
    static constexpr int kLoads = kPLoads + kQLoads;     // per wave and slice
    static constexpr int kP0 = (NS + 1) * Q::kBytes;     // Q's stages, then P's
    static constexpr int kLds = kP0 + NS * P::kBytes;
    // loads that may be under way at a slice's barrier: those issued after
    // P(t + 1)'s
    static constexpr int kFlying = (NS - 1) * kQLoads + (NS - 2) * kPLoads;
    static_assert(kPLoads * kWaves * 8 == BI && kQLoads * kWaves * 8 == BJ, "loads split over the waves");
    static_assert(kWaves * 4096 <= kLds, "the output is staged in the ring");
    static_assert(NS >= 2 && kLds <= 163840 && (NS - 1) * kLoads < 64, "LDS, vmcnt range");
    // matrix instructions from one load to the next: early is better than
    // even (every 2nd and 4th: 193 us; 4th and 8th: 204; 8th and 8th: 206, on
    // 8192 x 4096 x 4096 bf16)
    static constexpr int kPEvery = kTI * kTJ >= 2 * kPLoads ? 2 : 1;
    static constexpr int kQEvery = kTI * kTJ >= 4 * kQLoads ? 4 : 1;
    static_assert(kPLoads <= kTI * kTJ && kQLoads <= kTI * kTJ, "loads between the matrix instructions");

    typedef floatx4 Acc[kTI][kTJ];

    struct Src {
        const char* p;      // the tile's first row (or column) at r = 0
        const char* q;
        int64_t ldp, ldq, r_all;
        int rows, cols;     // that exist, from the tile's origin to the edge
    };

    struct Lane {
        uint32_t p_ld[kPLoads], q_ld[kQLoads];
        PRead p;
        QRead q;
    };

    struct Window {
        __amdgpu_buffer_rsrc_t p, q;
        int left;           // r that exist from the slice's first on
    };

    __device__ static Window window(const Src& s, int64_t r0)
    {
        return {P::window(s.p, s.ldp, r0, s.r_all, s.rows), Q::window(s.q, s.ldq, r0, s.r_all, s.cols),
                (int)(s.r_all - r0 < kR ? s.r_all - r0 : kR)};
    }

    // Load u of this wave for a slice's P (or Q) part.  A piece past r_all in
    // an r-contiguous row holds the next row's values, so on the last slice it
    // is pushed out of range.
    __device__ __forceinline__ static void load_p(char* stage, const Window& w, const Lane& L,
                                                  int wave, int u)
    {
        uint32_t off = L.p_ld[u];
        if (!kPS && w.left < kR) {
            int row, piece;
            P::place(wave * kPLoads + u, threadIdx.x & 63, row, piece);
            if (piece * (16 / T::kElt) >= w.left) off = kOutOfRange;
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            w.p, (LDS_PTR void*)(stage + (wave * kPLoads + u) * 1024), 16, off, 0, 0, 0);
    }
    __device__ __forceinline__ static void load_q(char* stage, const Window& w, const Lane& L,
                                                  int wave, int u)
    {
        uint32_t off = L.q_ld[u];
        if (!kQS && w.left < kR) {
            int row, piece;
            Q::place(wave * kQLoads + u, threadIdx.x & 63, row, piece);
            if (piece * (16 / T::kElt) >= w.left) off = kOutOfRange;
        }
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            w.q, (LDS_PTR void*)(stage + (wave * kQLoads + u) * 1024), 16, off, 0, 0, 0);
    }

    __device__ static void init_lane(Lane& L, const Src& s, int wave)
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int u = 0; u < kPLoads; ++u)
            L.p_ld[u] = P::load_offset(wave * kPLoads + u, lane, s.ldp, s.rows);
#pragma unroll
        for (int u = 0; u < kQLoads; ++u)
            L.q_ld[u] = Q::load_offset(wave * kQLoads + u, lane, s.ldq, s.cols);
        L.p.init(lane, wave / WJ * (BI / WI));
        L.q.init(lane, wave % WJ * (BJ / WJ));
    }

    // The first NS slices under way, slice 0 in.
    __device__ __forceinline__ static void prologue(char* ring, const Src& s, const Lane& L, int wave)
    {
#pragma unroll
        for (int k = 0; k < NS; ++k) {
            const Window w = window(s, (int64_t)k * kR);
#pragma unroll
            for (int u = 0; u < kQLoads; ++u) load_q(ring + k * Q::kBytes, w, L, wave, u);
#pragma unroll
            for (int u = 0; u < kPLoads; ++u) load_p(ring + kP0 + k * P::kBytes, w, L, wave, u);
        }
        wait_vm_lgkm0<(NS - 1) * kLoads>();
        bare_barrier();
    }

    // ---- 16-bit values: two steps a slice ----

    struct Frags {
        typename T::Frag p[kTI], q[kTJ];
    };

    // The matrix instructions of one step on the operands in f, column block
    // by column block; each operand is re-read from step `step` of `st` once
    // its last instruction here is issued.  between(n) runs after
    // instruction n; a fence after each keeps this order.
    template <class Between>
    __device__ __forceinline__ static void roll(Frags& f, const char* sp, const char* sq, const Lane& L, int step,
                                                Acc& acc, Between between)
    {
#pragma unroll
        for (int j = 0; j < kTJ; ++j)
#pragma unroll
            for (int i = 0; i < kTI; ++i) {
                acc[i][j] = T::mma(f.q[j], f.p[i], acc[i][j]);
                if (j == kTJ - 1) f.p[i] = L.p.read(sp, step, i);
                if (i == kTI - 1) f.q[j] = L.q.read(sq, step, j);
                between(j * kTI + i);
                __builtin_amdgcn_sched_barrier(0);
            }
    }

    // One slice.  cur, nxt and ld are restrict so that the compiler does not
    // make reads wait for the loads in flight; ld is cur's memory, written
    // only behind the barrier that ends every wave's reads of cur.
    __device__ __attribute__((always_inline)) static void slice(
        const char* __restrict__ cp, const char* __restrict__ cq, const char* __restrict__ np,
        const char* __restrict__ nq, char* __restrict__ lp, char* __restrict__ lq,
        const Src& s, const Lane& L, int wave, int64_t r_load, Frags& f, Acc& acc)
    {
        const Window w = window(s, r_load);
        roll(f, cp, cq, L, 1, acc, [&](int n) {
            if (n % kQEvery == 0 && n / kQEvery < kQLoads) load_q(lq, w, L, wave, n / kQEvery);
        });
        wait_vm_lgkm0<kFlying>();
        bare_barrier();
        roll(f, np, nq, L, 0, acc, [&](int n) {
            if (n % kPEvery == 0 && n / kPEvery < kPLoads) load_p(lp, w, L, wave, n / kPEvery);
        });
    }

    __device__ __attribute__((always_inline)) static void run16(char* ring, const Src& s, Acc& acc)
    {
        const int wave = uniform((int)(threadIdx.x >> 6));
        Lane L;
        init_lane(L, s, wave);
        const int nk = (int)((s.r_all + kR - 1) / kR);
        prologue(ring, s, L, wave);
        Frags f;
#pragma unroll
        for (int j = 0; j < kTJ; ++j) f.q[j] = L.q.read(ring, 0, j);
#pragma unroll
        for (int i = 0; i < kTI; ++i) f.p[i] = L.p.read(ring + kP0, 0, i);
        int p = 0, q = 0;      // t % NS, t % (NS + 1)
        for (int t = 0; t < nk; ++t) {
            const int p1 = p == NS - 1 ? 0 : p + 1, q1 = q == NS ? 0 : q + 1, q2 = q == 0 ? NS : q - 1;
            slice(ring + kP0 + p * P::kBytes, ring + q * Q::kBytes, ring + kP0 + p1 * P::kBytes,
                  ring + q1 * Q::kBytes, ring + kP0 + p * P::kBytes, ring + q2 * Q::kBytes, s, L, wave,
                  (int64_t)(t + NS) * kR, f, acc);
            p = p1;
            q = q1;
        }
        // every load has landed and every wave is done reading: the ring may
        // be used for the output
        wait_vm_lgkm0<0>();
        bare_barrier();
    }

    // ---- E4M3: one step a slice, one scale block ----
    //
    // A block's sum starts from zero and is added to the accumulators times
    // the row's and the column block's scale, two matrix instructions behind the
    // one that made it.  The operands of a whole slice would
    // not fit beside the accumulators: P's blocks are held, Q's pass through
    // kBuf buffers, read kBuf - 1 blocks ahead.  The row scales sit in registers, four k blocks at a
    // time: lane group g loads those of blocks g * kXR .. of the wave's rows
    // (one 16-byte load a row and four slices), and each slice swaps of lane
    // halves and rows hand them to all groups.

    static constexpr int kXR = kTI >= 4 ? kTI / 4 : 1;
    static constexpr int kBuf = kTJ >= 4 ? 4 : 2;
    static_assert(kTJ % kBuf == 0, "the buffers of one slice end where the next begin");

    struct Scales {
        const float* ps;     // the tile's first row
        const float* qs;     // the column block's row
        int64_t ldps;
        int kb, rows;
    };

    struct Quad { float v[4]; };

    __device__ __forceinline__ static Quad load4(__amdgpu_buffer_rsrc_t r, uint32_t off)
    {
        return __builtin_bit_cast(Quad, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
    }

    __device__ __forceinline__ static void to_all_groups(float x, float (&out)[4])
    {
        const uint32_t b = __builtin_bit_cast(uint32_t, x);
        const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const auto q = __builtin_amdgcn_permlane16_swap(h[u], h[u], false, false);
            const uint32_t q0 = q[0], q1 = q[1];
            out[2 * u] = __builtin_bit_cast(float, q0);
            out[2 * u + 1] = __builtin_bit_cast(float, q1);
        }
    }

    struct State8 {
        typename T::Frag p[kTI], q[kBuf];
        Quad x[kXR], n[kXR], nb;     // scale products of this and the next slices; the next four
        float s[kTI];
        uint32_t x_ld[kXR];
    };

    __device__ __forceinline__ static void next_scales(State8& f, int t, __amdgpu_buffer_rsrc_t rp,
                                                       __amdgpu_buffer_rsrc_t rq)
    {
        if ((t & 3) == 3) {
#pragma unroll
            for (int r = 0; r < kXR; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) f.x[r].v[e] = f.n[r].v[e] * f.nb.v[e];
#pragma unroll
            for (int r = 0; r < kXR; ++r) f.n[r] = load4(rp, f.x_ld[r] + 4u * (uint32_t)(t + 5));
            f.nb = load4(rq, 4u * (uint32_t)(t + 5));
        } else {
#pragma unroll
            for (int r = 0; r < kXR; ++r)
#pragma unroll
                for (int e = 0; e < 3; ++e) f.x[r].v[e] = f.x[r].v[e + 1];
        }
    }

    __device__ __forceinline__ static void spread_scales(State8& f)
    {
#pragma unroll
        for (int r = 0; r < kXR; ++r) {
            float out[4];
            to_all_groups(f.x[r].v[0], out);
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (kXR * g + r < kTI) f.s[kXR * g + r] = out[g];
        }
    }

    __device__ __attribute__((always_inline)) static void slice8(
        const char* __restrict__ cq, const char* __restrict__ np, const char* __restrict__ nq,
        char* __restrict__ lp, char* __restrict__ lq, const Src& s, const Lane& L, int wave, int t,
        State8& f, Acc& acc, __amdgpu_buffer_rsrc_t rp, __amdgpu_buffer_rsrc_t rq)
    {
        constexpr int kLast = kTJ - (kBuf - 1);   // from this block on the next slice is read
        constexpr int kBefore = kLast * kTI, kAfter = kTI * kTJ - kBefore;   // instructions
        constexpr int kQ8 = kBefore >= 2 * kQLoads ? 2 : 1;
        constexpr int kP8 = kAfter >= 2 * kPLoads ? 2 : 1;
        static_assert(kBefore >= kQLoads && kAfter >= kPLoads, "loads between the matrix instructions");
        const Window w = window(s, (int64_t)(t + NS) * kR);
        floatx4 part[3];
#pragma unroll
        for (int j = 0; j < kTJ; ++j) {
            if (j == kLast) {
                wait_vm_lgkm0<kFlying>();
                bare_barrier();
                next_scales(f, t, rp, rq);
            }
            f.q[(j + kBuf - 1) % kBuf] =
                j < kLast ? L.q.read(cq, 0, j + kBuf - 1) : L.q.read(nq, 0, j - kLast);
#pragma unroll
            for (int i = 0; i < kTI; ++i) {
                const int n = j * kTI + i;
                part[n % 3] = T::mma(f.q[j % kBuf], f.p[i], floatx4{});
                __builtin_amdgcn_sched_barrier(0);   // the sums before it are scaled behind this
                if (j == kTJ - 1) f.p[i] = L.p.read(np, 0, i);
                if (n < kBefore) {
                    if (n % kQ8 == 0 && n / kQ8 < kQLoads) load_q(lq, w, L, wave, n / kQ8);
                } else if ((n - kBefore) % kP8 == 0 && (n - kBefore) / kP8 < kPLoads) {
                    load_p(lp, w, L, wave, (n - kBefore) / kP8);
                }
                if (n > 1) add(acc[(n - 2) % kTI][(n - 2) / kTI], part[(n - 2) % 3], f.s[(n - 2) % kTI]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int n = kTI * kTJ - 2; n < kTI * kTJ; ++n)
            add(acc[n % kTI][n / kTI], part[n % 3], f.s[n % kTI]);
        spread_scales(f);
    }

    __device__ __forceinline__ static void add(floatx4& acc, const floatx4& part, float scale)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += part[e] * scale;
        asm volatile("" : "+v"(acc));   // here, and not sunk behind the slice's branch
    }

    __device__ __attribute__((always_inline)) static void run8(char* ring, const Src& s,
                                                               const Scales& sc, Acc& acc)
    {
        const int lane = threadIdx.x & 63;
        const int wave = uniform((int)(threadIdx.x >> 6));
        Lane L;
        init_lane(L, s, wave);
        const int nk = (int)((s.r_all + kR - 1) / kR);
        const __amdgpu_buffer_rsrc_t rp = scalar_rsrc(sc.ps, ((sc.rows - 1) * sc.ldps + sc.kb) * 4);
        const __amdgpu_buffer_rsrc_t rq = scalar_rsrc(sc.qs, (int64_t)sc.kb * 4);
        State8 f;
#pragma unroll
        for (int r = 0; r < kXR; ++r) {
            const int row = wave / WJ * (BI / WI) + (kXR * (lane >> 4) + r) * 16 + (lane & 15);
            f.x_ld[r] = (uint32_t)(row * sc.ldps * 4);
            f.x[r] = load4(rp, f.x_ld[r]);
            f.n[r] = load4(rp, f.x_ld[r] + 16u);
        }
        f.nb = load4(rq, 0u);
        const Quad nb1 = load4(rq, 16u);
        prologue(ring, s, L, wave);
#pragma unroll
        for (int r = 0; r < kXR; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) f.x[r].v[e] *= f.nb.v[e];
        f.nb = nb1;
        spread_scales(f);
#pragma unroll
        for (int i = 0; i < kTI; ++i) f.p[i] = L.p.read(ring + kP0, 0, i);
#pragma unroll
        for (int j = 0; j < kBuf - 1; ++j) f.q[j] = L.q.read(ring, 0, j);
        int p = 0, q = 0;      // t % NS, t % (NS + 1)
        for (int t = 0; t < nk; ++t) {
            const int p1 = p == NS - 1 ? 0 : p + 1, q1 = q == NS ? 0 : q + 1, q2 = q == 0 ? NS : q - 1;
            slice8(ring + q * Q::kBytes, ring + kP0 + p1 * P::kBytes, ring + q1 * Q::kBytes,
                   ring + kP0 + p * P::kBytes, ring + q2 * Q::kBytes, s, L, wave, t, f, acc, rp, rq);
            p = p1;
            q = q1;
        }
        wait_vm_lgkm0<0>();
        bare_barrier();
    }

    // This wave's LDS accesses are done, and the compiler keeps to the order.
    __device__ __forceinline__ static void staged()
    {
        wait_vm_lgkm0<63>();
        asm volatile("" ::: "memory");
    }

    // Rows [0, rows) x columns [0, cols) of the tile to c (the tile's first
    // output), rounded to kType, through 4 KiB of LDS a wave at `stage`, a
    // part of the wave's block at a time: the first stores leave early (8192 x
    // 4096 x 4096 bf16 197 us, all staged at once 202; from registers, 64 bytes
    // of a row a store, 195, but 247 against 229 us for the 268 MB of fp32 of
    // 64 weight gradients).  cols and ldc are whole 16-byte pieces.  kStream:
    // non-temporal stores.
    template <int kType, bool kStream>
    __device__ __forceinline__ static void store(char* stage, char* c, int64_t ldc, int rows, int cols,
                                                 Acc& acc)
    {
        constexpr int kOut = kType == kTypeF32 ? 4 : 2;
        constexpr int kPJ = kTJ * 16 * kOut <= 256 ? kTJ : 256 / (16 * kOut);   // blocks of a part
        constexpr int kWant = 4096 / (16 * 16 * kOut * kPJ), kPI = kTI < kWant ? kTI : kWant;
        typedef Stager<kOut, kPJ> S;
        static_assert(kTI % kPI == 0 && kTJ % kPJ == 0 && kPI >= 1, "whole parts");
        const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
        const int wi = wave / WJ * (BI / WI), wj = wave % WJ * (BJ / WJ);
        char* own = stage + wave * 4096;
        const __amdgpu_buffer_rsrc_t rc = scalar_rsrc(c, ((rows - 1) * ldc + cols) * kOut);
        constexpr int kLanesRow = S::kPieces;            // lanes that store one row
        constexpr int kRowsPer = 64 / kLanesRow;
        const uint32_t row_out = (uint32_t)ldc * kOut;
#pragma unroll
        for (int i0 = 0; i0 < kTI; i0 += kPI)
#pragma unroll
            for (int j0 = 0; j0 < kTJ; j0 += kPJ) {
#pragma unroll
                for (int i = 0; i < kPI; ++i)
#pragma unroll
                    for (int j = 0; j < kPJ; ++j) {
                        const int row = i * 16 + (lane & 15);
                        const floatx4 x = acc[i0 + i][j0 + j];
                        if constexpr (kOut == 4) {
                            *reinterpret_cast<floatx4*>(own + S::at(row, 4 * j + (lane >> 4))) = x;
                        } else {
                            const uint32_t lo = to_bits16(x[0], kType) | (uint32_t)to_bits16(x[1], kType) << 16;
                            const uint32_t hi = to_bits16(x[2], kType) | (uint32_t)to_bits16(x[3], kType) << 16;
                            *reinterpret_cast<uint2*>(own + S::at(row, 2 * j + (lane >> 5)) +
                                                      8 * ((lane >> 4) & 1)) = make_uint2(lo, hi);
                        }
                    }
                staged();      // own part only: no barrier
                const int col = wj + j0 * 16 + lane % kLanesRow * (16 / kOut);
#pragma unroll
                for (int u = 0; u < kPI * 16 / kRowsPer; ++u) {
                    const int row = u * kRowsPer + lane / kLanesRow;
                    const uint4 v = *reinterpret_cast<const uint4*>(own + S::at(row, lane % kLanesRow));
                    const int out = wi + i0 * 16 + row;
                    const uint32_t off = out < rows && col < cols
                                             ? (uint32_t)out * row_out + (uint32_t)col * kOut : kOutOfRange;
                    __builtin_amdgcn_raw_buffer_store_b128(
                        (__attribute__((ext_vector_type(4))) unsigned int){v.x, v.y, v.z, v.w}, rc, off, 0,
                        kStream ? kStoreStream : 0);
                }
                staged();      // before the next part is written over it
            }
    }
};

}  // namespace

}  // namespace agg
