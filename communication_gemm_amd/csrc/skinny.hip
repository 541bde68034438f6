// skinny.hip -- grouped products with few rows a group (decoding): bound by
// the weights' bytes, so the kernels are shaped to keep many loads of w in
// flight.  A workgroup owns 16 kMB rows of a group and a strip of columns;
// its waves share r, each walking every kWaves-th piece of it with loads of
// its own (no barrier until the end), and their sums are added in wave
// order in LDS.
//
// Measured on one MI355X: 100 rows over 32 experts of [2048, 4096] fp16 82 us,
// 5.7 TB/s (28 experts' weights and the rows, each read once: 471 MB by the
// counters); 16 rows over 64 experts of [2048, 1024] bf16 11.8 us, 4.6 TB/s;
// fp8 5 x 7168 x 4096 8.4 us where the last-level cache holds the weights
// (3.5 TB/s), 10.0 from HBM, of which about 4 us are launch, finding the tile,
// the first loads' latency and the join.
#include <atomic>
#include <type_traits>

#include "device.hpp"
#include "experts.hpp"
#include "groups.hpp"
#include "launch.hpp"
#include "mfma.hpp"
#include "tile.hpp"

namespace agg {

namespace {

// The waves' accumulators (kBlocks blocks of 16 x 16) added in wave order
// and stored: thread 64 b + l holds four columns of one row of block b =
// (column block) * kMB + (row block).
template <class T, int kWaves, int kMB, int kNB>
__device__ __forceinline__ void join_and_store(float* lds, const ProductArgs& a, int64_t row0, int j0,
                                               int rows, int cols, const floatx4 (&acc)[kMB][kNB])
{
    constexpr int kBlocks = kMB * kNB;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    floatx4* all = reinterpret_cast<floatx4*>(lds);
#pragma unroll
    for (int j = 0; j < kNB; ++j)
#pragma unroll
        for (int i = 0; i < kMB; ++i) all[(wave * kBlocks + j * kMB + i) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int u = threadIdx.x; u < kBlocks * 64; u += 64 * kWaves) {
        floatx4 x = all[u];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            const floatx4 y = all[w * kBlocks * 64 + u];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] += y[e];
        }
        const int l = u & 63, b = u >> 6;
        const int row = b % kMB * 16 + (l & 15), col = b / kMB * 16 + 4 * (l >> 4);
        if (row >= rows || col >= cols) continue;   // cols: whole groups of four
        const int64_t at = (row0 + row) * a.ldc + j0 + col;
        const int t = a.out_type;
        if constexpr (T::can(kTypeF32))
            if (!(T::can(kTypeF16) || T::can(kTypeBF16)) || t == kTypeF32) {
                *reinterpret_cast<floatx4*>(reinterpret_cast<float*>(a.c) + at) = x;
                continue;
            }
        const uint32_t lo = to_bits16(x[0], t) | (uint32_t)to_bits16(x[1], t) << 16;
        const uint32_t hi = to_bits16(x[2], t) | (uint32_t)to_bits16(x[3], t) << 16;
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.c) + at) = make_uint2(lo, hi);
    }
}

// ---- weights with r along memory ([N, K]; 16-bit and E4M3) -----------------
//
// Fragments come straight from memory: 16 rows of w times 64 bytes an
// instruction, two of them a 128-byte slice.  kU slices are loaded while the
// kU before them are multiplied.

template <class T, int kMB, int kNB, int kU>
struct Batch {
    uint4 p[kU][kMB][2], q[kU][kNB][2];
    float ps[kU][kMB], qs[kU];
};

template <class T, int kMB, int kNB, int kWaves, int kU>
__global__ __launch_bounds__(64 * kWaves) void skinny_contig_kernel(ProductArgs a)
{
    constexpr int BI = 16 * kMB, BJ = 16 * kNB;
    __shared__ __attribute__((aligned(16))) float lds[kWaves * kMB * kNB * 256];
    TileRef t;
    if (!find_tile<BI, 1>(a, blockIdx.x, (a.J + BJ - 1) / BJ, t)) return;
    const int j0 = t.j * BJ;
    const int cols = a.J - j0 < BJ ? a.J - j0 : BJ;
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const int l = lane & 15, g = lane >> 4;
    const uint32_t r_bytes = (uint32_t)a.R * T::kElt;
    const __amdgpu_buffer_rsrc_t rp =
        scalar_rsrc(a.p + t.row0 * a.ldp * T::kElt, ((t.rows - 1) * a.ldp + a.R) * T::kElt);
    const __amdgpu_buffer_rsrc_t rq = scalar_rsrc(
        a.q + (t.group * a.q_stride + j0 * a.ldq) * T::kElt, ((cols - 1) * a.ldq + a.R) * T::kElt);
    const int kb = (a.R + kScaleBlock - 1) / kScaleBlock;
    const __amdgpu_buffer_rsrc_t rps =
        scalar_rsrc(a.ps + t.row0 * a.ldps, ((t.rows - 1) * a.ldps + kb) * 4);
    const __amdgpu_buffer_rsrc_t rqs =
        scalar_rsrc(a.qs + t.group * a.qs_stride + j0 / kScaleBlock * a.ldqs, kb * 4);
    uint32_t p_row[kMB], q_row[kNB];
#pragma unroll
    for (int i = 0; i < kMB; ++i) p_row[i] = (uint32_t)((16 * i + l) * a.ldp * T::kElt);
#pragma unroll
    for (int j = 0; j < kNB; ++j) q_row[j] = (uint32_t)((16 * j + l) * a.ldq * T::kElt);
    const int nk = (int)((r_bytes + 127) / 128);

    typedef Batch<T, kMB, kNB, kU> B;
    // slices first, first + kWaves, ... (past the last: out of range, zeros)
    auto load = [&](B& b, int first) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int s = first + u * kWaves;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t byte = (uint32_t)s * 128u + (uint32_t)(h * 64 + g * 16);
                const bool in = byte < r_bytes;
#pragma unroll
                for (int j = 0; j < kNB; ++j)
                    b.q[u][j][h] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                        rq, in ? q_row[j] + byte : kOutOfRange, 0, 0));
#pragma unroll
                for (int i = 0; i < kMB; ++i)
                    b.p[u][i][h] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                        rp, in ? p_row[i] + byte : kOutOfRange, 0, 0));
            }
            if constexpr (T::kElt == 1) {
                const uint32_t at = s < kb ? (uint32_t)s * 4u : kOutOfRange;
                b.qs[u] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rqs, at, 0, 0));
#pragma unroll
                for (int i = 0; i < kMB; ++i)
                    b.ps[u][i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                        rps, s < kb ? (uint32_t)((16 * i + l) * a.ldps * 4) + at : kOutOfRange, 0, 0));
            }
        }
    };
    floatx4 acc[kMB][kNB] = {};
    auto multiply = [&](const B& b) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if constexpr (T::kElt == 1) {
#pragma unroll
                for (int i = 0; i < kMB; ++i) {
                    const float s = b.ps[u][i] * b.qs[u];
#pragma unroll
                    for (int j = 0; j < kNB; ++j) {
                        const floatx4 part = T::mma({b.q[u][j][0], b.q[u][j][1]},
                                                    {b.p[u][i][0], b.p[u][i][1]}, floatx4{});
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][e] += part[e] * s;
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < kMB; ++i)
#pragma unroll
                        for (int j = 0; j < kNB; ++j)
                            acc[i][j] = T::mma({b.q[u][j][h]}, {b.p[u][i][h]}, acc[i][j]);
            }
        }
    };
    constexpr int kStep = kWaves * kU;
    B b0, b1;
    load(b0, wave);
    for (int s = wave; s < nk; s += 2 * kStep) {
        load(b1, s + kStep);
        multiply(b0);
        load(b0, s + 2 * kStep);
        multiply(b1);
    }
    join_and_store<T, kWaves, kMB, kNB>(lds, a, t.row0, j0, t.rows, cols, acc);
}

// ---- weights with r as the row index ([K, N], 16-bit) ----------------------
//
// A wave moves slabs of 32 r x 64 columns of w (128 bytes of a row, a whole
// cache line) and its rows' 32 r of x into LDS slots of its own, kSlots in
// flight, and reads w back with transpose loads.

template <class T, int kMB, int kSlots>
struct Slab {
    typedef Operand<2, 64, true> Q;
    static constexpr int kQBytes = 32 * 128;
    static constexpr int kBytes = kQBytes + kMB * 1024;
    static constexpr int kLoads = 4 + kMB;

    struct Src {
        const char* p;
        const char* q;
        int64_t ldp, ldq;
        int R, rows, cols;
    };

    struct Lane {
        uint32_t p_ld[kMB], q_ld[4];
        uint32_t p_rd;
        Reader<T, 64, true, 4> q;
    };

    // x: 16 rows of 64 bytes an instruction; 16 lanes read one piece of 16 rows
    __device__ static int swizzle(int row) { return (row >> 2) & 3; }

    __device__ static void init(Lane& L, const Src& s, int lane)
    {
#pragma unroll
        for (int u = 0; u < 4; ++u) L.q_ld[u] = Q::load_offset(u, lane, s.ldq, s.cols);
#pragma unroll
        for (int i = 0; i < kMB; ++i) {
            const int row = lane >> 2;
            L.p_ld[i] = (uint32_t)((16 * i + row) * s.ldp * 2 + (((lane & 3) ^ swizzle(row)) << 4));
        }
        L.p_rd = (uint32_t)((lane & 15) * 64 + (((lane >> 4) ^ swizzle(lane & 15)) << 4));
        L.q.init(lane, 0);
    }

    __device__ __forceinline__ static void load(char* slot, const Lane& L, const Src& s, int lane,
                                                int64_t r0)
    {
        const __amdgpu_buffer_rsrc_t rq = Q::window(s.q, s.ldq, r0, s.R, s.cols);
        const __amdgpu_buffer_rsrc_t rp = Operand<2, 16, false>::window(s.p, s.ldp, r0, s.R, s.rows);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rq, (LDS_PTR void*)(slot + u * 1024), 16,
                                                     L.q_ld[u], 0, 0, 0);
        const int piece = (lane & 3) ^ swizzle(lane >> 2);
        const bool in = r0 + piece * 8 < s.R;
#pragma unroll
        for (int i = 0; i < kMB; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rp, (LDS_PTR void*)(slot + kQBytes + i * 1024), 16,
                                                     in ? L.p_ld[i] : kOutOfRange, 0, 0, 0);
    }

    // One slab: multiplied from `cur`, whose slot is then refilled through
    // `ld` (the same memory: restrict, with the reads waited for in between,
    // keeps the compiler from making them wait for the loads in flight).
    __device__ __attribute__((always_inline)) static void step(const char* __restrict__ cur,
                                                               char* __restrict__ ld, const Lane& L,
                                                               const Src& s, int lane, int64_t r_load,
                                                               floatx4 (&acc)[kMB][4])
    {
        wait_vm_lgkm0<(kSlots - 1) * kLoads>();
        asm volatile("" ::: "memory");   // the reads below stay behind the wait
        typename T::Frag fp[kMB], fq[4];
#pragma unroll
        for (int i = 0; i < kMB; ++i)
            fp[i].v[0] = *reinterpret_cast<const uint4*>(cur + kQBytes + i * 1024 + L.p_rd);
#pragma unroll
        for (int j = 0; j < 4; ++j) fq[j] = L.q.read(cur, 0, j);
        asm volatile("" ::: "memory");   // and before this one
        wait_vm_lgkm0<63>();
        __builtin_amdgcn_sched_barrier(0);
        load(ld, L, s, lane, r_load);
#pragma unroll
        for (int i = 0; i < kMB; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = T::mma(fq[j], fp[i], acc[i][j]);
    }
};

template <class T, int kMB, int kWaves, int kSlots>
__global__ __launch_bounds__(64 * kWaves) void skinny_strided_kernel(ProductArgs a)
{
    typedef Slab<T, kMB, kSlots> S;
    constexpr int BI = 16 * kMB, BJ = 64;
    extern __shared__ __attribute__((aligned(16))) char ring[];
    TileRef t;
    if (!find_tile<BI, 1>(a, blockIdx.x, (a.J + BJ - 1) / BJ, t)) return;
    const int j0 = t.j * BJ, cols = uniform(a.J - j0);
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const typename S::Src src{a.p + t.row0 * a.ldp * 2, a.q + (t.group * a.q_stride + j0) * 2,
                              a.ldp, a.ldq, a.R, t.rows, cols};
    typename S::Lane L;
    S::init(L, src, lane);
    char* own = ring + wave * (kSlots * S::kBytes);
    const int slabs = (a.R + 31) / 32;
#pragma unroll
    for (int k = 0; k < kSlots; ++k)
        S::load(own + k * S::kBytes, L, src, lane, (int64_t)(wave + k * kWaves) * 32);
    floatx4 acc[kMB][4] = {};
    int slot = 0;
    for (int s = wave; s < slabs; s += kWaves) {
        char* at = own + slot * S::kBytes;
        S::step(at, at, L, src, lane, (int64_t)(s + kSlots * kWaves) * 32, acc);
        slot = slot == kSlots - 1 ? 0 : slot + 1;
    }
    wait_vm_lgkm0<0>();     // the loads past the end still write the slots
    __syncthreads();
    join_and_store<T, kWaves, kMB, 4>(reinterpret_cast<float*>(ring), a, t.row0, j0, t.rows,
                                   cols < BJ ? cols : BJ, acc);
}

// ---- launches -----------------------------------------------------------

template <class T, int kMB, int kNB, int kWaves, int kU>
hipError_t launch_contig(const ProductArgs& a, hipStream_t st)
{
    const int64_t nj = (a.J + 16 * kNB - 1) / (16 * kNB);
    const uint32_t grid = grid_of(row_tiles(a, 16 * kMB) * nj, 64 * kWaves);
    if (!grid) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((skinny_contig_kernel<T, kMB, kNB, kWaves, kU>), dim3(grid), dim3(64 * kWaves), 0,
                       st, a);
    return hipGetLastError();
}

template <class T, int kMB, int kWaves, int kSlots>
hipError_t launch_strided(const ProductArgs& a, hipStream_t st)
{
    constexpr int kRing = kWaves * kSlots * Slab<T, kMB, kSlots>::kBytes, kJoin = kWaves * kMB * 4 * 1024;
    constexpr int kLds = kRing > kJoin ? kRing : kJoin;
    static_assert(kLds <= 163840, "LDS");
    const uint32_t grid = grid_of(row_tiles(a, 16 * kMB) * ((a.J + 63) / 64), 64 * kWaves);
    if (!grid) return hipErrorInvalidConfiguration;
    static std::atomic<uint64_t> done{0};
    const auto kernel = skinny_strided_kernel<T, kMB, kWaves, kSlots>;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), kLds, done);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(64 * kWaves), kLds, st, a);
    return hipGetLastError();
}

// Strips of 16 columns where strips of 32 would leave CUs idle.  us, 16 / 32
// columns, weights from HBM: fp8, K 7168, N 4096, 5 rows 10.0 / 11.9; 8 groups
// of 5, K 4096, N 2048 19.9 / 18.6; bf16, K 7168, N 4096, one group of 24 and of
// 64 rows 21.6 / 32.6, 45.7 / 35.1.
// 16 rows of 16-bit weights are never better off with 32 (32 groups of 5
// rows, K 4096, N 2048: 100 / 105).  Four waves and two slices a batch, or
// eight and one, are the best of 4, 8, 16 and 1, 2, 4 (fp8, 8 groups of 5
// rows, eight waves: 15 with one slice, 15.3 with two, 22 with four).
bool narrow(const ProductArgs& a, int rows)
{
    return row_tiles(a, rows) * ((a.J + 31) / 32) < a.cus;
}

template <class T>
hipError_t launch_skinny16(const ProductArgs& a, bool q_strided, int variant, hipStream_t st)
{
    if (q_strided)
        return variant == kSkinny16 ? launch_strided<T, 1, 8, 4>(a, st) : launch_strided<T, 2, 8, 3>(a, st);
    if (variant == kSkinny16) return launch_contig<T, 1, 1, 4, 2>(a, st);
    return narrow(a, 32) ? launch_contig<T, 2, 1, 8, 1>(a, st) : launch_contig<T, 2, 2, 8, 2>(a, st);
}

template <class T>
hipError_t launch_skinny8(const ProductArgs& a, int variant, hipStream_t st)
{
    if (variant == kSkinny16)
        return narrow(a, 16) ? launch_contig<T, 1, 1, 4, 2>(a, st) : launch_contig<T, 1, 2, 8, 1>(a, st);
    return narrow(a, 32) ? launch_contig<T, 2, 1, 8, 1>(a, st) : launch_contig<T, 2, 2, 8, 2>(a, st);
}

}  // namespace

hipError_t launch_skinny(const ProductArgs& a, int type, bool q_strided, int variant, hipStream_t st)
{
    if (type == kTypeF16) return launch_skinny16<F16>(a, q_strided, variant, st);
    if (type == kTypeBF16) return launch_skinny16<BF16>(a, q_strided, variant, st);
    return a.out_type == kTypeF32 ? launch_skinny8<FP8Exact>(a, variant, st)
                                  : launch_skinny8<FP8>(a, variant, st);
}

}  // namespace agg
