/*
 * aggemm.h -- streamed AllGather + GEMM on AMD Instinct MI355X (gfx950).
 *
 * C ABI of libaggemm.so.  No C++ or torch types cross this boundary: data
 * arguments are plain device pointers, sizes are int64_t, a stream is a
 * hipStream_t passed as void* (NULL = the default stream).
 *
 * The operation (PTO-ISA AllGather+GEMM README, "compute function"; the
 * Triton-distributed AllGather GEMM tutorial's reference function):
 *
 *   A = [A_0; A_1; ...; A_{n-1}]       row blocks stacked in shard order,
 *                                       shard s = rows [s*S, (s+1)*S), S = M/n
 *   C = A x B                           B: K x N, replicated
 *
 * computed as a stream: the shards other than the local one reach a
 * workspace chunk by chunk (a chunk = chunk_rows consecutive rows of one
 * shard, all of K), each chunk released by a monotonic per-source counter;
 * the GEMM starts on the local shard, which needs no wait, and consumes the
 * remote chunks in the order they are sent (PTO-ISA README, "streaming
 * pipeline" and "optimisation notes").  On one GPU every shard is a local
 * allocation; a producer kernel on a side stream plays the links.
 *
 * Result: C rows [s*S, (s+1)*S) = A_s x B for every shard s, whatever the
 * local shard, the send order, the chunk size, the mode or the pacing.
 *
 * Return values: AGG_OK (0) or a positive agg_status.  Argument errors are
 * reported synchronously and nothing is enqueued.  Kernel time-outs (a
 * counter that never reaches its value) are reported by ag_gemm_check().
 * Faults of asynchronous work surface at stream synchronisation, as in HIP.
 *
 * Threading: calls that use the library's internal workspace on one device
 * must be issued from one host thread at a time and are ordered on their
 * streams; two calls in flight on different streams of one device would
 * share the workspace and race.
 *
 * Streams (pipelined mode): the consumer GEMM runs on `stream`; the producer
 * runs on a stream of the library's own, with no event between the two
 * (unless both run in one launch on `stream`: AGG_PRODUCER_FUSED).
 * The producer reads no shard before the consumer has started (the
 * consumer's start, in `stream` order, proves that the work queued ahead of
 * the call is done; the producer waits for it on the device, for at most
 * 120 s or the call's time limit if that is longer, so work queued ahead
 * of a call does not count against the chunk waits' limit).  `stream` does
 * not wait for the producer: the consumer ends only after every chunk is
 * released, which comes after all of the producer's reads of the shards
 * and writes of the workspace.  After a failed call the producer may still
 * be running when `stream` passes the call; ag_gemm_check() waits for it.
 */
#ifndef AGGEMM_H
#define AGGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum agg_status {
    AGG_OK = 0,
    AGG_E_INVALID = 1,      /* null pointer, bad size, bad permutation ...   */
    AGG_E_UNSUPPORTED = 2,  /* K or N not a multiple of the vector width,
                               misaligned pointer, too many shards, or a
                               size past the limits below                   */
    AGG_E_NOMEM = 3,        /* workspace allocation failed                   */
    AGG_E_HIP = 4,          /* a HIP call failed while enqueueing            */
    AGG_E_TIMEOUT = 5,      /* a counter wait exceeded its limit (reported
                               by ag_gemm_check)                             */
    AGG_E_TOO_LARGE = 6     /* ag_gemm_f16_noalloc: the call needs more
                               workspace than its fixed scratch holds
                               (AGG_NOALLOC_MAX_BYTES)                       */
};

/* What one call runs (PTO-ISA README, "benchmark and output"). */
enum agg_mode {
    AGG_MODE_PIPELINED = 0,    /* producer and consumer run concurrently     */
    AGG_MODE_COMPUTE_ONLY = 1, /* consumer only; every chunk taken as ready,
                                  remote rows read from the workspace as the
                                  previous call on it left them              */
    AGG_MODE_SEQUENTIAL = 2,   /* producer finishes, then the consumer runs  */
    AGG_MODE_COPY_ONLY = 3     /* producer only; C is not written            */
};

/* How the consumer learns that rows are there. */
enum agg_scheme {
    AGG_SCHEME_COUNTERS = 0, /* per-source summary counters; the local shard
                                first, then remote tiles as their rows
                                arrive (PTO-ISA README)                   */
    AGG_SCHEME_BARRIER = 1   /* comparison scheme after the Triton-distributed
                                AllGather GEMM tutorial: iterations of
                                `pvalue` row panels of every shard; each
                                tile of an iteration, the local shard's
                                included, waits until every source has
                                delivered the iteration (a barrier in place
                                of per-source counters)                  */
};

/* What moves the remote chunks (PTO-ISA README, "AI Core resources": the
 * communication runs on engines of its own beside the compute). */
enum agg_producer {
    AGG_PRODUCER_KERNEL = 0, /* the producer kernel: compute-unit loads and
                                stores, per-piece release (default).  In a
                                pipelined call whose consumer tile has four
                                waves and at most 128 x 128 outputs, and
                                whose producer and consumer grids fit on
                                the device's CUs together, both run in one
                                launch (as AGG_PRODUCER_FUSED); otherwise as
                                AGG_PRODUCER_SEPARATE                      */
    AGG_PRODUCER_SDMA = 1,   /* the DMA engines: one copy per row group of
                                one m-tile and source, in send order, on the
                                library's stream, each followed by a stream
                                write of the source's counter (the release,
                                ordered after the copy by the stream).  No
                                compute unit moves data.  Chunks span all of
                                K; no pacing, workspace ring, trace of
                                releases or test hooks (AGG_E_UNSUPPORTED)  */
    AGG_PRODUCER_SEPARATE = 2, /* the producer kernel as a launch of its own:
                                on the library's stream in pipelined calls
                                (see "Streams" above)                      */
    AGG_PRODUCER_FUSED = 3   /* pipelined calls: producer and consumer in one
                                launch on `stream`, the producer's
                                workgroups first in the grid (one host
                                launch instead of two; the small calls are
                                bound by launch cost).  Stream order puts
                                the work ahead of the call before it, so
                                there is no start word.  Consumer tiles with
                                four waves and at most 128 x 128 outputs
                                only; no workspace ring or producer_cus
                                (AGG_E_UNSUPPORTED).  Outside the pipelined
                                mode, as AGG_PRODUCER_KERNEL              */
};

/* How the emulated links are paced when link_gbps > 0. */
enum agg_link_model {
    AGG_LINKS_PARALLEL = 0,  /* one link per source, all in parallel (full
                                mesh): chunk j of every source is released
                                no earlier than t0 + bytes(chunks 0..j)/rate */
    AGG_LINKS_SERIAL = 1     /* one link shared by all sources in send order */
};

#define AGG_MAX_SHARDS 64

typedef struct agg_options {
    uint32_t struct_size;   /* sizeof(agg_options); set by ag_gemm_options_init */
    int local_shard;        /* shard read in place, never waited on (default 0) */
    const int *send_order;  /* HOST array of the n-1 remote shard ids in send
                               order, or NULL for local+1, local+2, ... mod n */
    int mode;               /* enum agg_mode (default PIPELINED)              */
    double link_gbps;       /* per-link pacing in GB/s (1e9 B/s); 0 = none    */
    int link_model;         /* enum agg_link_model (default PARALLEL)         */
    int producer_wgs;       /* producer workgroups; 0 = automatic; a
                               pipelined call with the producer kernel on
                               every CU (no producer_cus, not fused) takes at
                               most one per CU (AGG_E_UNSUPPORTED above)      */
    int consumer_wgs;       /* consumer workgroups; 0 = automatic; at most
                               as many as can be resident at once are used */
    int tile;               /* consumer tile shape id; 0 = automatic          */
    int32_t *acc_out;       /* int8 path only: optional DEVICE int32 [M, N]
                               receiving A x B + bias before the dequant     */
    void *workspace;        /* optional caller-owned DEVICE workspace, made
                               ready once by ag_gemm_workspace_reset()       */
    size_t workspace_bytes; /* its size (>= ag_gemm_workspace_bytes(...))    */
    double timeout_ms;      /* bound on every counter wait; 0 = 2000 ms      */
    int debug_drop_chunk;   /* test hook: index (in send order) of a chunk
                               whose release is withheld; -1 = off           */
    void *consumer_events[2]; /* optional hipEvent_t pair recorded right
                                 before and after the consumer kernel, on
                                 the stream it runs on                       */
    int workspace_stages;   /* 0 (default): the workspace holds every remote
                               shard whole (S rows each).  1..8: a ring of
                               that many row panels (one consumer tile high)
                               per remote shard; the producer writes panel m
                               over panel m - stages only after the consumer
                               has finished every tile of that panel
                               (catccos page: a double-buffered workspace with
                               per-slot flags; Triton-distributed tutorial:
                               WORKSPACE_STAGES).  Needs chunks inside one
                               panel: an explicit chunk_rows must divide the
                               tile height (AGG_E_UNSUPPORTED otherwise); the
                               automatic one is cut to a divisor of it.  Not
                               with AGG_MODE_SEQUENTIAL (AGG_E_UNSUPPORTED);
                               a copy-only call does not wait for stages.
                               agg_plan_info.workspace_bytes gives the size. */
    int scheme;             /* enum agg_scheme (default COUNTERS)             */
    int pvalue;             /* barrier scheme: row panels (consumer tiles
                               high) per iteration; 0 = 1.  With a workspace
                               ring, workspace_stages must be at least this
                               (AGG_E_UNSUPPORTED otherwise): a stage is
                               reused only after the tiles of its panel,
                               which wait for their whole iteration; and a
                               ring is refused with AGG_LINKS_SERIAL, whose
                               source-by-source order would have the
                               producer wait on tiles that wait for it.     */
    uint64_t *trace;        /* optional DEVICE buffer of at least
                               agg_plan_info.trace_words uint64, 8-byte
                               aligned, receiving 100 MHz device timestamps:
                                 [0]            consumer start (its first
                                                workgroup; the consumer is
                                                launched before the producer)
                                 [1 + c]        release of producer position c
                                 [1 + C + 3p + 0..2]  consumer position p:
                                                wait start, compute start, end
                               (C = total_chunks).  Entries a call does not
                               reach keep their contents; the caller clears
                               the buffer.  A chunk's release is stamped
                               before its flag is published.                 */
    int64_t producer_piece_bytes; /* bytes a producer wave copies before it
                               counts them towards their chunk: a multiple
                               of 8192; 0 = automatic, 8192 to 65536:
                               pipelined calls about 4 pieces a chunk,
                               copy-only and sequential calls the copy's
                               bytes over the producer's waves.  Smaller pieces
                               spread a chunk over more waves, so chunks
                               land closer to their send order.  Invalid
                               (AGG_E_INVALID) if negative or not a
                               multiple of 8192; a chunk may be cut into at
                               most 2^18 pieces (AGG_E_UNSUPPORTED).        */
    int k_splits;           /* parts K is cut into per output tile (split-K):
                               each part's workgroup writes its partial sums
                               to the workspace and the last to finish adds
                               the parts in part order, then runs the
                               epilogue.  0 or 1 = no split (the automatic
                               choice; on the decode-like shapes measured
                               the unsplit small tile was faster).  > 1
                               needs the counters scheme, no workspace
                               ring, tile 3, 12, 13 or 14 (14: 32 x 256),
                               at most 64 parts and 4096 output tiles
                               (AGG_E_UNSUPPORTED otherwise).  Parts hold a
                               multiple of 256 of K, so the count used may
                               be lower (agg_plan_info.k_splits), and the
                               workspace grows by the partial sums
                               (agg_plan_info.workspace_bytes).  The sum
                               order is fixed, so results do not depend on
                               which part finishes last.                   */
    double debug_delay_us;  /* test hook: each producer piece starts after a
                               pseudo-random delay in [0, debug_delay_us]
                               (a hash of debug_delay_seed and the piece),
                               so pieces and chunks complete in an order
                               unrelated to the send order; 0 = off; must be
                               below the time limit (AGG_E_INVALID if
                               negative or not finite)                     */
    uint32_t debug_delay_seed;
    int producer;           /* enum agg_producer (default KERNEL)            */
    int producer_cus;       /* 0 (default): producer and consumer share every
                               CU.  32 or 64: in pipelined calls the
                               producer kernel runs on a stream masked to
                               that many CUs (the same number on each of
                               the 8 XCDs) and the consumer on a stream
                               masked to the others, with a grid sized to
                               them; the two are forked from and joined to
                               `stream` by events.  Other values, or with
                               SDMA: AGG_E_UNSUPPORTED (smaller masks leave
                               the remaining CUs unable to hold a full
                               consumer grid at once).  Ignored outside the
                               pipelined mode.                             */
    int64_t k_block;        /* elements of K per chunk; 0 (default): the
                               automatic choice that goes with chunk_rows 0
                               (see ag_gemm_f16), or all of K for an
                               explicit chunk_rows; >= K: a chunk spans all
                               of K.  Otherwise a chunk is
                               chunk_rows rows x one K-block of this many
                               elements (the last K-block also takes the
                               remainder of K): the chunk flag matrix of the
                               PTO-ISA README read as row groups x K-blocks.
                               A source's chunks are sent and counted
                               K-block after K-block, and a tile waits at
                               each K-block it enters, not for all of its
                               rows x K at once.  The same results, bit for
                               bit.  Needs k_block and K to be whole KiB of
                               elements (multiples of 512 for fp16/bf16, of
                               1024 for int8/fp8), at most 1024 chunks per
                               source (rows chunks x K-blocks), and the
                               counters scheme without a workspace ring or
                               split-K (AGG_E_UNSUPPORTED otherwise);
                               negative: AGG_E_INVALID.                    */
} agg_options;

/* Fill *opt with the defaults above. */
void ag_gemm_options_init(agg_options *opt);

/*
 * fp16 x fp16 -> fp32 streamed AllGather + GEMM.
 *   shards     HOST array of n_shards DEVICE pointers, each an fp16 [S, K]
 *              row-major block (S = M / n_shards), 16-byte aligned.
 *   B          DEVICE fp16 [K, N] row-major, 16-byte aligned.
 *   C          DEVICE fp32 [M, N] row-major, fully overwritten; must not
 *              alias any input.
 *   chunk_rows rows per chunk; 0 = automatic: with agg_options.k_block
 *              also 0 and K-blocks allowed (K a multiple of 4 KiB of
 *              elements, the counters scheme, no workspace ring or
 *              split-K), S/16 rows x one quarter of K (64 chunks per
 *              source), or x one eighth of K (128 chunks per source) in a
 *              pipelined call with three or more remote shards where K is
 *              a multiple of 8 KiB of elements; otherwise
 *              ag_gemm_pick_chunk_rows(S) rows x all of K.  agg_plan_info
 *              reports the choice.
 * Requires K % 8 == 0 and N % 8 == 0 (AGG_E_UNSUPPORTED otherwise).
 * Size limits (both paths, AGG_E_UNSUPPORTED past them): n_shards <= 64,
 * S <= 2^30, K <= 2^21, N <= 2^20, at most 1024 chunks per shard, and one
 * chunk (chunk_rows x K elements) below 2 GiB.
 * Inputs are read only; the caller owns every buffer.
 * PTO-ISA AllGather+GEMM README, "spec" table: A M x K fp16 (split on M
 * across ranks), B K x N fp16 (replicated), C M x N fp32.
 */
int ag_gemm_f16(const void *const *shards, int n_shards, const void *B,
                float *C, int64_t M, int64_t K, int64_t N, int chunk_rows,
                void *stream);
int ag_gemm_f16_ex(const void *const *shards, int n_shards, const void *B,
                   float *C, int64_t M, int64_t K, int64_t N, int chunk_rows,
                   void *stream, const agg_options *opt);

/*
 * ag_gemm_f16_ex for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same operation, arguments, kernels and results (bit for bit), but
 * the workspace is a fixed device array of AGG_NOALLOC_MAX_BYTES that the
 * library holds on every GPU it runs on, from the first use of its code on
 * that GPU until the process ends.  The call makes no hipMalloc or hipFree
 * and calls no allocating routine.
 *   opt         as for ag_gemm_f16_ex (may be NULL); opt->workspace must be
 *               NULL (AGG_E_INVALID otherwise).
 *   Size limit  the workspace the call needs (a counter header plus the
 *               remote shards' slots, agg_plan_info.workspace_bytes) must
 *               fit in AGG_NOALLOC_MAX_BYTES, else AGG_E_TOO_LARGE and
 *               nothing is enqueued.  With full slots that is
 *               (n_shards - 1) * S * K * 2 bytes plus about 0.8 MiB (8
 *               shards of 1024 x 4096 fit); a workspace ring
 *               (opt->workspace_stages) brings larger shapes under it.
 *   Set-up      the library's per-device set-up (run by the first call of
 *               any entry point on a device, with that device current)
 *               takes the array's address there, which loads the code that
 *               holds it, and zeroes its counter header on that call's
 *               stream (a kernel, no memset); allocation-free calls then go
 *               straight to the kernels.
 *   Sharing     every call on one GPU uses the same array, which keeps what
 *               the last call left in it: calls that overlap in time on one
 *               GPU (two streams, two host threads) race and give wrong
 *               results.  Serialise them, as for the internal workspace.
 *   Errors      as ag_gemm_f16_ex; a time-out is reported by
 *               ag_gemm_check(), which also re-arms the array's header.
 */
#define AGG_NOALLOC_MAX_BYTES ((size_t)64 << 20)
int ag_gemm_f16_noalloc(const void *const *shards, int n_shards, const void *B,
                        float *C, int64_t M, int64_t K, int64_t N,
                        int chunk_rows, void *stream, const agg_options *opt);

/*
 * bf16 x bf16 -> fp32 streamed AllGather + GEMM: the fp16 operation above
 * with bfloat16 shards and B (same layouts, alignment, size limits and
 * errors; C fp32).  A variant of the PTO-ISA README's fp16 path in the
 * other 16-bit input format.
 */
int ag_gemm_bf16(const void *const *shards, int n_shards, const void *B,
                 float *C, int64_t M, int64_t K, int64_t N, int chunk_rows,
                 void *stream);
int ag_gemm_bf16_ex(const void *const *shards, int n_shards, const void *B,
                    float *C, int64_t M, int64_t K, int64_t N, int chunk_rows,
                    void *stream, const agg_options *opt);

/*
 * fp8 x fp8 -> fp32 streamed AllGather + GEMM: the fp16 operation above
 * with OCP FP8 E4M3 shards and B (1 byte per element, the float8_e4m3fn
 * format of the FP8 grouped-GEMM variant on the Ascend SHMEM blog page).
 * Same layouts, alignment, size limits and errors as ag_gemm_f16, except
 * that K must be a multiple of 16 (one 16-byte load holds 16 elements; N
 * stays a multiple of 8); C fp32.  NaN inputs propagate as the matrix
 * cores make them.
 */
int ag_gemm_fp8(const void *const *shards, int n_shards, const void *B,
                float *C, int64_t M, int64_t K, int64_t N, int chunk_rows,
                void *stream);
int ag_gemm_fp8_ex(const void *const *shards, int n_shards, const void *B,
                   float *C, int64_t M, int64_t K, int64_t N, int chunk_rows,
                   void *stream, const agg_options *opt);

/*
 * int8 x int8 -> int32, + bias, x per-channel scale -> fp16
 * (catccos AllGatherMatmulDequant design doc, sections 1.2 and 2.2):
 *   v = A x B + bias[n]        exact int32
 *   C = fp16_rne(fp32_rne(v) * scale[n])
 *   shards  HOST array of n_shards DEVICE int8 [S, K] row-major blocks.
 *   B       DEVICE int8 [K, N] row-major.
 *   bias    DEVICE int32 [N];  scale DEVICE fp32 [N] (per output channel).
 *   C       DEVICE fp16 [M, N] row-major, fully overwritten.
 * Requires K % 16 == 0 and N % 8 == 0.  The caller guarantees that every
 * |v| < 2^31 (int32 accumulation does not saturate).
 */
int ag_gemm_i8_dequant(const int8_t *const *shards, int n_shards,
                       const int8_t *B, const int32_t *bias,
                       const float *scale, void *C, int64_t M, int64_t K,
                       int64_t N, int chunk_rows, void *stream);
int ag_gemm_i8_dequant_ex(const int8_t *const *shards, int n_shards,
                          const int8_t *B, const int32_t *bias,
                          const float *scale, void *C, int64_t M, int64_t K,
                          int64_t N, int chunk_rows, void *stream,
                          const agg_options *opt);

/*
 * Rows per chunk so that each source has 64 to 127 chunks of all of K:
 * max(1, S / 64) (PTO-ISA README, "dynamic chunk size": 64-128 chunks per
 * source).  The automatic choice for whole-K chunks; where K-blocks are
 * allowed the automatic chunks are S/16 rows x K/4 (see ag_gemm_f16).
 * Returns 0 for S < 1.
 */
int ag_gemm_pick_chunk_rows(int64_t shard_rows);

/* Bytes of workspace one call needs with full slots (workspace_stages 0):
 * a counter header plus one slot of S x K elements for every remote shard.
 * 0 on invalid sizes.  A call with a workspace ring needs less, as
 * ag_gemm_plan reports in agg_plan_info.workspace_bytes. */
size_t ag_gemm_workspace_bytes(int n_shards, int64_t M, int64_t K,
                               int elt_bytes);

/* Make a caller-owned workspace ready (zeroes its counter header on
 * `stream`); needed once after allocating it, and again before a memory
 * area that held another workspace (or anything else) is used as one.
 * The library's side stream is ordered after the reset (one event), so no
 * producer of a later call reads the header before it is zeroed.  Call
 * ag_gemm_check() after the last call that used it before freeing it.
 * A library convention (query the size, prepare, then execute), not an
 * operation of the pages. */
int ag_gemm_workspace_reset(void *workspace, size_t bytes, void *stream);

/*
 * Synchronise `stream` and the library's side stream and report whether
 * the calls issued since the last check on this device timed out
 * (AGG_E_TIMEOUT) or failed in HIP (AGG_E_HIP).  Looks only at workspaces
 * used since the last check; clears the recorded error and re-arms the
 * counters of a workspace whose call failed.
 */
int ag_gemm_check(void *stream);

/* Human-readable text for an agg_status value. */
const char *ag_gemm_status_string(int status);

/* Free the internal workspaces and side streams of every device. */
void ag_gemm_release(void);

/* ---- products of rows grouped by expert -------------------------------- *
 *
 * T rows sorted by the weights they go through: group e holds rows
 * [offsets[e], offsets[e + 1]).
 *   offsets    DEVICE int32 [n_groups + 1], not decreasing, read by the
 *              kernels (the host never waits for it).  A group may be empty.
 *              Rows before offsets[0] and from offsets[n_groups] on belong
 *              to no group: they are neither read nor written.  Values
 *              outside [0, T] are taken as 0 or T and a group that ends
 *              before it begins as empty, so no access leaves the buffers;
 *              where the values decrease, some rows' results are undefined.
 *
 * Common to the entry points below:
 *   - matrices are row-major with unit column stride; ld* is the distance
 *     of two rows in elements (at least the row's width, at most 2^21), the
 *     *_stride arguments the distance of two groups' matrices;
 *   - any K, N >= 1, any stride, and pointers aligned to their elements are
 *     taken.  Where every pointer and row starts on a 16-byte boundary and
 *     K and N are whole 16-byte pieces, the fast kernels run; otherwise one
 *     that loads element by element;
 *   - sums are held in fp32 and rounded once to the output's type, in an
 *     order that depends only on the sizes (equal calls give equal bits);
 *   - no workspace, no allocation, no state: calls may be issued from any
 *     thread to any stream and captured into a graph;
 *   - limits: T < 2^31 - 256, K and N <= 2^20, n_groups <= 65536, and fewer
 *     than 2^32 threads in the launch (AGG_E_UNSUPPORTED past them);
 *   - outputs must not alias inputs.  T = 0 is allowed.
 * ag_gemm_check() does not concern these calls: nothing in them waits.
 */
enum agg_type {           /* element types, numbered as ag_gemm_plan's kinds */
    AGG_TYPE_F16 = 0,
    AGG_TYPE_BF16 = 2,
    AGG_TYPE_FP8 = 3,     /* OCP E4M3 */
    AGG_TYPE_F32 = 4
};

/*
 * y[r, :] = x[r, :] W_e for every row r of every group e.
 *   type      AGG_TYPE_F16 or AGG_TYPE_BF16: x and w.
 *   x         DEVICE [T, K].
 *   w         DEVICE, W_e at w + e * w_stride (0: one matrix for all groups):
 *             [K, N]; with trans_w [N, K], and y = x W_e^T.
 *   y         DEVICE [T, N] of `out_type` (`type` or AGG_TYPE_F32).
 * The forward product of a layer of experts, and with the other trans_w the
 * gradient of its input (x := dy, K and N exchanged).
 */
int ag_gemm_grouped(int type, const void *x, int64_t ldx, const void *w,
                    int64_t ldw, int64_t w_stride, int trans_w,
                    const int32_t *offsets, int n_groups, void *y,
                    int64_t ldy, int out_type, int64_t T, int64_t K,
                    int64_t N, void *stream);

/*
 * dW_e = (rows of e of x)^T (rows of e of dy): the gradient of the weights.
 *   x         DEVICE [T, K];  dy  DEVICE [T, N], both of `type`.
 *   dw        DEVICE, dW_e [K, N] at dw + e * dw_stride, of `out_type` (`type`
 *             or AGG_TYPE_F32), fully overwritten; zeros for an empty group.
 * For weights kept as [N, K] exchange x and dy.
 */
int ag_gemm_grouped_wgrad(int type, const void *x, int64_t ldx,
                          const void *dy, int64_t lddy,
                          const int32_t *offsets, int n_groups, void *dw,
                          int64_t lddw, int64_t dw_stride, int out_type,
                          int64_t T, int64_t K, int64_t N, void *stream);

/*
 * c[m, n] = sum over blocks j of 128 k of
 *           a_scale[m, j] * b_scale[n / 128, j] * sum over k in j of a[m, k] b[n, k]
 *   a         DEVICE E4M3 [M, K];  a_scale  DEVICE fp32 [M, ceil(K / 128)].
 *   b         DEVICE E4M3 [N, K] (a row holds one output channel);
 *             b_scale  DEVICE fp32 [ceil(N / 128), ceil(K / 128)].
 *   c         DEVICE [M, N] of out_type: F16, BF16 or F32.
 * The last blocks along K and N may be partial.  The sum of scaled blocks is
 * held in fp32.  For F32 outputs so is each block's sum.  For 16-bit outputs a
 * block is summed by the fp8 matrix instruction, which cuts off low bits: of
 * each eight neighbouring k less than 7 * 2^-13 of the largest product
 * (operands below 2^-6 counted as 2^-6), about 1e-5 of the result for normal
 * draws.  The product of a row's and a column block's scale is a float32: below
 * 2^-126 it loses bits, past 2^128 it is infinite.
 */
int ag_gemm_fp8_block(const void *a, int64_t lda, const float *a_scale,
                      int64_t ldas, const void *b, int64_t ldb,
                      const float *b_scale, int64_t ldbs, void *c,
                      int64_t ldc, int out_type, int64_t M, int64_t K,
                      int64_t N, void *stream);

/* The same for rows grouped by expert: b [N, K] and b_scale of group e at
 * b + e * b_stride and b_scale + e * bs_stride. */
int ag_gemm_grouped_fp8_block(const void *a, int64_t lda,
                              const float *a_scale, int64_t ldas,
                              const void *b, int64_t ldb, int64_t b_stride,
                              const float *b_scale, int64_t ldbs,
                              int64_t bs_stride, const int32_t *offsets,
                              int n_groups, void *c, int64_t ldc,
                              int out_type, int64_t T, int64_t K, int64_t N,
                              void *stream);

/*
 * E4M3 codes and block scales of a matrix, as the two products take them:
 *   amax = max |x| over the block, at least 2^-100;  scale = amax / 448;
 *   q = E4M3(x * (448 / amax)), to nearest, ties to even.
 *   type        of x: F16, BF16 or F32.
 *   x           DEVICE [M, K];  q  DEVICE [M, K].
 *   block_rows  1: blocks of 1 x 128, scale [M, ceil(K / 128)] (a operand);
 *               128: blocks of 128 x 128, scale [ceil(M / 128), ceil(K / 128)]
 *               (b operand).
 * A block that holds an infinity or a NaN gets a scale that is not finite.
 */
int ag_gemm_quant_fp8_block(int type, const void *x, int64_t ldx, void *q,
                            int64_t ldq, float *scale, int64_t lds,
                            int block_rows, int64_t M, int64_t K,
                            void *stream);

/* ---- around the products: sorting by expert and back, norm ---------------- *
 *
 * The conventions of the expert products hold here too: row-major matrices
 * with unit column stride and any row stride of at most 2^21 elements (16
 * bytes a lane where every pointer and row starts on a 16-byte boundary and
 * rows are whole groups of eight, element by element otherwise), no state,
 * any thread and stream, capture into graphs, equal bits for equal calls,
 * outputs that alias no input (but for h, see ag_gemm_rmsnorm), T = 0 allowed.
 * A workspace belongs to the calls that are in flight with it: two streams, or
 * two graphs that may run at a time, need one each.
 */

/*
 * Assignments sorted by expert, in a stable order:
 *   ids        DEVICE [T, top] signed integers of `id_bytes` (4 or 8) bytes, rows
 *              ldi apart; a value outside [0, n_experts) assigns nothing (a
 *              padded or dropped token).  One expert may occur twice in a row.
 *   offsets    DEVICE int32 [n_experts + 1]: offsets[e] = number of assignments to
 *              experts below e, as the grouped products take it.
 *   place      DEVICE int32 [T, top], contiguous: the row of each assignment
 *              among the sorted ones (those of one expert in the order of
 *              (t, j)), or -1.
 *   workspace  DEVICE, 4-byte aligned, ag_gemm_expert_sort_workspace_bytes() bytes
 *              (0 up to 8192 assignments); its contents do not matter.
 * Limits: T * top < 2^31 - 256, top <= 1024, n_experts <= 4096
 * (AGG_E_UNSUPPORTED past them; the query then returns 0).
 */
size_t ag_gemm_expert_sort_workspace_bytes(int64_t T, int top, int n_experts);
int ag_gemm_expert_sort(const void *ids, int id_bytes, int64_t ldi, int64_t T,
                        int top, int n_experts, int32_t *offsets,
                        int32_t *place, void *workspace,
                        size_t workspace_bytes, void *stream);

/*
 * xs[place[t, j], :] = x[t, :]: tokens into the order of the experts.
 *   type       F16, BF16, F32 or FP8 (any one-byte values) of x [T, K] and xs
 *              [rows, K].
 *   place      as ag_gemm_expert_sort writes it.  Values outside [0, rows)
 *              name no row; no two may name the same one.
 * Rows of xs that no place names are left as they were.  The gradient of x is
 * ag_gemm_expert_combine of xs's without weights.
 */
int ag_gemm_expert_dispatch(int type, const void *x, int64_t ldx,
                            const int32_t *place, int top, void *xs,
                            int64_t ldxs, int64_t rows, int64_t T, int64_t K,
                            void *stream);

/*
 * y[t, :] = sum over j of w[t, j] * h[place[t, j], :]: the experts' results back
 * at their tokens.  A place that names no row adds nothing, whatever its weight;
 * a token without any gets zeros.
 *   type       F16, BF16 or F32 of h [rows, K]; y [T, K] of `type` or F32.
 *   w          DEVICE fp32 [T, top], or NULL: ones.
 * Sums in fp32, in the order of j, rounded once.
 */
int ag_gemm_expert_combine(int type, const void *h, int64_t ldh, int64_t rows,
                           const int32_t *place, int top, const float *w,
                           int64_t ldw, void *y, int64_t ldy, int out_type,
                           int64_t T, int64_t K, void *stream);

/*
 * Its gradient: dh[place[t, j], :] = w[t, j] * dy[t, :] and
 * dw[t, j] = sum over k of dy[t, k] * h[place[t, j], k] (0 without a place).
 *   dh         [rows, K] of `type`, or NULL; rows that no place names are left
 *              as they were.
 *   dw         fp32 [T, top], or NULL (h is then not read and may be NULL).
 */
int ag_gemm_expert_combine_grad(int type, const void *dy, int64_t lddy,
                                const void *h, int64_t ldh, int64_t rows,
                                const int32_t *place, int top, const float *w,
                                int64_t ldw, void *dh, int64_t lddh, float *dw,
                                int64_t lddw, int64_t T, int64_t K,
                                void *stream);

/*
 * Root-mean-square norm of rows, with the residual's addition:
 *   h = x + residual, rounded to `type`;  rstd = 1 / sqrt(mean(h^2) + eps);
 *   y = h * rstd * weight
 *   type       F16, BF16 or F32 of x, residual, weight, h and y.
 *   x          [T, K];  residual  [T, K], or NULL: h = x.
 *   weight     [K], or NULL: ones.
 *   h          [T, K], or NULL where it is not wanted; may be x or the residual
 *              itself (same pointer and row stride).
 *   y          [T, K], or NULL.
 *   q, scale   E4M3 codes [T, K] of y (before its rounding) and fp32 [T,
 *              ceil(K / 128)], in the form of ag_gemm_quant_fp8_block's; or both
 *              NULL.  One of y and q is wanted.  A code is the nearest to 448 y /
 *              amax with the common rstd left out (of 16-bit rows, ties that are
 *              exact go to the even code), a scale amax(h * weight) * rstd / 448.
 *              Quantising y itself, whose elements are rounded first, may decide
 *              such a tie (one code in 10^4 of bf16 rows), or a scale's last bits,
 *              the other way.
 *   rstd       fp32 [T], or NULL: what the gradient takes.
 *   eps        finite, not negative.
 * Squares are summed in fp32: of a row whose sum passes 2^128 y is 0 (finite h),
 * and with eps 0 a row below 2^-63 loses bits, one up to 2^-75 is infinite or NaN.
 */
int ag_gemm_rmsnorm(int type, const void *x, int64_t ldx, const void *residual,
                    int64_t ldr, const void *weight, void *h, int64_t ldh,
                    void *y, int64_t ldy, void *q, int64_t ldq, float *scale,
                    int64_t lds, float *rstd, float eps, int64_t T, int64_t K,
                    void *stream);

/*
 * Its gradient, with g = dy * weight:
 *   dx = rstd * (g - h * rstd^2 * mean(g * h)) + dh      (x's, and the residual's)
 *   dw = sum over rows of dy * h * rstd
 *   dh         [T, K] of `type`, or NULL: the gradient that arrives at h itself.
 *   dw         [K] of `type` or F32, or NULL; zeros for T = 0.
 *   workspace  DEVICE, 16-byte aligned, ag_gemm_rmsnorm_grad_workspace_bytes() bytes
 *              where dw is wanted; its contents do not matter.
 */
size_t ag_gemm_rmsnorm_grad_workspace_bytes(int64_t T, int64_t K);
int ag_gemm_rmsnorm_grad(int type, const void *dy, int64_t lddy, const void *h,
                         int64_t ldh, const void *weight, const float *rstd,
                         const void *dh, int64_t lddh, void *dx, int64_t lddx,
                         void *dw, int dw_type, void *workspace,
                         size_t workspace_bytes, int64_t T, int64_t K,
                         void *stream);

/* ---- microscaled 4-bit values ---------------------------------------------- *
 *
 * Rows of E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two a byte
 * with the even column in the low half, and an E8M0 scale (2^(code - 127); 255 is
 * NaN) for each 32 columns.  K is even; the last block may be partial.  Row
 * strides of codes and scales are in bytes.
 */

/*
 * Codes and scales of a matrix: scale = 2^(floor(log2(max |x|)) - 2), at least
 * 2^-127; q = E2M1(x / scale), to nearest, ties to even, magnitudes above 6 to 6.
 *   type       of x [M, K]: F16, BF16 or F32.
 *   q          [M, K / 2] bytes;  scale  [M, ceil(K / 32)] bytes.
 * A block that holds an infinity or a NaN gets scale 255 and codes 0.
 */
int ag_gemm_quant_mxfp4(int type, const void *x, int64_t ldx, void *q,
                        int64_t ldq, uint8_t *scale, int64_t lds, int64_t M,
                        int64_t K, void *stream);

/* The values of codes and scales, rounded to y's type (F16, BF16 or F32). */
int ag_gemm_dequant_mxfp4(const void *q, int64_t ldq, const uint8_t *scale,
                          int64_t lds, void *y, int64_t ldy, int type,
                          int64_t M, int64_t K, void *stream);

/*
 * c[m, n] = sum over k of a[m, k] * b[n, k], both microscaled 4-bit values.
 *   a          DEVICE [M, K / 2] bytes;  a_scale  DEVICE [M, ceil(K / 32)].
 *   b          DEVICE [N, K / 2] bytes (a row holds one output channel);
 *              b_scale  DEVICE [N, ceil(K / 32)].
 *   c          DEVICE [M, N] of out_type: F16, BF16 or F32.
 * Sums are held in fp32.  The fast kernels take K in whole blocks and codes on
 * 16-byte boundaries; rows of c on such boundaries are stored faster, and rows
 * of scales on 4-byte boundaries read a little faster (scales are read in whole
 * words: up to 3 bytes before and behind a row's own, never a word without one
 * of the matrix's).  Other codes are read byte by byte.
 */
int ag_gemm_mxfp4(const void *a, int64_t lda, const uint8_t *a_scale,
                  int64_t ldas, const void *b, int64_t ldb,
                  const uint8_t *b_scale, int64_t ldbs, void *c, int64_t ldc,
                  int out_type, int64_t M, int64_t K, int64_t N, void *stream);

/* The same for rows grouped by expert (see ag_gemm_grouped): b and b_scale of
 * group e at b + e * b_stride and b_scale + e * bs_stride bytes. */
int ag_gemm_grouped_mxfp4(const void *a, int64_t lda, const uint8_t *a_scale,
                          int64_t ldas, const void *b, int64_t ldb,
                          int64_t b_stride, const uint8_t *b_scale,
                          int64_t ldbs, int64_t bs_stride,
                          const int32_t *offsets, int n_groups, void *c,
                          int64_t ldc, int out_type, int64_t T, int64_t K,
                          int64_t N, void *stream);

/* ---- planning queries (host only, no GPU needed) ----------------------- */

typedef struct agg_plan_info {
    int64_t shard_rows;     /* S */
    int chunk_rows;         /* rows per chunk */
    int chunks_per_source;  /* ceil(S / chunk_rows) x k_blocks */
    int tile_m, tile_n;     /* consumer output tile */
    int m_tiles_per_shard;  /* ceil(S / tile_m) */
    int n_tiles;            /* ceil(N / tile_n) */
    int64_t total_tiles;    /* n_shards * m_tiles_per_shard * n_tiles
                               (times k_splits with split-K)             */
    int64_t total_chunks;   /* (n_shards - 1) * chunks_per_source */
    int consumer_wgs;       /* persistent consumer grid */
    int producer_wgs;       /* producer grid */
    int tile_id;            /* consumer tile configuration (agg_options.tile) */
    int64_t trace_words;    /* 1 + total_chunks + 3 * total_tiles          */
    int workspace_stages;   /* ring stages per remote shard (0: full slots) */
    int64_t workspace_bytes; /* workspace this call needs (a caller-owned
                                workspace must be at least this large)     */
    int k_splits;           /* parts of K per output tile (1: no split-K)   */
    int k_blocks;           /* K-blocks per row chunk (1: chunks span K)    */
    int64_t k_block;        /* elements of K per K-block (K when 1 block)   */
    int producer_fused;     /* 1: producer and consumer in one launch        */
} agg_plan_info;

/*
 * The schedule one call would run, for inspection and tests.
 *   kind: 0 = fp16 path, 1 = int8 path, 2 = bf16 path, 3 = fp8 path; num_cus: CUs of
 *   the device to plan for (0 = 256).  tile_order (nullable, capacity total_tiles * 4 int32):
 *   per consumer position: shard, m-tile, n-tile, counter value waited for
 *   before the tile's first K-block (0 for the local shard), for a grid of
 *   consumer_wgs workgroups (when its rounds do not hold whole row panels,
 *   positions walk groups of a few panels column by column, so that each
 *   XCD's stretch of a round is a compact block); with split-K the positions run part after
 *   part, each part's positions in the same order, so each (shard, m-tile,
 *   n-tile) appears once per part.  chunk_order (nullable, capacity
 *   total_chunks * 2 int32): per producer position: shard, chunk index
 *   (K-block * ceil(S / chunk_rows) + row chunk).
 */
int ag_gemm_plan(int kind, int n_shards, int64_t M, int64_t K, int64_t N,
                 int chunk_rows, const agg_options *opt, int num_cus,
                 agg_plan_info *info, int32_t *tile_order,
                 int32_t *chunk_order);

#ifdef __cplusplus
}
#endif
#endif /* AGGEMM_H */
