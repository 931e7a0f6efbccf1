// kvq_decode_split.cuh -- paged decode attention over an FP8 e4m3 (or BF16) KV
// cache, split along the context, with the log-sum-exp combine of the splits
// fused into the same launch (the builds without a window always, the others
// where that is faster).  Compiled three times: kvq_decode.cu (per-head
// scales, every token), kvq_decode_window.cu (the same caches behind a sliding
// window with sinks) and kvq_decode_blocks.cu (the block-scaled cache).
//
// What it computes (blog post "Smaller, faster, safer: running Kimi and GLM
// at scale", page-1 mirror section "量化KV缓存"; page-3 mirror section
// "FP8 省的不仅是显存"): decode attention whose kernel converts the FP8
// values it reads.  For query head h of request r, KV head kvh = h / g:
//   out = sum_j exp(s_j - max s) V^_j / sum_j exp(s_j - max s),
//   s_j = softmax_scale * <q, K^_j>,  K^ = e4m3 value * k_scale[kvh].
//
// One CTA per (split, KV head, request) covers every query head of the
// group, so each cache byte is fetched from HBM and converted once.  Four
// warps; each warp owns every 4th 32-token chunk of the split and a private
// 2-stage ring of shared-memory tiles filled by 2-D tensor bulk copies (TMA,
// 128-byte swizzle) that an mbarrier per stage tracks, a chunk's copies
// issued from several lanes at once; three CTAs fit on an SM, so twelve
// independent copy streams keep HBM busy.  Per chunk the warp
// runs, on the tensor cores (mma.sync m16n8k16, f16 in, fp32 accumulate),
// S^T = K Q^T with tokens as M and the g <= 8 query heads as N, an fp32
// online softmax, and O^T += V^T P^T.  e4m3 codes become f16 in registers
// (exact); movmatrix turns the score fragment into the PV operand.  The four
// warps merge in shared memory.  A request that fits in one split gets its
// output here.  Otherwise the splits merge (the combine) in one of three forms:
// when every (request, KV head)'s splits can be resident at once as one
// thread-block cluster, through distributed shared memory after a cluster
// barrier; else each split publishes (lse, o) to the workspace, and either the
// last split of the (request, KV head) to finish merges them all, counted by
// an arrival counter that it resets to zero (every build without a window, and
// balanced launches with fewer than eight resident CTAs per pair), or a second
// launch does (kvq_combine_rows.cu: every grid of splits of the windowed and
// block-scaled builds, and the other balanced launches).
//
// Window (kWindow): the query at position p sees the positions j <= p with
// j < num_sinks or j > p - window.  The kernel walks a shortened context: the
// pages that hold a sink, then the pages from the first one that the call's
// first query's window reaches; the pages between them (the hole) are never
// looked up.  In these shortened coordinates everything below is unchanged
// (splits, chunks, causal limits, the combine); only the table lookup skips
// the hole and the chunks at the window's two borders mask, per query row,
// the tokens from num_sinks to the row's window start.
//
// Block scales (kBlocks): K^ = code * 2^ek, V^ = code * 2^ev with one exponent
// per 16 tokens and KV head, so an m-tile of 16 tokens has one ek and one ev.
// ek multiplies the scores.  ev joins the exponent: with M the running
// maximum of s_j + ev_j (log2 domain), w_j = 2^(s_j + ev_j - M) <= 1 is what
// the PV product takes in f16, and l = sum_j w_j 2^-ev_j (exact powers of two
// in fp32) is the softmax's denominator in the same unit, so out = O / l and
// the split's log-sum-exp is M + log2 l: one exponential per score, no pass
// over the accumulators for the block's scale, and nothing overflows f16
// whatever the blocks' scales are.  What bounds the exponents that are read as
// they are is l (kReadValueExpMin).
#pragma once

#include <cfloat>
#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>

#include <cuda_bf16.h>

#include "kvq_internal.h"
#include "kvq_ptx.cuh"
#include "kvq_rowops.cuh"
#include "kvq_view.cuh"

namespace kvq {

namespace {

// Sticky device error word of this build of the kernel.  Bit 0: a bulk-copy
// wait timed out.  Bit 1: the drain that follows also gave up, so a copy may
// still land in the shared memory the CTA leaves behind.
__device__ unsigned int g_device_error = 0;

#ifdef KVQ_PHASE_STAMPS
// Instrumented build only (-DKVQ_PHASE_STAMPS, a library of its own): thread
// 0 of every CTA of a decode launch records %globaltimer at fixed points;
// the host reads them back after the launch (nothing is cleared in between,
// so no extra operation separates the launch from the one before it: a point
// a CTA did not reach keeps an older time than its entry).  Points:
// 0 entry, 1 the programmatic-launch wait returned, 2 warp 0's first chunk
// landed, 3 every warp done streaming, 4 in-CTA merge done, 5 the combine's
// first synchronisation passed (cluster barrier or arrival counter),
// 6 exit of a CTA that streamed.
constexpr int kStampCtas = 8192;
constexpr int kStampPoints = 8;
__device__ unsigned long long g_phase_stamps[kStampCtas * kStampPoints];
__device__ __forceinline__ void phase_stamp(int point)
{
    if (threadIdx.x == 0) {
        const unsigned cta = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
        if (cta < kStampCtas)
            g_phase_stamps[cta * kStampPoints + point] = global_timer_ns();
    }
}
#define KVQ_STAMP(p) phase_stamp(p)
#else
#define KVQ_STAMP(p) ((void)0)
#endif

constexpr int kWarps = 4;
constexpr int kCtasPerSm = 3;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxPageList = 8192 / 16 + 8;       // page ids of one split (<= 8192 tokens)
constexpr int kMaxShareTokens = 8192;             // of a balanced launch's CTA
// Published lse of a split that has no result: both are NaN, so the combine
// zeroes the request either way; the payload tells a failed tag check (the
// request is aborted and its new token not written) from a copy timeout.
constexpr uint32_t kLseInvalid = 0x7FC00000u;
constexpr uint32_t kLseStale = 0x7FC0A5A5u;

template <bool kBf16Cache, int kRingStages = 2>
struct Tile {
    static constexpr int kRowBytes = kBf16Cache ? 256 : 128;      // one token of one head
    static constexpr int kBytes = kChunkTokens * kRowBytes;       // K (or V) part of a stage
    static constexpr int kStages = kRingStages;
    static constexpr int kStageBytes = 2 * kBytes;
    static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
    static constexpr int kSmemBytes = 1024 /* alignment slack */ + kRingBytes +
                                      kWarps * kStages * 8 /* barriers */ + kMaxPageList * 4 +
                                      2 * kMaxPageList * 4 /* tags of the split's pages */ +
                                      512 /* the new token's K and V row */ + 16;
};

// Windowed builds hold no tags and no new token; the block-scaled ones keep
// the exponents of a split's blocks there (ek in the low byte, ev in the high
// one), the multi-token ones the query fragments (smem_q).  A bf16 cache's
// windowed builds give a warp one stage instead of two: the ring is half as
// large, three CTAs fit on an SM like the FP8 builds', and what one warp does
// not overlap its eleven neighbours do.
constexpr int kExpBytes = 2 * (8192 / kBlockTokens) + 16;
__host__ __device__ constexpr bool smem_q(bool multi, bool window) { return window && multi; }
template <bool kBf16, bool kWindow>
using BuildTile = Tile<kBf16, kBf16 && kWindow ? 1 : 2>;
constexpr int kQFragBytes = 8 * 2 * 32 * 8;       // [k-step][n-tile][lane] two words
template <bool kBf16, bool kMulti, bool kWindow>
constexpr int smem_bytes()
{
    if (!kWindow)
        return Tile<kBf16>::kSmemBytes;
    using T = BuildTile<kBf16, kWindow>;
    return 1024 + T::kRingBytes + kWarps * T::kStages * 8 + kMaxPageList * 4 + kExpBytes +
           (smem_q(kMulti, kWindow) ? kQFragBytes : 0);
}
// Resident CTAs per SM that the registers are compiled for.  Multi-token
// builds: 2, with both n-tiles' query fragments in registers; the windowed
// ones read them from shared memory, which leaves registers for 3.
__host__ __device__ constexpr int min_ctas(bool multi, bool window)
{
    return multi && !smem_q(multi, window) ? 2 : kCtasPerSm;
}

// Byte offset of 16-byte chunk `c` of 128-byte line `line` in a tile written
// by a 128-byte-swizzled tensor copy into a 1024-byte-aligned buffer.
__device__ __forceinline__ uint32_t swz(int line, int c)
{
    return static_cast<uint32_t>(line * 128 + ((c ^ (line & 7)) << 4));
}

// The exponent e that puts a row's largest magnitude, given as the bf16 bits
// `mx` of |q| (sign cleared), in [2^14, 2^15): e = 14 - floor(log2 |q|max),
// at most 100 (a row below 2^-86 is scaled up less; its scores are that much
// closer to 0 anyway), so that 2^e and 2^-e are normal fp32 numbers (e is at
// least -113 for finite bf16).  A row of zeros keeps e = 0.
__device__ __forceinline__ int row_pow2_exponent(uint32_t mx)
{
    if (mx == 0)
        return 0;
    const int field = static_cast<int>(mx >> 7);           // biased exponent (no sign bit)
    const int e_floor = field != 0 ? field - 127 : (31 - __clz(static_cast<int>(mx))) - 133;
    const int e = 14 - e_floor;
    return e > 100 ? 100 : e;
}

__device__ __forceinline__ uint4 lds128(const uint8_t *base, uint32_t off)
{
    return *reinterpret_cast<const uint4 *>(base + off);
}

__device__ __forceinline__ float warp_max_over_rows(float v)
{
    // lanes that share lane % 4 hold the same query heads
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
    return v;
}

__device__ __forceinline__ float warp_sum_over_rows(float v)
{
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
    return v;
}

__device__ __forceinline__ void mbar_inval(uint64_t *bar)
{
    asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void store_out(void *out, int64_t idx, float v, bool fp32)
{
    if (fp32)
        static_cast<float *>(out)[idx] = v;
    else
        static_cast<__nv_bfloat16 *>(out)[idx] = __float2bfloat16_rn(v);
}


// Query rows of one CTA: one mma n-tile (8) for a single query token, two
// (16) for the multi-token kernel.
__host__ __device__ constexpr int rows_per_cta(bool multi) { return multi ? 2 * kMaxGroup : kMaxGroup; }

// The query rows one CTA serves.  The rows of (request b, KV head kvh) are
// (token i, head h) for the request's n_query new tokens and the g query
// heads of the group, row i * g + h; a CTA takes rows row0 .. row0 + nrows - 1
// (at most rows_per_cta(kMulti)).  With one query token (kMulti false, the
// kernel compiled for that case) the rows are the group's heads, one mma
// n-tile of 8, and one CTA takes them all; the multi-token kernel gives each
// warp two n-tiles (16 rows), so every chunk's conversions serve 16 rows.
template <bool kMulti, bool kSlots>
struct Rows {
    int b, kvh, row0, nrows;
    int64_t slot;                            // this (request, KV head, row block)'s arrival counter
    int64_t base;                            // kSlots: workspace slot of its first split, or -1
    const int64_t *ids;                      // kSlots: id of every row, in shared memory

    // Row of q and out ([B][n_query][Hq][D], in units of head_dim) of local row r.
    __device__ __forceinline__ int64_t id(const DecodeArgs &a, int r) const
    {
        if constexpr (!kMulti)
            return static_cast<int64_t>(b) * a.num_q_heads + kvh * a.group + r;
        const int rr = row0 + r;
        return (static_cast<int64_t>(b) * a.n_query + rr / a.group) * a.num_q_heads + kvh * a.group +
               rr % a.group;
    }

    // Place of local row r of split s among the workspace's partials (an lse
    // each, and head_dim floats of output).  A balanced launch gives every
    // split of the launch a slot of rows_per_cta rows of its own.
    __device__ __forceinline__ int64_t part(const DecodeArgs &a, int r, int s) const
    {
        if constexpr (kSlots)
            return base >= 0 ? (base + s) * rows_per_cta(kMulti) + r : ids[r] * a.max_splits + s;
        return id(a, r) * a.max_splits + s;
    }

    // Distance of a row's partials of consecutive splits (kSlots, where splits
    // merge by arrival: a balanced launch).
    __device__ __forceinline__ int64_t part_step() const { return rows_per_cta(kMulti); }

    __device__ __forceinline__ int64_t out_row(const DecodeArgs &a, int r) const
    {
        if constexpr (kSlots)
            return ids[r];
        return id(a, r);
    }
};

__device__ __forceinline__ void store_out4(void *out, int64_t idx, float4 v, bool fp32)
{
    if (fp32)
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + idx) = v;
    else
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(out) + idx) =
            make_uint2(f32x2_to_bf16x2(v.x, v.y), f32x2_to_bf16x2(v.z, v.w));
}

// The warps' merge area holds one row of 128 floats per (warp, head).  Row
// stride and a skew of 2 words per 32 dims make the fragment stores (a lane
// writes dims 16*(lane/4) + 2i, +1 of heads 2*(lane%4), +1) hit 16 distinct
// bank pairs per half-warp, and keep the row reads (thread d) conflict-free.
constexpr int kMergeStride = 146;                 // >= 128 + 6, == 2 (mod 16)
__device__ __forceinline__ int merge_col(int d) { return d + 2 * (d >> 5); }


// Shared-memory offset (in floats) of the cluster partial: just past the
// warps' merge area, inside the ring (idle by then).  The workspace combine's
// scratch starts at offset 0: it runs after the CTA's own partial has left
// the merge area for global memory.
__host__ __device__ constexpr int scratch_offset(bool multi)
{
    return (kWarps * rows_per_cta(multi) * kMergeStride + 3 * kWarps * rows_per_cta(multi) +
            2 * rows_per_cta(multi) + 3) / 4 * 4;
}
constexpr int kScratchOffset = scratch_offset(false);
static_assert((kMaxGroup + kMaxGroup * kMaxSplitsTotal) * 4 <= Tile<false>::kRingBytes,
              "the workspace combine's scratch fits in the idle ring");
static_assert((2 * kMaxGroup + 2 * kMaxGroup * kMultiMaxSplitsPerRequest) * 4 <= Tile<false>::kRingBytes,
              "the multi-token workspace combine's scratch fits in the idle ring");
static_assert((kScratchOffset + kMaxGroup + kMaxGroup * kHeadDim) * 4 <= Tile<false>::kRingBytes,
              "the cluster combine's partial fits in the idle ring");
static_assert((scratch_offset(true) + 2 * kMaxGroup + 2 * kMaxGroup * kHeadDim) * 4 <= Tile<false>::kRingBytes,
              "the multi-token cluster partial fits in the idle ring");

// Count this split's arrival for (request b, KV head kvh).  The last split
// to arrive merges the partials of all nsplit splits of the group:
//   M = max_s lse_s,  out = sum_s 2^(lse_s - M) o_s / sum_s 2^(lse_s - M),
// for every query head of the group at once, writes the output (zeros for
// a head if any split was invalid) and resets the counter.
// kvq_decode_step, once per (request, KV head), by the CTA that knows the
// verdict of all the request's splits: KV head 0 writes the abort flag, and
// a request that passed gets its new token written for this KV head (the
// codes kvq_append writes).  A split holding the token has already patched
// them into its own tile, and no other CTA of this launch reads that row.
__device__ void finish_step(const DecodeArgs &a, int b, int kvh, bool stale)
{
    if (kvh == 0 && threadIdx.x == 0)
        a.abort_out[b] = stale ? 1 : 0;
    if (stale || threadIdx.x >= 32)
        return;
    const int lane = threadIdx.x;
    const int64_t tpos = static_cast<int64_t>(a.seq_lens[b]) - 1;     // > 0: the request was not empty
    const int32_t page = a.block_table[static_cast<int64_t>(b) * a.max_pages_per_seq + tpos / a.page_size];
    if (page < 0 || page >= a.num_pages)                                 // excluded by the check
        return;
    const int64_t row = (static_cast<int64_t>(page) * a.num_kv_heads + kvh) * a.page_size + tpos % a.page_size;
    const int64_t src = (static_cast<int64_t>(b) * a.num_kv_heads + kvh) * kHeadDim + 4 * lane;
    const uint2 xk = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.k_new) + src);
    const uint2 xv = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.v_new) + src);
    if (a.bf16_cache) {
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.k_cache) + row * 256 + 8 * lane) = xk;
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.v_cache) + row * 256 + 8 * lane) = xv;
    } else {
        *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.k_cache) + row * 128 + 4 * lane) =
            encode4_e4m3(xk.x, xk.y, a.k_scale[kvh]);
        *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.v_cache) + row * 128 + 4 * lane) =
            encode4_e4m3(xv.x, xv.y, a.v_scale[kvh]);
    }
}

// kNanFlows (the windowed and block-scaled builds): a NaN score or value of a
// visible token reaches its row's output whatever the splits are; such a split
// publishes lse = +inf, which makes the weights and their sum NaN here.
template <bool kMulti, bool kNanFlows>
__device__ void publish_and_combine(const DecodeArgs &a, const Rows<kMulti, kNanFlows> &R, int nsplit, float *scratch)
{
    if (kNanFlows && a.combine_apart)                      // launch_combine_rows does it
        return;
    __shared__ int s_last;
    // The block barrier orders every thread's partial before thread 0's
    // release; the last split's acquire, then its barrier, orders all the
    // peers' partials before its loads (the counter is the only
    // synchronisation between the splits).
    __syncthreads();
    unsigned int *counter = a.counters + R.slot;
    if (threadIdx.x == 0)
        s_last = atom_add_acq_rel_gpu(counter, 1u) == static_cast<unsigned int>(nsplit - 1);
    __syncthreads();
    KVQ_STAMP(5);
    if (!s_last)
        return;
    constexpr int kRowsT = rows_per_cta(kMulti);
    const int g = R.nrows, n = nsplit;
    if constexpr (kNanFlows) {
        // Few splits: every lse and partial in one trip to L2, each thread
        // working out its row's weights itself (no barrier in the tail).
        constexpr int kFew = 8;
        if (n <= kFew) {
            const int d = 4 * (threadIdx.x % 32);
            const int64_t step = R.part_step();
            for (int h = threadIdx.x / 32; h < g; h += kWarps) {
                const int64_t at = R.part(a, h, 0);
                float lse[kFew];
                float4 v[kFew];
#pragma unroll
                for (int s = 0; s < kFew; ++s) {
                    lse[s] = s < n ? __ldcg(a.ws_lse + at + s * step) : -INFINITY;
                    v[s] = s < n ? __ldcg(reinterpret_cast<const float4 *>(a.ws_o + (at + s * step) * kHeadDim + d))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                float m = -INFINITY, sum = 0.f;
                bool bad = false;
#pragma unroll
                for (int s = 0; s < kFew; ++s) {
                    bad |= lse[s] != lse[s];
                    m = fmaxf(m, lse[s]);
                }
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int s = 0; s < kFew; ++s)
                    if (lse[s] != -INFINITY) {
                        const float w = fast_exp2(lse[s] - m);
                        sum += w;
                        acc.x += w * v[s].x;
                        acc.y += w * v[s].y;
                        acc.z += w * v[s].z;
                        acc.w += w * v[s].w;
                    }
                const bool zero = bad || sum == 0.f;
                store_out4(a.out, R.ids[h] * kHeadDim + d,
                           zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                                : make_float4(acc.x / sum, acc.y / sum, acc.z / sum, acc.w / sum),
                           a.out_fp32);
            }
            if (threadIdx.x == 0)
                *counter = 0;                // ready for the next call
            return;
        }
    }
    float *s_tot = scratch;                  // [kRowsT] sum of weights (0: drop the row)
    float *s_w = scratch + kRowsT;           // [g][n]: lse, then weights
    for (int i = threadIdx.x; i < g * n; i += kThreads)
        s_w[i] = __ldcg(a.ws_lse + R.part(a, i / n, i % n));
    __syncthreads();
    // one warp per head: max, validity, weights, their sum
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int h = warp; h < g; h += kWarps) {
        float *w = s_w + h * n;
        float m = -INFINITY;
        bool bad = false;
        for (int s = lane; s < n; s += 32) {
            bad |= w[s] != w[s];
            m = fmaxf(m, w[s]);
        }
        bad = __any_sync(0xFFFFFFFFu, bad);
        for (int off = 16; off > 0; off >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        float sum = 0.f;
        for (int s = lane; s < n; s += 32) {         // a split that saw no token: lse -inf, weight 0
            const float e = (bad || w[s] == -INFINITY) ? 0.f : fast_exp2(w[s] - m);
            w[s] = e;
            sum += e;
        }
        for (int off = 16; off > 0; off >>= 1)
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
        if (lane == 0)
            s_tot[h] = bad ? 0.f : sum;
    }
    __syncthreads();
    // thread t: the (row, 4 dims) pairs t, t + 128, ... of the rows x 32;
    // kRound splits per round, every 16-byte load of a round issued before
    // any is used, so a round costs one trip to L2. The windowed and
    // block-scaled builds (balanced launches of few splits per pair) take short
    // rounds: this code runs once per pair and cold, and the unrolled rounds'
    // instruction misses cost more than the trips saved (48 splits by one CTA:
    // 4 query tokens 48 -> 33 us, single 25 -> 23 us)
    constexpr int kPairs = kRowsT * (kHeadDim / 4) / kThreads;          // 2, or 4 with 16 rows
    constexpr int kRound = (kMulti ? 4 : 8) / (kNanFlows ? 4 : 1);
    static_assert(kRowsT * (kHeadDim / 4) == kPairs * kThreads, "whole (row, 4 dims) pairs per thread");
    int hp[kPairs];
#pragma unroll
    for (int q = 0; q < kPairs; ++q)
        hp[q] = static_cast<int>(threadIdx.x + q * kThreads) / 32;
    const int cp = 4 * (threadIdx.x % 32);
    float4 acc[kPairs];
#pragma unroll
    for (int q = 0; q < kPairs; ++q)
        acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    [[maybe_unused]] const float *from[kPairs];
    [[maybe_unused]] int64_t step = 0;
    if constexpr (kNanFlows) {
        step = R.part_step() * kHeadDim;
#pragma unroll
        for (int q = 0; q < kPairs; ++q)
            from[q] = a.ws_o + R.part(a, min(hp[q], g - 1), 0) * kHeadDim + cp;
    }
    for (int s0 = 0; s0 < n; s0 += kRound) {
        float4 v[kPairs][kRound];
#pragma unroll
        for (int q = 0; q < kPairs; ++q)
#pragma unroll
            for (int j = 0; j < kRound; ++j) {
                const float *p;
                if constexpr (kNanFlows)
                    p = from[q] + (s0 + j) * step;
                else
                    p = a.ws_o + R.part(a, hp[q], s0 + j) * kHeadDim + cp;
                v[q][j] = (hp[q] < g && s0 + j < n) ? __ldcg(reinterpret_cast<const float4 *>(p))
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
        for (int q = 0; q < kPairs; ++q)
#pragma unroll
            for (int j = 0; j < kRound; ++j)
                if (hp[q] < g && s0 + j < n) {
                    const float wt = s_w[hp[q] * n + s0 + j];
                    acc[q].x += wt * v[q][j].x;
                    acc[q].y += wt * v[q][j].y;
                    acc[q].z += wt * v[q][j].z;
                    acc[q].w += wt * v[q][j].w;
                }
    }
#pragma unroll
    for (int q = 0; q < kPairs; ++q)
        if (hp[q] < g) {
            const int64_t o0 = R.out_row(a, hp[q]) * kHeadDim + cp;
            if constexpr (kNanFlows) {
                const float t = s_tot[hp[q]];
                store_out4(a.out, o0,
                           t != 0.f ? make_float4(acc[q].x / t, acc[q].y / t, acc[q].z / t, acc[q].w / t)
                                    : make_float4(0.f, 0.f, 0.f, 0.f),
                           a.out_fp32);
                continue;
            }
            const bool some = s_tot[hp[q]] > 0.f;
            store_out(a.out, o0, some ? acc[q].x / s_tot[hp[q]] : 0.f, a.out_fp32);
            store_out(a.out, o0 + 1, some ? acc[q].y / s_tot[hp[q]] : 0.f, a.out_fp32);
            store_out(a.out, o0 + 2, some ? acc[q].z / s_tot[hp[q]] : 0.f, a.out_fp32);
            store_out(a.out, o0 + 3, some ? acc[q].w / s_tot[hp[q]] : 0.f, a.out_fp32);
        }
    if (a.expected_tags != nullptr) {        // kvq_decode_step: the request's verdict
        __shared__ int s_stale_any;
        if (threadIdx.x == 0) {
            int any = 0;
            for (int sp = 0; sp < n; ++sp)
                any |= __float_as_uint(__ldcg(a.ws_lse + R.part(a, 0, sp))) == kLseStale;
            s_stale_any = any;
        }
        __syncthreads();
        finish_step(a, R.b, R.kvh, s_stale_any != 0);
    }
    if (threadIdx.x == 0)
        *counter = 0;                        // ready for the next call
}

// A split that cannot produce a result (invalid page id, or a copy that
// timed out): a single-split request gets zeros; otherwise the split
// publishes an invalid (NaN) lse so the combine zeroes the request.
template <bool kMulti, bool kNanFlows>
__device__ void drop_split(const DecodeArgs &a, const Rows<kMulti, kNanFlows> &R, int split, int nsplit, float *smem,
                           uint32_t lse_bits = kLseInvalid)
{
    if (nsplit == 1) {
        for (int i = threadIdx.x; i < R.nrows * kHeadDim; i += kThreads)
            store_out(a.out, R.out_row(a, i / kHeadDim) * kHeadDim + i % kHeadDim, 0.f, a.out_fp32);
        if (a.expected_tags != nullptr)
            finish_step(a, R.b, R.kvh, lse_bits == kLseStale);
        return;
    }
    if (threadIdx.x < R.nrows)
        a.ws_lse[R.part(a, threadIdx.x, split)] = __uint_as_float(lse_bits);
    publish_and_combine<kMulti, kNanFlows>(a, R, nsplit, kMulti ? smem : smem + kScratchOffset);
}

// What a split contributes to the cluster form of the combine.
// Cluster-wide barrier with a relaxed arrive: it orders no memory access,
// only the threads' progress (the wait still acquires).
__device__ __forceinline__ void cluster_sync_relaxed_arrive()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\t"
                 "barrier.cluster.wait.aligned;" ::: "memory");
}

enum PartialStatus { kPartialOk = 0, kPartialEmpty = 1, kPartialInvalid = 2, kPartialStale = 3 };

// Cluster form of the combine, used when the splits of each (request, KV
// head) are the CTAs of one thread-block cluster (every split resident at
// once).  Each CTA leaves its partial in its own shared memory at `part`:
// [rows] lse (log2 domain), then [rows][128] normalised o (rows =
// rows_per_cta(kMulti)); an empty
// split (no tokens) publishes lse = -inf (weight 0), an invalid one NaN (its
// heads get zeros).  After a cluster barrier CTA r merges the query heads
// h = r, r + n, ... of the group from every peer's partial, read through
// distributed shared memory:
//   M = max_s lse_s,  out = sum_s 2^(lse_s - M) o_s / sum_s 2^(lse_s - M).
// A second barrier keeps every CTA's shared memory alive until its peers
// have read it.  It needs no release: a thread reaches it only after the
// values it loaded from its peers have been consumed by its output stores,
// and a release there would make every CTA wait for those global stores.
// Every CTA of the cluster calls this exactly once, with the same
// `finisher`: for kvq_decode_step the rank that reads every peer's verdict,
// else -1.  Returns, on the finisher, whether any split of the
// request failed its tag check (false elsewhere).
template <bool kMulti, bool kNanFlows>
__device__ bool cluster_finish(const DecodeArgs &a, const Rows<kMulti, kNanFlows> &R, PartialStatus status, float *part,
                               int finisher)
{
    __shared__ int s_any_stale;
    constexpr int kRowsT = rows_per_cta(kMulti);
    if (status != kPartialOk && threadIdx.x < kRowsT)
        part[threadIdx.x] = status == kPartialEmpty ? -INFINITY
                            : __uint_as_float(status == kPartialStale ? kLseStale : kLseInvalid);
    cluster_sync();
    KVQ_STAMP(5);
    const int g = R.nrows, n = a.max_splits;
    const int rank = static_cast<int>(cluster_ctarank());
    const uint32_t base = smem_addr(part);
    if (rank == finisher && threadIdx.x == 0) {            // every peer's head-0 lse carries its verdict
        int stale = 0;
        for (int sp = 0; sp < n; ++sp)
            stale |= __float_as_uint(ld_shared_cluster_f32(map_shared_rank(base, static_cast<uint32_t>(sp)))) ==
                     kLseStale;
        s_any_stale = stale;
    }
    // thread t takes dims 4 (t % 32) .. + 3 of head h0 + t / 32 (16-byte
    // loads from each peer), 4 of this CTA's heads per pass
    for (int h0 = rank; h0 < g; h0 += kThreads / 32 * n) {
        const int h = h0 + (threadIdx.x / 32) * n;
        if (h >= g)
            continue;
        const int d = 4 * (threadIdx.x % 32);
        float lse[kMaxCluster];
        float4 ov[kMaxCluster];
#pragma unroll
        for (int s = 0; s < kMaxCluster; ++s) {
            lse[s] = -INFINITY;
            ov[s] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s < n) {
                const uint32_t peer = map_shared_rank(base, static_cast<uint32_t>(s));
                lse[s] = ld_shared_cluster_f32(peer + 4u * h);
                ov[s] = ld_shared_cluster_v4(peer + 4u * (kRowsT + h * kHeadDim + d));
            }
        }
        float m = -INFINITY;
        bool bad = false;
#pragma unroll
        for (int s = 0; s < kMaxCluster; ++s) {
            bad |= lse[s] != lse[s];
            m = fmaxf(m, lse[s]);
        }
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s = 0; s < kMaxCluster; ++s) {
            if (lse[s] != -INFINITY) {
                const float w = fast_exp2(lse[s] - m);
                sum += w;
                acc.x += w * ov[s].x;
                acc.y += w * ov[s].y;
                acc.z += w * ov[s].z;
                acc.w += w * ov[s].w;
            }
        }
        const bool zero = bad || (kNanFlows ? sum == 0.f : !(sum > 0.f));
        const int64_t o0 = R.out_row(a, h) * kHeadDim + d;
        if constexpr (kNanFlows) {
            store_out4(a.out, o0,
                       zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : make_float4(acc.x / sum, acc.y / sum, acc.z / sum, acc.w / sum),
                       a.out_fp32);
            continue;
        }
        store_out(a.out, o0, zero ? 0.f : acc.x / sum, a.out_fp32);
        store_out(a.out, o0 + 1, zero ? 0.f : acc.y / sum, a.out_fp32);
        store_out(a.out, o0 + 2, zero ? 0.f : acc.z / sum, a.out_fp32);
        store_out(a.out, o0 + 3, zero ? 0.f : acc.w / sum, a.out_fp32);
    }
    __syncthreads();                         // orders s_any_stale within the CTA
    cluster_sync_relaxed_arrive();           // peers' reads of this CTA's partial are done
    return rank == finisher && s_any_stale != 0;
}

// One split: tokens t0 .. t0 + span - 1 (span at most 8,192, t0 a multiple of
// the page size) of the context that (request b, KV head kvh, row block rb)
// shows, the split-th of nsplit (0: as many as split_tokens gives the
// request); base as in Rows.
struct Job {
    int b, kvh, rb, split, nsplit, span;
    int64_t t0, base, real;                  // real: the request's tokens, or -1 (read them)
};

template <bool kBf16Cache, bool kPreciseP, bool kCluster, bool kMulti, bool kWindow, bool kBlocks>
__device__ __forceinline__ void run_split(const CUtensorMap &k_map, const CUtensorMap &v_map, const DecodeArgs &a,
                                          const Job &job, bool first)
{
    using T = BuildTile<kBf16Cache, kWindow>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + T::kRingBytes);
    int32_t *page_list = reinterpret_cast<int32_t *>(full + kWarps * T::kStages);
    uint32_t *tag_live = reinterpret_cast<uint32_t *>(page_list + kMaxPageList);   // kvq_decode_step:
    uint32_t *tag_want = tag_live + kMaxPageList;                                  // the split's tags
    uint8_t *new_tok = reinterpret_cast<uint8_t *>(tag_want + kMaxPageList);       // [K row][V row]
    // windowed builds, in the place of the tags (kExpBytes, kQFragBytes)
    [[maybe_unused]] uint16_t *blk_exp = reinterpret_cast<uint16_t *>(page_list + kMaxPageList);
    [[maybe_unused]] uint2 *q_frag =
        reinterpret_cast<uint2 *>(reinterpret_cast<uint8_t *>(page_list + kMaxPageList) + kExpBytes);
    constexpr bool kSmemQ = smem_q(kMulti, kWindow);
    __shared__ int s_failed;
    __shared__ int s_stale;                                // kvq_decode_step: a page of this split failed

    // The builds without a window always run the split that their place in
    // the grid names.
    const int split = kWindow ? job.split : static_cast<int>(blockIdx.x);
    const int b = kWindow ? job.b : static_cast<int>(blockIdx.z);
    // with several query tokens, blockIdx.y = KV head x row blocks
    const int line = static_cast<int>(blockIdx.y);
    const int kvh = kWindow ? job.kvh : kMulti ? line / a.row_blocks : line;
    const int rb = kWindow ? job.rb : kMulti ? line % a.row_blocks : 0;
    const int split_tokens = kWindow ? job.span : a.split_tokens;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int gq = lane >> 2, tq = lane & 3;
    const int g = a.group, ps = a.page_size;
    const int ps_shift = __ffs(ps) - 1;                  // ps is 16, 32, 64 or 128
    Rows<kMulti, kWindow> R;
    R.b = b;
    R.kvh = kvh;
    R.row0 = rb * rows_per_cta(kMulti);
    R.nrows = kMulti ? min(rows_per_cta(true), a.n_query * g - R.row0) : g;
    R.slot = kWindow ? (static_cast<int64_t>(b) * a.num_kv_heads + kvh) * (kMulti ? a.row_blocks : 1) + rb
                     : static_cast<int64_t>(b) * gridDim.y + line;
    R.base = job.base;
    if constexpr (kWindow) {
        __shared__ int64_t s_ids[rows_per_cta(kMulti)];
        if (threadIdx.x < R.nrows)
            s_ids[threadIdx.x] = R.id(a, threadIdx.x);
        R.ids = s_ids;
    }

    const int first_page = kWindow ? static_cast<int>(job.t0 >> ps_shift)
                                   : static_cast<int>(static_cast<int64_t>(split) * a.split_tokens / ps);
    const int span_left = a.max_pages_per_seq - first_page;
    const int span = split_tokens / ps < span_left ? split_tokens / ps : span_left;
    const int32_t *bt = a.block_table + static_cast<int64_t>(b) * a.max_pages_per_seq + first_page;
    const int lines_per_tok = kBf16Cache ? 2 : 1;

    // A lane's part of query row nt * 8 + gq: dims 32 tq .. 32 tq + 31.  The
    // single-token windowed builds fetch it here, beside the first table
    // entries (0.3 us sooner under way); only what follows the first copies
    // uses it.
    constexpr bool kEarlyQ = kWindow && !kMulti;
    constexpr int kNT = rows_per_cta(kMulti) / kMaxGroup;   // mma n-tiles of query rows per warp
    constexpr int kRowsT = rows_per_cta(kMulti);
    uint32_t q_raw[kNT][16];
    auto load_q = [&](int nt) {
        uint32_t (&w)[16] = q_raw[nt];
        if (nt * kMaxGroup + gq < R.nrows) {
            const uint4 *src = reinterpret_cast<const uint4 *>(
                static_cast<const uint16_t *>(a.q) + (R.id(a, nt * kMaxGroup + gq) * kHeadDim + 32 * tq));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = __ldg(src + i);
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                w[i] = 0;
        }
    };

    // The block-table entries this split can use depend only on the split
    // index, so they are loaded together with the request's length.
    constexpr int kIdsPerThread = (kMaxPageList + kThreads - 1) / kThreads;
    int32_t ids[kIdsPerThread];
    if (!kWindow || a.window == 0) {
#pragma unroll
        for (int k = 0; k < kIdsPerThread; ++k) {
            const int i = threadIdx.x + k * kThreads;
            ids[k] = i < span ? __ldg(bt + i) : -1;
        }
    }
    const int64_t real_len = kWindow && job.real >= 0 ? job.real : a.seq_lens[b];
    if constexpr (kEarlyQ)
        load_q(0);
    // kvq_decode_step: each split checks the tags of its own pages (together
    // the request's used entries) while it streams them, and publishes a
    // failure with its partial; the CTA that sees every split's partial
    // writes the flag and, if the request passed, its new token
    // (finish_here, or finish_step in the workspace form).  A request
    // without tokens to check is decided here.
    const bool step_check = !kWindow && a.expected_tags != nullptr;
    const bool reporter = step_check && split == 0 && kvh == 0 && threadIdx.x == 0;
    const bool aborted = !step_check && a.abort_flags != nullptr && a.abort_flags[b] != 0;
    const int64_t cap = static_cast<int64_t>(a.max_pages_per_seq) * ps;
    const bool zero_request = aborted || real_len <= 0 || real_len > cap;
    // Window: from here on `len` and every position count the shortened
    // context (shown_context).
    int64_t len = real_len;
    [[maybe_unused]] int64_t win0 = 0;                     // where the first query's window starts
    if constexpr (kWindow) {
        if (a.window > 0) {
            const Shown shown = shown_context(a, real_len, ps_shift);
            len = shown.len;
            win0 = shown.win0;
            // only entries of pages with a token of the shortened context are read
#pragma unroll
            for (int k = 0; k < kIdsPerThread; ++k) {
                const int i = threadIdx.x + k * kThreads;
                const int64_t v = static_cast<int64_t>(first_page) + i;
                const bool held = !zero_request && i < split_tokens / ps && (v << ps_shift) < len;
                ids[k] = held ? __ldg(bt + i + (v < shown.sink_pages ? 0 : shown.hole)) : -1;
            }
        }
    }
    if (reporter && zero_request)                          // the check's verdict without a look:
        a.abort_out[b] = real_len > cap ? 1 : 0;                // too long fails, empty passes
    const int nsplit = zero_request ? 1
                       : kWindow && job.nsplit > 0
                           ? job.nsplit
                           : static_cast<int>((len + a.split_tokens - 1) / a.split_tokens);
    float *part = reinterpret_cast<float *>(smem) + scratch_offset(kMulti);   // cluster partial
    // kvq_decode_step: the split that finishes the step of a request with
    // tokens in the cluster form and when there is one split -- the last
    // split, which holds the new token (the workspace form's combine
    // finishes in whichever split arrives last)
    const int finisher = step_check && !zero_request ? nsplit - 1 : -1;
    if constexpr (kCluster) {
        if (zero_request || split >= nsplit) {             // no tokens: weight 0
            cluster_finish<kMulti, kWindow>(a, R, kPartialEmpty, part, finisher);
            return;
        }
    }
    if (split >= nsplit)
        return;

    if (zero_request) {                                    // split 0 writes the zeros
        for (int i = threadIdx.x; i < R.nrows * kHeadDim; i += kThreads)
            store_out(a.out, R.id(a, i / kHeadDim) * kHeadDim + i % kHeadDim, 0.f, a.out_fp32);
        return;
    }

    const int64_t t0 = kWindow ? job.t0 : static_cast<int64_t>(split) * a.split_tokens;
    const int64_t t1 = min(len, t0 + split_tokens);
    // page ids of this split (t0 is a multiple of the page size)
    const int n_pages = static_cast<int>((t1 - 1) / ps) - first_page + 1;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kIdsPerThread; ++k) {
        const int i = threadIdx.x + k * kThreads;
        if (i < n_pages) {
            bad |= (ids[k] < 0 || ids[k] >= a.num_pages);
            page_list[i] = ids[k];
        }
    }
    if (threadIdx.x == 0) {
        s_failed = 0;
        s_stale = 0;
        for (int i = 0; i < kWarps * T::kStages; ++i) {
            if (kWindow && !first)
                mbar_inval(&full[i]);
            mbar_init(&full[i], 1);
        }
        fence_mbar_init();
    }
    bad = __syncthreads_or(bad);

    // Fused append (kvq_decode_attn_append): the split holding token len - 1
    // writes that token's codes for KV head kvh into the cache now (when its
    // page id is valid, as kvq_append would) and patches them into its tile
    // when the chunk's copy lands, so its own attention uses them without
    // reading them back.
    int it_new = -1;
    using NewRow = std::conditional_t<kBf16Cache, uint2, uint32_t>;   // a lane's part of the row
    NewRow new_k{}, new_v{};
    int64_t new_row = -1;                                  // cache row of the new token
    if (!kWindow && a.k_new != nullptr && split == nsplit - 1) {
        const int64_t tpos = len - 1;
        const int c_last = static_cast<int>((tpos - t0) / kChunkTokens);
        const int32_t page = page_list[static_cast<int>(tpos / ps) - first_page];
        if (warp == c_last % kWarps && page >= 0 && page < a.num_pages) {
            it_new = c_last / kWarps;
            const int64_t src = (static_cast<int64_t>(b) * a.num_kv_heads + kvh) * kHeadDim + 4 * lane;
            const uint2 xk = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.k_new) + src);
            const uint2 xv = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.v_new) + src);
            new_row = (static_cast<int64_t>(page) * a.num_kv_heads + kvh) * ps + tpos % ps;
            if constexpr (kBf16Cache) {
                new_k = xk;
                new_v = xv;
            } else {
                new_k = encode4_e4m3(xk.x, xk.y, a.k_scale[kvh]);
                new_v = encode4_e4m3(xv.x, xv.y, a.v_scale[kvh]);
            }
            if (step_check) {                              // kept for the end of the step
                reinterpret_cast<NewRow *>(new_tok)[lane] = new_k;
                reinterpret_cast<NewRow *>(new_tok + T::kRowBytes)[lane] = new_v;
            }
        }
    }
    // kvq_decode_step, on the split that holds the new token (the request's
    // last split) once the request's verdict is known: KV head 0 reports
    // it, and a request that passed gets the staged row written.
    auto finish_here = [&](bool stale) {
        if (kvh == 0 && threadIdx.x == 0)
            a.abort_out[b] = stale ? 1 : 0;
        const int64_t tpos = len - 1;
        const int32_t page = page_list[static_cast<int>(tpos / ps) - first_page];
        if (stale || threadIdx.x >= 32 || page < 0 || page >= a.num_pages)
            return;
        const int64_t row = (static_cast<int64_t>(page) * a.num_kv_heads + kvh) * ps + tpos % ps;
        const int ln = threadIdx.x;
        *reinterpret_cast<NewRow *>(static_cast<uint8_t *>(a.k_cache) + row * T::kRowBytes + sizeof(NewRow) * ln) =
            reinterpret_cast<const NewRow *>(new_tok)[ln];
        *reinterpret_cast<NewRow *>(static_cast<uint8_t *>(a.v_cache) + row * T::kRowBytes + sizeof(NewRow) * ln) =
            reinterpret_cast<const NewRow *>(new_tok + T::kRowBytes)[ln];
    };
    auto write_new = [&]() {
        if (new_row < 0)
            return;
        if constexpr (kBf16Cache) {
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.k_cache) + new_row * 256 + 8 * lane) = new_k;
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.v_cache) + new_row * 256 + 8 * lane) = new_v;
        } else {
            *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.k_cache) + new_row * 128 + 4 * lane) = new_k;
            *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.v_cache) + new_row * 128 + 4 * lane) = new_v;
        }
    };
    if (!step_check)                                       // kvq_decode_step: finish_step writes it
        write_new();

    if (bad) {                                             // for kvq_decode_step a failed check
        if constexpr (kCluster) {
            cluster_finish<kMulti, kWindow>(a, R, step_check ? kPartialStale : kPartialInvalid, part, finisher);
            if (split == finisher)                         // this split failed: so did the request
                finish_here(true);
        } else
            drop_split<kMulti, kWindow>(a, R, split, nsplit, reinterpret_cast<float *>(smem),
                       step_check ? kLseStale : kLseInvalid);
        return;
    }

    // ---------------------------------------------------------------- setup
    const int n_chunks = static_cast<int>((t1 - t0 + kChunkTokens - 1) / kChunkTokens);
    const int my_chunks = n_chunks > warp ? (n_chunks - warp + kWarps - 1) / kWarps : 0;
    uint8_t *ring = smem + warp * T::kStages * T::kStageBytes;
    uint64_t *my_full = full + warp * T::kStages;
    const int box_tok = ps < kChunkTokens ? ps : kChunkTokens;
    const int parts = kChunkTokens / box_tok;                       // 1 or 2 copies per tensor
    const uint32_t part_bytes = static_cast<uint32_t>(box_tok * T::kRowBytes);
    // evict-first unless other row blocks of the split read the same pages
    auto make_policy = [&]() {
        return kMulti && a.row_blocks > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
    };
    uint64_t policy = 0;
    if constexpr (!kWindow)
        policy = make_policy();


    // Issue the copies of this warp's local chunk `it`: the whole warp, one
    // copy per lane (lanes 0 .. np - 1 the K parts, np .. 2 np - 1 the V
    // parts), which issues them about twice as fast as one lane in turn.
    auto issue = [&](int it) {
        const int c = warp + it * kWarps;
        const int64_t tok = t0 + static_cast<int64_t>(c) * kChunkTokens;
        const int st = it % T::kStages;
        const int64_t left = t1 - tok;
        const int np = left >= kChunkTokens ? parts : static_cast<int>((left + box_tok - 1) / box_tok);
        if (lane == 0)
            mbar_arrive_expect_tx(&my_full[st], 2u * part_bytes * np);
        __syncwarp();
        if (lane < 2 * np) {
            const int part = lane < np ? lane : lane - np;
            const int64_t ptok = tok + part * box_tok;
            const int32_t page = page_list[static_cast<int>(ptok >> ps_shift) - first_page];
            const int64_t row = (static_cast<int64_t>(page) * a.num_kv_heads + kvh) * ps + (ptok & (ps - 1));
            uint8_t *dst = ring + st * T::kStageBytes + (lane < np ? 0 : T::kBytes) + part * part_bytes;
            tma_load_2d(dst, lane < np ? static_cast<const void *>(&k_map) : static_cast<const void *>(&v_map), 0,
                        static_cast<int32_t>(row * lines_per_tok), &my_full[st], kWindow ? make_policy() : policy);
        }
    };

    const int pro = my_chunks < T::kStages ? my_chunks : T::kStages;
    for (int it = 0; it < pro; ++it)
        issue(it);

    if (step_check) {
        // kvq_decode_step: this split's share of the tag check, its own pages
        // (whose ids are in range here).  The live and expected tags come in
        // by asynchronous copies behind the first bulk copies and are compared
        // once the split has attended: a failure only changes what it
        // publishes.  Thread t copies (and later compares) entries t, t + 128, ...
        const uint32_t *want = a.expected_tags + static_cast<int64_t>(b) * a.max_pages_per_seq + first_page;
#pragma unroll
        for (int k = 0; k < kIdsPerThread; ++k) {
            const int i = threadIdx.x + k * kThreads;
            if (i < n_pages) {
                cp_async_4(tag_live + i, a.page_tags + page_list[i]);
                cp_async_4(tag_want + i, want + i);
            }
        }
        cp_async_commit();
    }

    // Behind the first copies, in one trip: the exponents of the split's
    // blocks, one byte each (through L2: the append that wrote them may have
    // run on this SM beside this CTA), and in the multi-token windowed builds
    // the query rows.
    constexpr int kExpsPerThread = (8192 / kBlockTokens + kThreads - 1) / kThreads;
    [[maybe_unused]] int exps[kExpsPerThread][2];
    if constexpr (kBlocks) {
        const int n_blocks = static_cast<int>((t1 - t0 + kBlockTokens - 1) / kBlockTokens);
        const int bpp_shift = ps_shift - 4;                // blocks per page: ps / 16
#pragma unroll
        for (int k = 0; k < kExpsPerThread; ++k) {
            const int i = threadIdx.x + k * kThreads;
            exps[k][0] = exps[k][1] = 0;                   // the last chunk's second m-tile may hold no token
            if (i < n_blocks) {
                const int64_t at =
                    ((static_cast<int64_t>(page_list[i >> bpp_shift]) * a.num_kv_heads + kvh) << bpp_shift) +
                    (i & ((1 << bpp_shift) - 1));
                exps[k][0] = __ldcg(a.k_exp + at);
                exps[k][1] = __ldcg(a.v_exp + at);
            }
        }
    }
    constexpr bool kMidQ = kWindow && kMulti;
    if constexpr (kMidQ)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
            load_q(nt);
    if constexpr (kBlocks) {
#pragma unroll
        for (int k = 0; k < kExpsPerThread; ++k) {
            const int i = threadIdx.x + k * kThreads;
            if (i < 2 * n_chunks)
                blk_exp[i] = static_cast<uint16_t>(
                    (max(exps[k][0], kReadKeyExpMin) & 0xFF) |
                    (min(max(exps[k][1], kReadValueExpMin), kReadValueExpMax) << 8));
        }
    }

    // Query fragments (mma B operand): lane (gq, tq) holds query row gq of
    // this CTA (with one query token: head gq of the group) at dims 32*tq ..
    // 32*tq+31; k-slot pairs of k-step c map to dims 32*tq + 4*c + {0,1} and
    // {2,3}.
    //
    // FP8 cache: the product runs in f16, whose range is narrower than
    // bf16's.  Each q row is first multiplied by 2^e_h, the power of two that
    // puts its largest magnitude in [2^14, 2^15) (exact: only the exponent
    // changes), so no element overflows and every element within 2^28 of the
    // row's largest keeps all its bits; the score multiplier of head h then
    // carries 2^-e_h.
    uint32_t qf[kNT][8][2];
    int q_exp[kNT];                                        // e of row nt * 8 + gq
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
        q_exp[nt] = 0;
        uint32_t (&w)[16] = q_raw[nt];
        if constexpr (!kEarlyQ && !kMidQ)
            load_q(nt);
        float q_mul = 1.f;
        if constexpr (!kBf16Cache) {
            uint32_t mx = 0;                               // largest |q| of the row, as bf16 bits
#pragma unroll
            for (int i = 0; i < 16; ++i)
                mx = max(mx, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            q_exp[nt] = row_pow2_exponent(mx);
            q_mul = __int_as_float((127 + q_exp[nt]) << 23);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if constexpr (kBf16Cache) {
                    qf[nt][c][j] = w[2 * c + j];
                } else {
                    const float2 f = bf16x2_to_f32x2(w[2 * c + j]);
                    qf[nt][c][j] = f32x2_to_f16x2(f.x * q_mul, f.y * q_mul);
                }
            }
        }
    }

    const float kscale = kBf16Cache || kBlocks ? 1.f : a.k_scale[kvh];
    const float vscale = kBf16Cache || kBlocks ? 1.f : a.v_scale[kvh];
    // score multiplier (log2 domain) of the two query heads 2tq, 2tq + 1
    // whose scores this lane holds: the softmax scale, the K scale and the
    // undoing of their q rows' power-of-two scaling
    float qk_col[kNT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int e = __shfl_sync(0xFFFFFFFFu, q_exp[nt], 4 * (2 * tq + j));
            qk_col[nt][j] = a.qk_scale_log2 * kscale * __int_as_float((127 - e) << 23);
        }
    // Causal limit of those two rows: query token i sees the positions below
    // len - n_query + 1 + i (with one query token: all of them), kept as a
    // count from the split's start, at most one chunk past its end.  Below
    // full_end every row of the CTA sees every token.
    [[maybe_unused]] int vis_col[kNT][2] = {};
    [[maybe_unused]] int64_t full_end = t1;
    if constexpr (kMulti && !kWindow) {
        const int64_t vis0 = len - a.n_query + 1;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int64_t v = vis0 + (R.row0 + nt * kMaxGroup + 2 * tq + j) / g - t0;
                vis_col[nt][j] = static_cast<int>(
                    v < -1 ? -1 : (v > split_tokens + kChunkTokens ? split_tokens + kChunkTokens : v));
            }
        full_end = min(t1, vis0 + R.row0 / g);
    }
    // Windowed builds keep less in registers, counts from the split's start
    // (t0) all: query token i of the call sees the positions below vis0 + i
    // but for those from sink_end to win + i; the tokens i of this lane's score
    // columns lie in a nibble each of tok_col.  V rows that no row of the CTA
    // sees (sink_end up to win_first) are zeroed, so what they hold cannot
    // reach the product.  Below full_to and outside [sink_end, mask_hi) no
    // token is masked.
    [[maybe_unused]] uint32_t tok_col = 0;
    [[maybe_unused]] int vis0 = 0, sink_end = 0, full_to = 0;
    [[maybe_unused]] int win = -2 * kChunkTokens, win_first = win, mask_hi = win;      // window 0: before everything
    if constexpr (kWindow) {
        auto rel = [&](int64_t v) {                        // query tokens are at most 15 further on
            v -= t0;
            const int64_t most = split_tokens + 2 * kChunkTokens;
            return static_cast<int>(v < -2 * kChunkTokens ? -2 * kChunkTokens : (v > most ? most : v));
        };
        const int first = kMulti ? R.row0 / g : 0, last = kMulti ? (R.row0 + R.nrows - 1) / g : 0;
        vis0 = rel(len - a.n_query + 1);
        full_to = rel(min(t1, len - a.n_query + 1 + first));
        if constexpr (kMulti)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    tok_col |= static_cast<uint32_t>(min((R.row0 + nt * kMaxGroup + 2 * tq + j) / g, 15))
                               << (4 * (2 * nt + j));
        if (a.window > 0) {
            win = rel(win0);
            sink_end = rel(a.num_sinks);
            win_first = rel(win0 + first);
            mask_hi = rel(win0 + last);
        }
    }
    if constexpr (kSmemQ) {                                // each warp stores a quarter of the fragments
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            if (kk / 2 == warp)
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
                    q_frag[(kk * kNT + nt) * 32 + lane] = make_uint2(qf[nt][kk][0], qf[nt][kk][1]);
    }
    if constexpr (kBlocks || kSmemQ)
        __syncthreads();                                   // the exponents and fragments are in place

    // The windowed and block-scaled builds over FP8 keep weights, sums and
    // accumulators 2^15 times larger (the quotient is the same, and f16 ends at
    // 65504): an f16 weight, and with it the second term of the precise form,
    // is then cut at 2^-39 of the largest weight instead of 2^-24.  A bf16
    // cache's weights are bf16 terms, whose range needs no lift, and its values
    // (up to 2^128) leave no room for one.
    constexpr float kLift = kWindow && !kBf16Cache ? 15.f : 0.f;
    // 16-bit terms of a weight in the PV product: one for bf16 output (f16
    // 2^-12, for a bf16 cache bf16 2^-9: an output of many tokens averages
    // them below its own 2^-9; a second bf16 term cost 2 to 10 %), for fp32
    // output two f16 terms (2^-24) or two bf16 ones (2^-18), in the windowed
    // builds three (2^-27).
    constexpr int kTerms = !kPreciseP ? 1 : kWindow && kBf16Cache ? 3 : 2;
    // For fp32 output a tile's products are summed from zero and added to O
    // by fp32 additions that round: the tensor core cuts what it adds to a
    // large accumulator, always towards zero (error against fp64, 64 requests
    // of up to 5,000 tokens: bf16 cache 1.6e-6, 3.9e-7 so; FP8 9.9e-7, 3.7e-7).
    constexpr bool kSumApart = kWindow && kPreciseP;
    float m_run[kNT][2], l_run[kNT][2];
    float o[kNT][8][4];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
        m_run[nt][0] = m_run[nt][1] = -INFINITY;
        l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }

    bool failed = false;
    int it = 0;
    for (; it < my_chunks; ++it) {
        const int st = it % T::kStages;
        // every lane polls; the warp gives up as one if any lane did
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&my_full[st], (it / T::kStages) & 1, a.copy_wait_ns))) {
            failed = true;
            break;
        }
        if (it == 0 && warp == 0)
            KVQ_STAMP(2);
        const uint8_t *ks = ring + st * T::kStageBytes;
        const uint8_t *vs = ks + T::kBytes;
        const int c = warp + it * kWarps;
        const int64_t tok = t0 + static_cast<int64_t>(c) * kChunkTokens;
        if (it == it_new) {                  // fused append: the new token's row
            const int r = static_cast<int>(len - 1 - tok);
            uint8_t *kt = ring + st * T::kStageBytes;
            uint8_t *vt = kt + T::kBytes;
            if constexpr (kBf16Cache) {
                const uint32_t off = swz(2 * r + (lane >> 4), (lane & 15) >> 1) + 8 * (lane & 1);
                *reinterpret_cast<uint2 *>(kt + off) = new_k;
                *reinterpret_cast<uint2 *>(vt + off) = new_v;
            } else {
                const uint32_t off = swz(r, lane >> 2) + 4 * (lane & 3);
                *reinterpret_cast<uint32_t *>(kt + off) = new_k;
                *reinterpret_cast<uint32_t *>(vt + off) = new_v;
            }
            __syncwarp();
        }
        const int64_t left = t1 - tok;
        const int n_valid = left < kChunkTokens ? static_cast<int>(left) : kChunkTokens;   // V rows
        [[maybe_unused]] int s_valid[kNT][2];            // tokens of the chunk each score column sees
        if constexpr (!kWindow)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    s_valid[nt][j] = kMulti ? min(n_valid, vis_col[nt][j] - c * kChunkTokens) : n_valid;
        [[maybe_unused]] float blk_mul[2], blk_add[2];     // 2^ek and ev of the two 16-token m-tiles
        if constexpr (kBlocks) {
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                const int e = static_cast<int16_t>(blk_exp[2 * c + mt]);
                blk_mul[mt] = __int_as_float((127 + static_cast<int8_t>(e & 0xFF)) << 23);
                blk_add[mt] = static_cast<float>(e >> 8);
            }
        }

        // The chunk's arithmetic; a full chunk (every token valid, the
        // common case) is compiled without the masking of tail tokens.
        auto chunk = [&](auto full) {
            constexpr bool kFull = decltype(full)::value;
            // ---- S^T = K Q^T for the two 16-token m-tiles; each K fragment,
            // converted once, feeds every n-tile of query rows
            float sc[kNT][2][4];
            if constexpr (kSmemQ && !kBf16Cache) {
                // both m-tiles together: a fragment of Q is read once for four products
                uint32_t kw[2][2][8];
    #pragma unroll
                for (int mt = 0; mt < 2; ++mt)
    #pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int r = mt * 16 + half * 8 + gq;
                        const uint4 xa = lds128(ks, swz(r, 2 * tq)), xb = lds128(ks, swz(r, 2 * tq + 1));
                        uint32_t(&w)[8] = kw[mt][half];
                        w[0] = xa.x; w[1] = xa.y; w[2] = xa.z; w[3] = xa.w;
                        w[4] = xb.x; w[5] = xb.y; w[6] = xb.z; w[7] = xb.w;
                    }
    #pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
    #pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
                        sc[nt][mt][0] = sc[nt][mt][1] = sc[nt][mt][2] = sc[nt][mt][3] = 0.f;
    #pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    uint2 qv[kNT];
    #pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
                        qv[nt] = q_frag[(kk * kNT + nt) * 32 + lane];
    #pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const uint32_t k0 = lo16_e4m3x2_to_f16x2(kw[mt][0][kk]), k1 = lo16_e4m3x2_to_f16x2(kw[mt][1][kk]);
                        const uint32_t k2 = hi16_e4m3x2_to_f16x2(kw[mt][0][kk]), k3 = hi16_e4m3x2_to_f16x2(kw[mt][1][kk]);
    #pragma unroll
                        for (int nt = 0; nt < kNT; ++nt)
                            mma_f16(sc[nt][mt], k0, k1, k2, k3, qv[nt].x, qv[nt].y);
                    }
                }
            } else {
    #pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
    #pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
                    sc[nt][mt][0] = sc[nt][mt][1] = sc[nt][mt][2] = sc[nt][mt][3] = 0.f;
                const int r0 = mt * 16 + gq, r1 = r0 + 8;
                if constexpr (kBf16Cache) {
                    uint32_t w0[16], w1[16];
    #pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int line0 = 2 * r0 + (tq >> 1), line1 = 2 * r1 + (tq >> 1);
                        const uint4 x0 = lds128(ks, swz(line0, (tq & 1) * 4 + j));
                        const uint4 x1 = lds128(ks, swz(line1, (tq & 1) * 4 + j));
                        w0[4 * j] = x0.x; w0[4 * j + 1] = x0.y; w0[4 * j + 2] = x0.z; w0[4 * j + 3] = x0.w;
                        w1[4 * j] = x1.x; w1[4 * j + 1] = x1.y; w1[4 * j + 2] = x1.z; w1[4 * j + 3] = x1.w;
                    }
    #pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
    #pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) {
                            uint2 qv;
                            if constexpr (kSmemQ)
                                qv = q_frag[(kk * kNT + nt) * 32 + lane];
                            else
                                qv = make_uint2(qf[nt][kk][0], qf[nt][kk][1]);
                            mma_bf16(sc[nt][mt], w0[2 * kk], w1[2 * kk], w0[2 * kk + 1], w1[2 * kk + 1], qv.x, qv.y);
                        }
                } else {
                    const uint4 x0a = lds128(ks, swz(r0, 2 * tq)), x0b = lds128(ks, swz(r0, 2 * tq + 1));
                    const uint4 x1a = lds128(ks, swz(r1, 2 * tq)), x1b = lds128(ks, swz(r1, 2 * tq + 1));
                    const uint32_t w0[8] = {x0a.x, x0a.y, x0a.z, x0a.w, x0b.x, x0b.y, x0b.z, x0b.w};
                    const uint32_t w1[8] = {x1a.x, x1a.y, x1a.z, x1a.w, x1b.x, x1b.y, x1b.z, x1b.w};
    #pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t k0 = lo16_e4m3x2_to_f16x2(w0[kk]), k1 = lo16_e4m3x2_to_f16x2(w1[kk]);
                        const uint32_t k2 = hi16_e4m3x2_to_f16x2(w0[kk]), k3 = hi16_e4m3x2_to_f16x2(w1[kk]);
    #pragma unroll
                        for (int nt = 0; nt < kNT; ++nt)
                            mma_f16(sc[nt][mt], k0, k1, k2, k3, qf[nt][kk][0], qf[nt][kk][1]);
                    }
                }
            }
            }

            // ---- online softmax (log2 domain); lane holds rows nt*8 + 2tq, +1
            float alpha[kNT][2];
    #pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                float mx[2] = {-INFINITY, -INFINITY};
    #pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    [[maybe_unused]] float mul[2];
                    if constexpr (kBlocks) {
                        mul[0] = qk_col[nt][0] * blk_mul[mt];
                        mul[1] = qk_col[nt][1] * blk_mul[mt];
                    }
    #pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = mt * 16 + gq + ((i & 2) ? 8 : 0);
                        float x;
                        if constexpr (kBlocks)
                            x = fmaf(sc[nt][mt][i], mul[i & 1], blk_add[mt]);
                        else
                            x = sc[nt][mt][i] * qk_col[nt][i & 1];
                        bool keep = true;
                        if constexpr (kWindow && !kFull) {
                            const int at = c * kChunkTokens + row, ti = (tok_col >> (4 * (2 * nt + (i & 1)))) & 15;
                            keep = row < n_valid && at < vis0 + ti && !(at >= sink_end && at < win + ti);
                        } else if constexpr (!kFull) {
                            keep = row < s_valid[nt][i & 1];
                        }
                        x = keep ? x : -INFINITY;
                        sc[nt][mt][i] = x;
                        mx[i & 1] = fmaxf(mx[i & 1], x);
                    }
                }
                float base[2];
    #pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float mnew = fmaxf(m_run[nt][j], warp_max_over_rows(mx[j]));
                    base[j] = mnew == -INFINITY ? 0.f : mnew;
                    alpha[nt][j] = fast_exp2(m_run[nt][j] - base[j]);
                    m_run[nt][j] = mnew;
                }
                const float lift[2] = {base[0] - kLift, base[1] - kLift};
                float psum[2] = {0.f, 0.f};
    #pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    [[maybe_unused]] float tsum[2] = {0.f, 0.f};
    #pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = fast_exp2(sc[nt][mt][i] - lift[i & 1]);
                        sc[nt][mt][i] = p;
                        if constexpr (kBlocks)
                            tsum[i & 1] += p;
                        else
                            psum[i & 1] += p;
                    }
                    if constexpr (kBlocks) {               // back to the softmax's own weights: times 2^-ev
                        const float undo = __int_as_float((127 - static_cast<int>(blk_add[mt])) << 23);
                        psum[0] = fmaf(tsum[0], undo, psum[0]);
                        psum[1] = fmaf(tsum[1], undo, psum[1]);
                    }
                }
    #pragma unroll
                for (int j = 0; j < 2; ++j)
                    l_run[nt][j] = l_run[nt][j] * alpha[nt][j] + psum[j];
    #pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[nt][i][0] *= alpha[nt][0];
                    o[nt][i][1] *= alpha[nt][1];
                    o[nt][i][2] *= alpha[nt][0];
                    o[nt][i][3] *= alpha[nt][1];
                }
            }

            // ---- O^T += V^T P^T; each V fragment, converted once, feeds
            // every n-tile
    #pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                // a weight as the sum of kTerms 16-bit terms, each carrying
                // what the rounding of those before it dropped
                uint32_t pb0[kNT], pb1[kNT];
                [[maybe_unused]] uint32_t pl0[kNT], pl1[kNT], pm0[kNT], pm1[kNT];
    #pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                    uint32_t x0, x1;
                    if constexpr (kBf16Cache) {
                        x0 = f32x2_to_bf16x2(sc[nt][mt][0], sc[nt][mt][1]);
                        x1 = f32x2_to_bf16x2(sc[nt][mt][2], sc[nt][mt][3]);
                    } else {
                        x0 = f32x2_to_f16x2(sc[nt][mt][0], sc[nt][mt][1]);
                        x1 = f32x2_to_f16x2(sc[nt][mt][2], sc[nt][mt][3]);
                    }
                    pb0[nt] = movmatrix_trans(x0);
                    pb1[nt] = movmatrix_trans(x1);
                    if constexpr (kTerms > 1) {
                        const float2 h0 = kBf16Cache ? bf16x2_to_f32x2(x0) : f16x2_to_f32x2(x0);
                        const float2 h1 = kBf16Cache ? bf16x2_to_f32x2(x1) : f16x2_to_f32x2(x1);
                        const float *p = sc[nt][mt];
                        const uint32_t y0 = kBf16Cache ? f32x2_to_bf16x2(p[0] - h0.x, p[1] - h0.y)
                                                       : f32x2_to_f16x2(p[0] - h0.x, p[1] - h0.y);
                        const uint32_t y1 = kBf16Cache ? f32x2_to_bf16x2(p[2] - h1.x, p[3] - h1.y)
                                                       : f32x2_to_f16x2(p[2] - h1.x, p[3] - h1.y);
                        pl0[nt] = movmatrix_trans(y0);
                        pl1[nt] = movmatrix_trans(y1);
                        if constexpr (kTerms > 2) {
                            const float2 l0 = bf16x2_to_f32x2(y0), l1 = bf16x2_to_f32x2(y1);
                            pm0[nt] = movmatrix_trans(f32x2_to_bf16x2(p[0] - h0.x - l0.x, p[1] - h0.y - l0.y));
                            pm1[nt] = movmatrix_trans(f32x2_to_bf16x2(p[2] - h1.x - l1.x, p[3] - h1.y - l1.y));
                        }
                    }
                }
                // V rows of token slots 2tq, 2tq+1, 2tq+8, 2tq+9 of this m-tile
                const int rv = mt * 16 + 2 * tq;
                const int rows[4] = {rv, rv + 1, rv + 8, rv + 9};
                if constexpr (kBf16Cache) {
                    uint32_t R[4][8];
    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int line = 2 * rows[q] + (gq >> 2);
                        const uint4 lo = lds128(vs, swz(line, (gq & 3) * 2));
                        const uint4 hi = lds128(vs, swz(line, (gq & 3) * 2 + 1));
                        bool keep = kFull || rows[q] < n_valid;
                        if constexpr (kWindow && !kFull)
                            keep = keep && !(c * kChunkTokens + rows[q] >= sink_end && c * kChunkTokens + rows[q] < win_first);
                        R[q][0] = keep ? lo.x : 0u; R[q][1] = keep ? lo.y : 0u;
                        R[q][2] = keep ? lo.z : 0u; R[q][3] = keep ? lo.w : 0u;
                        R[q][4] = keep ? hi.x : 0u; R[q][5] = keep ? hi.y : 0u;
                        R[q][6] = keep ? hi.z : 0u; R[q][7] = keep ? hi.w : 0u;
                    }
    #pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t a0 = prmt(R[0][i], R[1][i], 0x5410);
                        const uint32_t a1 = prmt(R[0][i], R[1][i], 0x7632);
                        const uint32_t a2 = prmt(R[2][i], R[3][i], 0x5410);
                        const uint32_t a3 = prmt(R[2][i], R[3][i], 0x7632);
    #pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) {
                            if constexpr (kSumApart) {
                                float t[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_bf16(t, a0, a1, a2, a3, pm0[nt], pm1[nt]);
                                mma_bf16(t, a0, a1, a2, a3, pl0[nt], pl1[nt]);
                                mma_bf16(t, a0, a1, a2, a3, pb0[nt], pb1[nt]);
    #pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    o[nt][i][q] += t[q];
                            } else {
                                mma_bf16(o[nt][i], a0, a1, a2, a3, pb0[nt], pb1[nt]);
                                if constexpr (kTerms > 1)
                                    mma_bf16(o[nt][i], a0, a1, a2, a3, pl0[nt], pl1[nt]);
                            }
                        }
                    }
                } else {
                    uint32_t R[4][4];
    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 v = lds128(vs, swz(rows[q], gq));
                        bool keep = kFull || rows[q] < n_valid;
                        if constexpr (kWindow && !kFull)
                            keep = keep && !(c * kChunkTokens + rows[q] >= sink_end && c * kChunkTokens + rows[q] < win_first);
                        R[q][0] = keep ? v.x : 0u; R[q][1] = keep ? v.y : 0u;
                        R[q][2] = keep ? v.z : 0u; R[q][3] = keep ? v.w : 0u;
                    }
    #pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
                        const uint32_t p01 = prmt(R[0][i >> 1], R[1][i >> 1], sel);
                        const uint32_t p23 = prmt(R[2][i >> 1], R[3][i >> 1], sel);
                        const uint32_t a0 = lo16_e4m3x2_to_f16x2(p01), a1 = hi16_e4m3x2_to_f16x2(p01);
                        const uint32_t a2 = lo16_e4m3x2_to_f16x2(p23), a3 = hi16_e4m3x2_to_f16x2(p23);
    #pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) {
                            if constexpr (kSumApart) {
                                float t[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_f16(t, a0, a1, a2, a3, pl0[nt], pl1[nt]);
                                mma_f16(t, a0, a1, a2, a3, pb0[nt], pb1[nt]);
    #pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    o[nt][i][q] += t[q];
                            } else {
                                mma_f16(o[nt][i], a0, a1, a2, a3, pb0[nt], pb1[nt]);
                                if constexpr (kTerms > 1)
                                    mma_f16(o[nt][i], a0, a1, a2, a3, pl0[nt], pl1[nt]);
                            }
                        }
                    }
                }
            }
        };
        const int chunk_end = (c + 1) * kChunkTokens;
        if (kWindow ? chunk_end <= full_to && (chunk_end <= sink_end || chunk_end - kChunkTokens >= mask_hi)
                    : tok + kChunkTokens <= full_end)
            chunk(std::true_type{});
        else
            chunk(std::false_type{});

        // ---- refill this stage with the chunk kStages ahead
        __syncwarp();
        if (it + T::kStages < my_chunks) {
            fence_proxy_async_smem();
            issue(it + T::kStages);
        }
    }

    if (failed) {
        // Drain the copies this warp still has in flight -- the one it gave
        // up on and those issued after it -- with the full limit, so none
        // lands in shared memory after the CTA has moved on.  A drain that
        // gives up too is reported as bit 1.
        if (lane == 0) {
            atomicOr(&g_device_error, 1u);
            s_failed = 1;
        }
        const int issued = my_chunks < it + T::kStages ? my_chunks : it + T::kStages;
        bool drained = true;
        for (int j = it; j < issued; ++j)
            drained &= mbar_wait_bounded(&my_full[j % T::kStages], (j / T::kStages) & 1, kCopyWaitLimitNs);
        if (!drained && lane == 0)
            atomicOr(&g_device_error, 2u);
    }
    if (step_check) {                                      // this thread's tag entries
        cp_async_wait_all();
        bool stale = false;
#pragma unroll
        for (int k = 0; k < kIdsPerThread; ++k) {
            const int i = threadIdx.x + k * kThreads;
            if (i < n_pages)
                stale |= tag_live[i] != tag_want[i];
        }
        if (stale)
            s_stale = 1;
    }
    __syncthreads();
    KVQ_STAMP(3);
    if (s_stale || s_failed) {                             // a failed check outranks a timeout
        if constexpr (kCluster) {
            const bool stale = cluster_finish<kMulti, kWindow>(a, R, s_stale ? kPartialStale : kPartialInvalid, part, finisher);
            if (split == finisher)
                finish_here(stale);
        } else
            drop_split<kMulti, kWindow>(a, R, split, nsplit, reinterpret_cast<float *>(smem),
                       s_stale ? kLseStale : kLseInvalid);
        return;
    }

    // ---- merge the four warps' states in shared memory (ring is free now)
    float *sm_o = reinterpret_cast<float *>(smem);                     // [kWarps][kRowsT][128]
    float *sm_m = sm_o + kWarps * kRowsT * kMergeStride;              // [kWarps][kRowsT]
    float *sm_l = sm_m + kWarps * kRowsT;                             // [kWarps][kRowsT]
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            l_run[nt][j] = warp_sum_over_rows(l_run[nt][j]);
    {
        float *ow = sm_o + warp * kRowsT * kMergeStride;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            const int r = nt * kMaxGroup + 2 * tq;                  // rows r, r + 1 of this lane
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = merge_col(16 * gq + 2 * i);
                *reinterpret_cast<float2 *>(ow + r * kMergeStride + c) = make_float2(o[nt][i][0], o[nt][i][2]);
                *reinterpret_cast<float2 *>(ow + (r + 1) * kMergeStride + c) =
                    make_float2(o[nt][i][1], o[nt][i][3]);
            }
            if (gq == 0) {
                sm_m[warp * kRowsT + r] = m_run[nt][0];
                sm_m[warp * kRowsT + r + 1] = m_run[nt][1];
                sm_l[warp * kRowsT + r] = l_run[nt][0];
                sm_l[warp * kRowsT + r + 1] = l_run[nt][1];
            }
        }
    }
    __syncthreads();

    // per-row merge factors of the four warps, computed once (thread h)
    float *sm_f = sm_l + kWarps * kRowsT;                             // [kRowsT][kWarps] weights
    float *sm_t = sm_f + kRowsT * kWarps;                             // [kRowsT] 1 / sum, [kRowsT] lse
    if (threadIdx.x < R.nrows) {
        const int h = threadIdx.x;
        float mmax = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            mmax = fmaxf(mmax, sm_m[w * kRowsT + h]);
        float lsum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = sm_m[w * kRowsT + h];
            const float f = mw == -INFINITY ? 0.f : fast_exp2(mw - mmax);
            sm_f[h * kWarps + w] = f;
            lsum += sm_l[w * kRowsT + h] * f;
        }
        // a row that saw no token of this split (causal limit): weight 0
        if constexpr (kWindow) {
            sm_t[h] = lsum == 0.f ? 0.f : vscale / lsum;
            sm_t[kRowsT + h] = lsum == 0.f ? -INFINITY : lsum == lsum ? mmax + __log2f(lsum) - kLift : INFINITY;
        } else {
            sm_t[h] = lsum > 0.f ? vscale / lsum : 0.f;
            sm_t[kRowsT + h] = lsum > 0.f ? mmax + __log2f(lsum) : -INFINITY;
        }
    }
    __syncthreads();
    if constexpr (kWindow) {
        // warp w takes rows w, w + 4, ..; a lane four dims of each
        const int d = 4 * lane, c = merge_col(d);
#pragma unroll
        for (int q = 0; q < kRowsT / kWarps; ++q) {
            const int h = warp + q * kWarps;
            if (h >= R.nrows)
                break;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float *row = sm_o + (w * kRowsT + h) * kMergeStride + c;
                const float2 lo = *reinterpret_cast<const float2 *>(row), hi = *reinterpret_cast<const float2 *>(row + 2);
                const float f = sm_f[h * kWarps + w];
                acc.x += lo.x * f;
                acc.y += lo.y * f;
                acc.z += hi.x * f;
                acc.w += hi.y * f;
            }
            const float t = sm_t[h];
            acc = make_float4(acc.x * t, acc.y * t, acc.z * t, acc.w * t);
            if constexpr (kCluster) {
                *reinterpret_cast<float4 *>(part + kRowsT + h * kHeadDim + d) = acc;
                if (lane == 0)
                    part[h] = sm_t[kRowsT + h];
            } else if (nsplit == 1) {
                store_out4(a.out, R.ids[h] * kHeadDim + d, acc, a.out_fp32);
            } else {
                const int64_t at = R.part(a, h, split);
                *reinterpret_cast<float4 *>(a.ws_o + at * kHeadDim + d) = acc;
                if (lane == 0)
                    a.ws_lse[at] = sm_t[kRowsT + h];
            }
        }
    } else
    for (int d = threadIdx.x; d < kHeadDim; d += kThreads)
#pragma unroll
    for (int h = 0; h < kRowsT; ++h) {
        if (h >= R.nrows)
            break;
        float acc = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            acc += sm_o[(w * kRowsT + h) * kMergeStride + merge_col(d)] * sm_f[h * kWarps + w];
        const float val = acc * sm_t[h];
        const int64_t bh = R.id(a, h);
        if constexpr (kCluster) {
            part[kRowsT + h * kHeadDim + d] = val;
            if (d == 0)
                part[h] = sm_t[kRowsT + h];
        } else if (nsplit == 1) {
            store_out(a.out, bh * kHeadDim + d, val, a.out_fp32);
        } else {
            a.ws_o[(bh * a.max_splits + split) * kHeadDim + d] = val;
            if (d == 0)
                a.ws_lse[bh * a.max_splits + split] = sm_t[kRowsT + h];
        }
    }
    KVQ_STAMP(4);
    if constexpr (kCluster) {
        const bool stale = cluster_finish<kMulti, kWindow>(a, R, kPartialOk, part, finisher);
        if (split == finisher)
            finish_here(stale);
    } else if (nsplit > 1) {
        publish_and_combine<kMulti, kWindow>(a, R, nsplit, reinterpret_cast<float *>(smem) + (kMulti ? 0 : kScratchOffset));
    } else if (step_check) {                               // one split: its own verdict
        finish_here(false);
    }
    KVQ_STAMP(6);
}

// Units (of 1 << unit_shift tokens) that a call shows of a request of `real`
// tokens; 0 if its outputs are zeros.
__device__ __forceinline__ int shown_units(const DecodeArgs &a, int64_t real, bool aborted, int ps_shift)
{
    if (aborted || real <= 0 || real > static_cast<int64_t>(a.max_pages_per_seq) << ps_shift)
        return 0;
    return static_cast<int>((shown_context(a, real, ps_shift).len + (1 << a.unit_shift) - 1) >> a.unit_shift);
}

// A balanced launch.  The host knows neither the lengths nor, with a table
// padded for growth, how far they are from the row's capacity; a grid of equal
// splits of the longest possible request leaves most of the GPU idle behind
// the longest real one.  Here the whole batch is one line of units, request
// after request, KV head after KV head, row block after row block, and CTA c
// takes places [c S, (c + 1) S) of it: S is the line's length divided by the
// resident CTAs (or by a whole number of waves of them, where a share would
// pass 8,192 tokens).  A share that crosses (request, KV head) borders is
// worked off border by border, one split each.  Such a border costs the CTA a
// drained and refilled pipeline, a merge and a publication, about as long as
// it streams pair_cost units, so every pair has that many empty places in
// front of its units: a CTA with a border gets less to stream and ends with
// the others.  Every CTA finds its share alone, from a block-wide scan of the
// lengths.  A pair's splits are consecutive CTAs, so (CTA + pair) numbers the
// launch's splits without collisions: the workspace slot.  S depends on
// nothing but the lengths, so results repeat.  (The host keeps the line's
// length within 31 bits.)
//
// Share finds CTA c's places and walks them.  It lies in shared memory, and
// thread 0 moves it on, so that a split's arithmetic keeps its registers.
template <bool kMulti>
struct Share {
    int lines;                               // pairs (KV head x row block) per request
    int share, x, end;                       // S, the next place, the end of the CTA's places
    int acc, u;                              // places before request r, places of each of its pairs
    int r;
    int64_t real;                            // tokens of request r
    Job job;                                 // the split at x

    // Places of each pair of request r.
    __device__ __forceinline__ int places(const DecodeArgs &a, int r, int ps_shift, int64_t &real) const
    {
        real = __ldcg(a.seq_lens + r);
        const bool aborted = a.abort_flags != nullptr && __ldcg(a.abort_flags + r) != 0;
        const int n = shown_units(a, real, aborted, ps_shift);
        return n > 0 ? n + a.pair_cost : 0;
    }

    // False if the CTA has none.  Also writes the zeros of the requests that
    // show nothing, one CTA each.  Called by the whole block.
    __device__ __forceinline__ bool find(const DecodeArgs &a, int ps_shift)
    {
        __shared__ int s_sum[kWarps];
        __shared__ bool s_some;
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        const int lines = a.num_kv_heads * (kMulti ? a.row_blocks : 1);
        // thread t sums requests [t m, (t + 1) m)
        const int m = (a.batch + kThreads - 1) / kThreads;
        const int r0 = min(a.batch, static_cast<int>(threadIdx.x) * m), r1 = min(a.batch, r0 + m);
        int64_t real = 0;
        int mine = 0, first = 0;
        for (int i = r0; i < r1; ++i) {
            const int n = places(a, i, ps_shift, real);
            first = i == r0 ? n : first;
            mine += n;
        }
        int upto = mine;                                   // inclusive scan over the warp
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, upto, off);
            upto += lane >= off ? o : 0;
        }
        if (lane == 31)
            s_sum[warp] = upto;
        if (threadIdx.x == 0)
            s_some = false;
        __syncthreads();
        int before = upto - mine, total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? s_sum[w] : 0;
            total += s_sum[w];
        }
        for (int64_t i = blockIdx.x; i < a.batch; i += gridDim.x) {
            int64_t unused;
            if (places(a, static_cast<int>(i), ps_shift, unused) == 0) {
                const int64_t n = static_cast<int64_t>(a.n_query) * a.num_q_heads * kHeadDim;
                for (int64_t j = threadIdx.x; j < n; j += kThreads)
                    store_out(a.out, i * n + j, 0.f, a.out_fp32);
            }
        }
        const int all = total * lines;
        const int wave = a.resident_ctas * (kMaxShareTokens >> a.unit_shift);
        const int parts = a.resident_ctas * max((all + wave - 1) / wave, 1);
        const int share = max(a.min_split_units, (all + parts - 1) / parts);
        const int x = static_cast<int>(blockIdx.x) * share, end = min(all, x + share);
        // the one thread whose requests hold place x
        if (static_cast<int64_t>(blockIdx.x) * share < all && x >= before * lines && x < (before + mine) * lines) {
            int sum = before, n = first, i = r0;
            if (m > 1)
                for (n = places(a, i, ps_shift, real); x >= (sum + n) * lines; n = places(a, ++i, ps_shift, real))
                    sum += n;
            *this = {lines, share, x, end, sum, n, i, real, {}};
            s_some = set_job(a);
        }
        __syncthreads();
        return s_some;
    }

    // The split at x; moves x to the share's next pair.  False if the share
    // ends in the empty places in front of the pair's units.
    __device__ __forceinline__ bool set_job(const DecodeArgs &a)
    {
        const int line = (x - acc * lines) / u, start = acc * lines + line * u + a.pair_cost;
        const int from = max(x, start), to = min(end, start - a.pair_cost + u);
        const int c0 = start / share;
        x = to;
        if (from >= to)
            return false;
        job.b = r;
        job.kvh = kMulti ? line / a.row_blocks : line;
        job.rb = kMulti ? line % a.row_blocks : 0;
        job.split = static_cast<int>(blockIdx.x) - c0;
        job.nsplit = (start - a.pair_cost + u - 1) / share - c0 + 1;
        job.t0 = static_cast<int64_t>(from - start) << a.unit_shift;
        job.span = (to - from) << a.unit_shift;
        job.base = c0 + static_cast<int64_t>(r) * lines + line;
        job.real = real;
        if (a.ws_pairs != nullptr && job.split == 0)       // for the combine
            a.ws_pairs[static_cast<int64_t>(r) * lines + line] = make_int2(static_cast<int>(job.base), job.nsplit);
        return true;
    }

    // On to the next job, by the whole block; false at the end of the share.
    __device__ __forceinline__ bool next(const DecodeArgs &a, int ps_shift)
    {
        __shared__ bool s_more;
        // the next split's copies overwrite what this one's merge read
        fence_proxy_async_smem();
        __syncthreads();
        if (threadIdx.x == 0)
            s_more = advance(a, ps_shift);
        __syncthreads();
        return s_more;
    }

    __device__ __forceinline__ bool advance(const DecodeArgs &a, int ps_shift)
    {
        if (x >= end)
            return false;
        if (x == (acc + u) * lines) {                      // the next request that shows something
            acc += u;
            do {
                if (++r >= a.batch)
                    return false;                          // only if the lengths changed meanwhile
                u = places(a, r, ps_shift, real);
            } while (u == 0);
        }
        return set_job(a);
    }
};

template <bool kBf16Cache, bool kPreciseP, bool kCluster, bool kMulti, bool kWindow, bool kBlocks>
__global__ void __launch_bounds__(kThreads, min_ctas(kMulti, kWindow))
decode_split_kernel(const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap v_map, const DecodeArgs a)
{
    static_assert(!kBlocks || (kWindow && !kBf16Cache), "the block-scaled build is an FP8 build with a window");
    KVQ_STAMP(0);
    // Launched as a programmatic dependent of the previous kernel on the
    // stream (in a decode step: the tag check): the CTA can be resident and
    // have its tensor maps fetched while that kernel runs, and it reads no
    // global memory until the wait has returned, that is until the previous
    // kernel has completed and its writes are visible.  (Asking L2 for the
    // split's first pages before the wait made the step slower: those
    // requests compete with the check for the memory system.)
    if (threadIdx.x == 0) {
        prefetch_tensor_map(&k_map);
        prefetch_tensor_map(&v_map);
    }
    grid_dependency_wait();
    KVQ_STAMP(1);

    Job job;                                               // unused without a window
    job.split = blockIdx.x;
    job.b = blockIdx.z;
    job.kvh = kMulti ? static_cast<int>(blockIdx.y) / a.row_blocks : static_cast<int>(blockIdx.y);
    job.rb = kMulti ? static_cast<int>(blockIdx.y) % a.row_blocks : 0;
    job.nsplit = 0;
    job.span = a.split_tokens;
    job.t0 = static_cast<int64_t>(job.split) * a.split_tokens;
    job.base = job.real = -1;
    if constexpr (kWindow && !kCluster) {
        const bool balanced = a.resident_ctas > 0;
        const int ps_shift = __ffs(a.page_size) - 1;
        __shared__ Share<kMulti> share;
        if (balanced && !share.find(a, ps_shift))
            return;
        for (bool first = true;; first = false) {
            if (balanced)
                job = share.job;
            run_split<kBf16Cache, kPreciseP, kCluster, kMulti, kWindow, kBlocks>(k_map, v_map, a, job, first);
            if (!balanced || !share.next(a, ps_shift))
                return;
        }
    } else {
        run_split<kBf16Cache, kPreciseP, kCluster, kMulti, kWindow, kBlocks>(k_map, v_map, a, job, true);
    }
}

template <bool kBf16, bool kPrecise, bool kCluster, bool kMulti = false, bool kWindow = false, bool kBlocks = false>
cudaError_t configure(int dev)
{
    static int configured[64] = {0};
    if (dev >= 0 && dev < 64 && configured[dev])
        return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(decode_split_kernel<kBf16, kPrecise, kCluster, kMulti, kWindow, kBlocks>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_bytes<kBf16, kMulti, kWindow>());
    if (e == cudaSuccess && dev >= 0 && dev < 64)
        configured[dev] = 1;
    return e;
}

template <bool kBf16, bool kCluster, bool kMulti, bool kWindow>
cudaLaunchConfig_t launch_config(const DecodeArgs &a, dim3 grid, cudaStream_t stream,
                                 cudaLaunchAttribute (&attr)[2])
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<kBf16, kMulti, kWindow>();
    cfg.stream = stream;
    // programmatic dependent launch: the grid may start while the previous
    // kernel on the stream finishes; the kernel waits before its first read
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (kCluster) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(a.max_splits);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    cfg.attrs = attr;
    return cfg;
}

template <bool kBf16, bool kPrecise, bool kCluster, bool kMulti, bool kWindow, bool kBlocks>
cudaError_t launch_split(const DecodeArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                         cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    e = configure<kBf16, kPrecise, kCluster, kMulti, kWindow, kBlocks>(dev);
    if (e != cudaSuccess)
        return e;
    const dim3 grid = kWindow && !kCluster && a.resident_ctas > 0
                          ? dim3(static_cast<unsigned>(a.balanced_ctas))
                          : dim3(static_cast<unsigned>(a.max_splits),
                                 static_cast<unsigned>(a.num_kv_heads * a.row_blocks),
                                 static_cast<unsigned>(a.batch));
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = launch_config<kBf16, kCluster, kMulti, kWindow>(a, grid, stream, attr);
    e = cudaLaunchKernelEx(&cfg, decode_split_kernel<kBf16, kPrecise, kCluster, kMulti, kWindow, kBlocks>, k_map,
                           v_map, a);
    if (e != cudaSuccess)
        return e;
    return cudaGetLastError();
}

// The build for the call's cache type, output type, split form and row count.
template <bool kWindow, bool kBlocks, bool kCluster, bool kMulti>
cudaError_t launch_variant(const DecodeArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                           cudaStream_t stream)
{
    if constexpr (!kBlocks)
        if (a.bf16_cache)
            return a.out_fp32 ? launch_split<true, true, kCluster, kMulti, kWindow, kBlocks>(a, k_map, v_map, stream)
                              : launch_split<true, false, kCluster, kMulti, kWindow, kBlocks>(a, k_map, v_map, stream);
    return a.out_fp32 ? launch_split<false, true, kCluster, kMulti, kWindow, kBlocks>(a, k_map, v_map, stream)
                      : launch_split<false, false, kCluster, kMulti, kWindow, kBlocks>(a, k_map, v_map, stream);
}

template <bool kWindow, bool kBlocks>
cudaError_t launch_build(const DecodeArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                         cudaStream_t stream)
{
    if (a.batch == 0)
        return cudaSuccess;
    if (a.n_query > 1)                      // several query tokens: the causal, row-blocked build
        return a.cluster ? launch_variant<kWindow, kBlocks, true, true>(a, k_map, v_map, stream)
                         : launch_variant<kWindow, kBlocks, false, true>(a, k_map, v_map, stream);
    return a.cluster ? launch_variant<kWindow, kBlocks, true, false>(a, k_map, v_map, stream)
                     : launch_variant<kWindow, kBlocks, false, false>(a, k_map, v_map, stream);
}

// How many clusters of n split CTAs can be resident at once on the current
// device (0 if clusters of n cannot be used).
template <bool kBf16, bool kMulti, bool kWindow>
int cluster_capacity_query(int n)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || configure<kBf16, false, true, kMulti, kWindow>(dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    DecodeArgs a = {};
    a.max_splits = n;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg =
        launch_config<kBf16, true, kMulti, kWindow>(a, dim3(static_cast<unsigned>(n), 1, 1), nullptr, attr);
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, decode_split_kernel<kBf16, false, true, kMulti, kWindow, false>,
                                       &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return clusters;
}

// The same, asked once per device, n and build.
template <bool kWindow>
int cluster_capacity(int n, bool bf16_cache, bool multi)
{
    if (n < 2 || n > kMaxCluster)
        return 0;
    static std::mutex mu;
    static std::map<std::tuple<int, int, bool, bool>, int> cache;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    std::lock_guard<std::mutex> lock(mu);
    const auto key = std::make_tuple(dev, n, bf16_cache, multi);
    auto it = cache.find(key);
    if (it != cache.end())
        return it->second;
    const int c = multi ? (bf16_cache ? cluster_capacity_query<true, true, kWindow>(n)
                                      : cluster_capacity_query<false, true, kWindow>(n))
                        : (bf16_cache ? cluster_capacity_query<true, false, kWindow>(n)
                                      : cluster_capacity_query<false, false, kWindow>(n));
    cache[key] = c;
    return c;
}

// Read (and, if asked, reset) this build's error word.
cudaError_t read_error_word(uint32_t *bits, bool clear)
{
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof v);
    if (e != cudaSuccess)
        return e;
    if (bits)
        *bits = v;
    if (clear) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero);
    }
    return e;
}

} // namespace
} // namespace kvq
