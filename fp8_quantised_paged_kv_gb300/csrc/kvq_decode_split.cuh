// kvq_decode_split.cuh -- paged decode attention over an FP8 e4m3 (or BF16) KV
// cache, split along the context, with the log-sum-exp combine of the splits
// fused into the same launch (the builds without a window always, the others
// where that is faster).  What works off one split stands in
// kvq_decode_split_body.cuh.  Compiled five times: kvq_decode.cu (per-head
// scales, every token), kvq_decode_window.cu (the same caches behind a sliding
// window with sinks), kvq_decode_blocks.cu (the block-scaled cache), and, with
// KVQ_OWN_ROWS, kvq_decode_own.cu and kvq_decode_own_blocks.cu (either cache
// past the pages that requests share: kSharing below).
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
#include "kvq_prefix.cuh"
#include "kvq_ptx.cuh"
#include "kvq_rowops.cuh"
#include "kvq_view.cuh"

namespace kvq {

namespace {

// Builds behind shared pages (kvq_prefix.cu attends to those): a request shows
// what its own row holds past them, as a context with the shared pages for a
// hole; balanced launches only; every split goes to the workspace, one of a
// request's only split among them, and launch_combine_prefix joins them.
#ifdef KVQ_OWN_ROWS
constexpr bool kSharing = true;
using CallArgs = PrefixArgs;
#else
constexpr bool kSharing = false;
using CallArgs = ViewArgs;
#endif
// An input of the call.  Behind shared pages through L2: those builds run
// without a wait for the grids before them (decode_split_kernel), so that what an
// SM still holds of an input may be older than what was written to it.
template <typename T>
__device__ __forceinline__ T read_input(const T *p)
{
    if constexpr (kSharing)
        return __ldcg(p);
    else
        return __ldg(p);
}
template <typename T>
__device__ __forceinline__ T read_plain(const T *p)
{
    if constexpr (kSharing)
        return __ldcg(p);
    else
        return *p;
}
template <bool kWindow>
using ArgsOf = std::conditional_t<kWindow, CallArgs, DecodeArgs>;

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
__device__ void publish_and_combine(const ArgsOf<kNanFlows> &a, const Rows<kMulti, kNanFlows> &R, int nsplit, float *scratch)
{
    if constexpr (kNanFlows)
        if (a.combine_apart)                               // launch_combine_rows does it
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
__device__ void drop_split(const ArgsOf<kNanFlows> &a, const Rows<kMulti, kNanFlows> &R, int split, int nsplit, float *smem,
                           uint32_t lse_bits = kLseInvalid)
{
    if (!kSharing && nsplit == 1) {
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
    int shared;                              // kSharing: those of them that are not its own row's
};

// Launched as a programmatic dependent of the previous kernel on the
// stream (in a decode step: the tag check): the CTA can be resident and
// have its tensor maps fetched while that kernel runs, and it reads no
// global memory until the wait has returned, that is until the previous
// kernel has completed and its writes are visible.  (Asking L2 for the
// split's first pages before the wait made the step slower: those
// requests compete with the check for the memory system.)
__device__ __forceinline__ void start_dependent(const CUtensorMap &k_map, const CUtensorMap &v_map)
{
    if (threadIdx.x == 0) {
        prefetch_tensor_map(&k_map);
        prefetch_tensor_map(&v_map);
    }
    grid_dependency_wait();
    KVQ_STAMP(1);
}

template <bool kBf16Cache, bool kPreciseP, bool kCluster, bool kMulti, bool kWindow, bool kBlocks>
__device__ __forceinline__ void run_split(const CUtensorMap &k_map, const CUtensorMap &v_map, const ArgsOf<kWindow> &a,
                                          const Job &job, bool first)
{
#include "kvq_decode_split_body.cuh"
}

// Units (of 1 << unit_shift tokens) that a call shows of a request of `real`
// tokens; 0 if its outputs are zeros.
__device__ __forceinline__ int shown_units(const CallArgs &a, int64_t real, bool aborted, int shared, int ps_shift)
{
    if (aborted || real <= 0 || real > static_cast<int64_t>(a.max_pages_per_seq) << ps_shift)
        return 0;
    return static_cast<int>((own_context(a, real, shared, ps_shift).len + (1 << a.unit_shift) - 1) >> a.unit_shift);
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
    int number;                              // of the share: the CTA's, but for kSharing
    int acc, u;                              // places before request r, places of each of its pairs
    int r;
    int64_t real;                            // tokens of request r
    int shared;                              // kSharing: those not its own row's
    Job job;                                 // the split at x

    // Places of each pair of request r.
    __device__ __forceinline__ int places(const CallArgs &a, int r, int ps_shift, int64_t &real, int &shared, Work &work) const
    {
        real = __ldcg(a.seq_lens + r);
        const bool aborted = a.abort_flags != nullptr && __ldcg(a.abort_flags + r) != 0;
        shared = shared_tokens(a, r, ps_shift, work);
        const int n = shown_units(a, real, aborted, shared, ps_shift);
        return n > 0 ? n + a.pair_cost : 0;
    }

    // False if the CTA has none.  Also writes the zeros of the requests that
    // show nothing, one CTA each.  Called by the whole block.  kSharing: of the
    // CTA's shares the turn-th; *past if there are none after it.
    __device__ __forceinline__ bool find(const CallArgs &a, int ps_shift, int turn = 0, bool *past = nullptr)
    {
        __shared__ int s_sum[kWarps];
        __shared__ bool s_some;
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        const int lines = a.num_kv_heads * (kMulti ? a.row_blocks : 1);
        // thread t sums requests [t m, (t + 1) m)
        const int m = (a.batch + kThreads - 1) / kThreads;
        const int r0 = min(a.batch, static_cast<int>(threadIdx.x) * m), r1 = min(a.batch, r0 + m);
        int64_t real = 0;
        int shared = 0;
        int mine = 0, first = 0;
        Work work = {0, 0};
        for (int i = r0; i < r1; ++i) {
            const int n = places(a, i, ps_shift, real, shared, work);
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
        if constexpr (kSharing) {
            __shared__ long long s_work[2][kWarps];
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                work.shared += __shfl_xor_sync(0xFFFFFFFFu, work.shared, off);
                work.own += __shfl_xor_sync(0xFFFFFFFFu, work.own, off);
            }
            if (lane == 0) {
                s_work[0][warp] = work.shared;
                s_work[1][warp] = work.own;
            }
            __syncthreads();
            work = {0, 0};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                work.shared += s_work[0][w];
                work.own += s_work[1][w];
            }
        }
        __syncthreads();
        int before = upto - mine, total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? s_sum[w] : 0;
            total += s_sum[w];
        }
        for (int64_t i = blockIdx.x; !kSharing && i < a.batch; i += gridDim.x) {
            int64_t unused;
            int unshared;
            if (places(a, static_cast<int>(i), ps_shift, unused, unshared, work) == 0) {
                const int64_t n = static_cast<int64_t>(a.n_query) * a.num_q_heads * kHeadDim;
                for (int64_t j = threadIdx.x; j < n; j += kThreads)
                    store_out(a.out, i * n + j, 0.f, a.out_fp32);
            }
        }
        const int all = total * lines;
        // (kSharing: the grid is what all SMs hold, its first `ctas` CTAs take the
        // shares in turn, and the workspace has places for balanced_ctas of them)
        const int ctas = own_ctas(a, work);
        const int wave = ctas * (kMaxShareTokens >> a.unit_shift);
        int parts = ctas * max((all + wave - 1) / wave, 1);
        if constexpr (kSharing)
            parts = min(parts, a.balanced_ctas);
        const int share = max(a.min_split_units, (all + parts - 1) / parts);
        const int64_t mine_at = kSharing ? blockIdx.x + static_cast<int64_t>(turn) * ctas : blockIdx.x;
        const bool none = mine_at * share >= all || (kSharing && static_cast<int>(blockIdx.x) >= ctas);
        if constexpr (kSharing)
            *past = none || (mine_at + ctas) * share >= all;
        const int x = static_cast<int>(mine_at) * share, end = min(all, x + share);
        // the one thread whose requests hold place x
        if (!none && x >= before * lines && x < (before + mine) * lines) {
            int sum = before, n = first, i = r0;
            if (m > 1)
                for (n = places(a, i, ps_shift, real, shared, work); x >= (sum + n) * lines;
                     n = places(a, ++i, ps_shift, real, shared, work))
                    sum += n;
            *this = {lines, share, x, end, static_cast<int>(mine_at), sum, n, i, real, shared, {}};
            s_some = set_job(a);
        }
        __syncthreads();
        return s_some;
    }

    // The split at x; moves x to the share's next pair.  False if the share
    // ends in the empty places in front of the pair's units.
    __device__ __forceinline__ bool set_job(const CallArgs &a)
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
        job.split = (kSharing ? number : static_cast<int>(blockIdx.x)) - c0;
        job.nsplit = (start - a.pair_cost + u - 1) / share - c0 + 1;
        job.t0 = static_cast<int64_t>(from - start) << a.unit_shift;
        job.span = (to - from) << a.unit_shift;
        job.base = c0 + static_cast<int64_t>(r) * lines + line;
        job.real = real;
        job.shared = shared;
        if (a.ws_pairs != nullptr && job.split == 0)       // for the combine
            a.ws_pairs[static_cast<int64_t>(r) * lines + line] = make_int2(static_cast<int>(job.base), job.nsplit);
        return true;
    }

    // On to the next job, by the whole block; false at the end of the share.
    __device__ __forceinline__ bool next(const CallArgs &a, int ps_shift)
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

    __device__ __forceinline__ bool advance(const CallArgs &a, int ps_shift)
    {
        if (x >= end)
            return false;
        if (x == (acc + u) * lines) {                      // the next request that shows something
            acc += u;
            do {
                if (++r >= a.batch)
                    return false;                          // only if the lengths changed meanwhile
                Work unused;
                u = places(a, r, ps_shift, real, shared, unused);
            } while (u == 0);
        }
        return set_job(a);
    }
};

template <bool kBf16Cache, bool kPreciseP, bool kCluster, bool kMulti, bool kWindow, bool kBlocks>
__global__ void __launch_bounds__(kThreads, min_ctas(kMulti, kWindow))
decode_split_kernel(const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap v_map, const ArgsOf<kWindow> a)
{
    static_assert(!kBlocks || (kWindow && !kBf16Cache), "the block-scaled build is an FP8 build with a window");
    KVQ_STAMP(0);
    if constexpr (!kWindow && kCluster) {                  // the split that the CTA's place in the grid names
        constexpr Job job{};                               // not looked at
        constexpr bool first = true;
#include "kvq_decode_split_body.cuh"
    } else {
        if constexpr (kSharing) {
            // Launched beside the kernel over the shared pages, once every CTA of
            // that one has waited for the launches before it and said so.  Nothing
            // here reads what that kernel writes but a number in own_takers; CTA 0
            // ends after it, so that the combine, which waits for this launch,
            // comes after both.
            //
            // A wait here would be one for that kernel's end.  In its place stands
            // the number: that kernel releases it after its wait, one thread of
            // each CTA here acquires it, and the barrier passes the order on to the
            // others, the fence to their bulk copies.  What that leaves to the
            // order in which the two start: that the number read is not an older one.
            // Every input is read through L2 (read_input).
            if (threadIdx.x == 0) {
                prefetch_tensor_map(&k_map);
                prefetch_tensor_map(&v_map);
            }
            grid_launch_dependents();
            // one thread looks for all: CTA 0 may write the number at any moment
            if constexpr (kWindow)
                if (__syncthreads_or(threadIdx.x == 0 && nothing_left(a)))
                    return;
            fence_proxy_async_global();
        } else {
            start_dependent(k_map, v_map);
        }
        Job job;                                           // unused without a window
        job.split = blockIdx.x;
        job.b = blockIdx.z;
        job.kvh = kMulti ? static_cast<int>(blockIdx.y) / a.row_blocks : static_cast<int>(blockIdx.y);
        job.rb = kMulti ? static_cast<int>(blockIdx.y) % a.row_blocks : 0;
        job.nsplit = 0;
        job.span = a.split_tokens;
        job.t0 = static_cast<int64_t>(job.split) * a.split_tokens;
        job.base = job.real = -1;
        job.shared = 0;
        if constexpr (kWindow && !kCluster) {
            const bool balanced = a.resident_ctas > 0;
            const int ps_shift = __ffs(a.page_size) - 1;
            __shared__ Share<kMulti> share;
            if constexpr (kSharing) {
                bool first = true, past = false;
                for (int turn = 0; !past; ++turn) {
                    if (share.find(a, ps_shift, turn, &past))
                        do {
                            job = share.job;
                            run_split<kBf16Cache, kPreciseP, kCluster, kMulti, kWindow, kBlocks>(k_map, v_map, a, job,
                                                                                                 first);
                            first = false;
                        } while (share.next(a, ps_shift));
                }
                if (blockIdx.x == 0)
                    grid_dependency_wait();
                return;
            }
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
cudaError_t launch_split(const ArgsOf<kWindow> &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                         cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    e = configure<kBf16, kPrecise, kCluster, kMulti, kWindow, kBlocks>(dev);
    if (e != cudaSuccess)
        return e;
    dim3 grid(static_cast<unsigned>(a.max_splits), static_cast<unsigned>(a.num_kv_heads * a.row_blocks),
              static_cast<unsigned>(a.batch));
    if constexpr (kWindow && !kCluster)
        if (a.resident_ctas > 0)
            grid = dim3(static_cast<unsigned>(kSharing ? a.resident_ctas : a.balanced_ctas));
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
cudaError_t launch_variant(const ArgsOf<kWindow> &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
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
cudaError_t launch_build(const ArgsOf<kWindow> &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
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
