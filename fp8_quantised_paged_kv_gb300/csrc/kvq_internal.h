// kvq_internal.h -- launch interfaces shared by the C ABI (kvq_abi.cu) and
// the kernel translation units.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace kvq {

constexpr int kHeadDim = 128;
constexpr int kChunkTokens = 32;     // tokens one warp consumes per pipeline stage
constexpr int kBlockTokens = 16;     // tokens of one KV head that share an exponent (block-scaled cache)
constexpr int kBlockExpMin = -48, kBlockExpMax = 48;   // exponents the append makes
// Exponents that the attention reads as they are (others as the nearer border).
// K's: 2^ek is a normal fp32 number.  V's are those that the append makes: the
// softmax's denominator is the sum of weights w = 2^(s + ev - M), held 2^15 times
// larger, times 2^-ev.  Exponents more than 96 apart would flush weights of
// 2^-45 of the largest and more to zero before 2^-ev brought them back, and 8,192
// of them at 2^-ev = 2^100 would overflow.
constexpr int kReadKeyExpMin = -126, kReadValueExpMin = kBlockExpMin, kReadValueExpMax = kBlockExpMax;
constexpr int kMaxGroup = 8;         // query heads per KV head on one mma n-tile
constexpr int kMaxCluster = 8;       // splits merged inside one thread-block cluster
constexpr int kMaxSplitsTotal = 1024;  // splits of one (request, KV head)

struct AppendArgs {
    const void *k_new, *v_new;       // bf16 [T][Hkv][D]
    const int64_t *slot_mapping;     // [T]
    const float *k_scale, *v_scale;  // [Hkv]
    const uint8_t *abort_flags;      // [T] or null
    void *k_cache, *v_cache;
    int32_t num_tokens, num_kv_heads, page_size;
    int64_t num_slots;               // num_pages * page_size
    bool bf16_cache;
};
cudaError_t launch_append(const AppendArgs &a, cudaStream_t stream);

struct TagCheckArgs {
    const int32_t *block_table;
    const uint32_t *expected_tags;
    const int32_t *seq_lens;
    const uint32_t *page_tags;
    uint8_t *abort_flags;
    int32_t batch, max_pages_per_seq, page_size, num_pages;
};
cudaError_t launch_tag_check(const TagCheckArgs &a, cudaStream_t stream);

// Prefill -> decode handoff of whole pages (bf16 source, e4m3 destination).
struct HandoffArgs {
    const void *k_src, *v_src;              // bf16 caches [src_num_pages][Hkv][ps][D]
    const int32_t *src_pages;               // [num_listed]
    void *k_dst, *v_dst;                    // e4m3 caches [dst_num_pages][Hkv][ps][D]
    const int32_t *dst_pages;               // [num_listed]
    const float *k_scale, *v_scale;         // [Hkv] (quantise)
    float *k_scale_out, *v_scale_out;       // [Hkv] (amax -> scale)
    int32_t num_listed, num_kv_heads, page_size, src_num_pages, dst_num_pages;
};
cudaError_t launch_amax_scales(const HandoffArgs &a, cudaStream_t stream);
cudaError_t launch_quantize_pages(const HandoffArgs &a, cudaStream_t stream);

// Tag check of every request, then the append of token r for request r
// unless it was aborted (decode step: one new token per request).
cudaError_t launch_tag_check_append(const TagCheckArgs &t, const AppendArgs &a, cudaStream_t stream);

// The tag check of requests that hold only the pages a window shows.
struct TagWindowArgs {
    TagCheckArgs t;
    int32_t window, num_sinks, num_query_tokens;
};
cudaError_t launch_tag_check_window(const TagWindowArgs &a, cudaStream_t stream);

// Quantise-on-append into the block-scaled cache.
struct AppendBlocksArgs {
    const void *k_new, *v_new;       // bf16 [num_tokens][Hkv][D]
    const int32_t *token_offsets;    // [batch + 1], or null: num_tokens / batch tokens per request
    const int32_t *block_table;      // [batch][max_pages]
    const int32_t *seq_lens;         // [batch], the new tokens included
    const uint8_t *abort_flags;      // [batch] or null
    void *k_cache, *v_cache;         // e4m3 codes
    int8_t *k_exp, *v_exp;           // [num_pages][Hkv][page_size / 16]
    int32_t num_tokens, batch, max_pages_per_seq, num_kv_heads, page_size, num_pages;
};
cudaError_t launch_append_blocks(const AppendBlocksArgs &a, cudaStream_t stream);

// Pages copied inside every cache of a pool.  One launch takes kCopyMaxArrays
// arrays: num_caches of cache_page_bytes per page (a multiple of 2,048), then
// num_exps of exp_page_bytes.
constexpr int kCopyMaxArrays = 256;
struct CopyPagesArgs {
    void *arrays[kCopyMaxArrays];
    const int32_t *src_pages, *dst_pages;   // [num_listed]
    int64_t cache_page_bytes, exp_page_bytes;
    int32_t num_caches, num_exps, num_listed, num_pages;
};
cudaError_t launch_copy_pages(const CopyPagesArgs &a, cudaStream_t stream);

// Page tables kept on the GPU.
struct PoolArgs {
    int32_t *free_pages, *free_count;       // [num_pages], [1]
    int32_t *page_refs;                     // [num_pages]
    uint32_t *page_tags;                    // [num_pages] or null
    uint32_t *scratch;                      // arrival counter, a flag, from kPoolBitmapWord on a bit per page
    int32_t num_pages, page_size;
};
constexpr int kPoolBitmapWord = 64;
struct ExtendArgs {
    PoolArgs pool;
    const int32_t *token_offsets;           // [batch + 1], or null: tokens_each per request
    int32_t *seq_lens, *block_table;        // [batch], [batch][max_pages]
    uint32_t *expected_tags;                // [batch][max_pages] or null
    int64_t *slot_mapping;                  // [num_tokens] or null
    uint8_t *refused;                       // [batch]
    int32_t num_tokens, tokens_each, batch, max_pages_per_seq;
    int32_t per_cta, team;                  // set by the launch
};
cudaError_t launch_extend_tables(ExtendArgs a, cudaStream_t stream);
struct ForkArgs {
    PoolArgs pool;
    const int32_t *parents, *fork_lens;     // [batch]
    int32_t *seq_lens, *block_table;
    uint32_t *expected_tags;
    int32_t *src_pages, *dst_pages;         // [batch]
    uint8_t *refused;
    int32_t batch, max_pages_per_seq;
    int32_t per_cta;                        // set by the launch
};
cudaError_t launch_fork_tables(ForkArgs a, cudaStream_t stream);
struct TrimArgs {
    PoolArgs pool;
    const int32_t *keep_lens;               // [batch]
    int32_t *seq_lens, *block_table;
    int32_t batch, max_pages_per_seq;
};
cudaError_t launch_trim_tables(const TrimArgs &a, cudaStream_t stream);

// INT4 weight-only product y[m][n] = sum_k x[m][k] q[n][k] s[n][k / 128] for
// up to 16 rows of x per launch.  The weights are read through a 2-D tensor
// map over W viewed as [N rows][K / 2 bytes].
struct W4Args {
    const void *x;                   // bf16 [rows][k] (this launch's rows)
    const void *scales;              // bf16 [n][k / 128]
    void *y;                         // [rows][n], bf16 or fp32
    int32_t rows, n, k;              // rows <= 16; k % 256 == 0; n % 64 == 0
    int32_t splits, k_split;         // K is cut into `splits` ranges of k_split
    bool out_fp32;
};
constexpr int kW4Cols = 64;          // output columns per CTA
constexpr int kW4BlockK = 256;       // granularity of K and of its split ranges
constexpr int kW4CopyK = 128;        // k per tensor copy: 64 bytes of every column, one scale group
constexpr int kW4MaxSplits = 8;      // splits of K (one thread-block cluster)
cudaError_t launch_w4a16(const W4Args &a, const CUtensorMap &w_map, cudaStream_t stream);
// Resident CTAs of the INT4 kernel per SM, and resident clusters of `splits`.
int w4a16_ctas_per_sm();
int w4a16_cluster_capacity(int splits);
cudaError_t read_w4_error(uint32_t *bits, bool clear);

// Workspace layout (bytes from the workspace base):
//   [0, counter_bytes)       uint32 arrivals[B][Hkv][row_blocks]: splits of each
//                            (request, KV head, row block) that have published;
//                            zero before the first call, and every call leaves
//                            them zero.  A windowed or block-scaled call's
//                            counter_bytes holds ceil(n_query * g / 16) per
//                            (request, KV head) whichever kernel runs.
//   [counter_bytes, +lse)    fp32 lse (log2 domain, NaN = invalid split, -inf = a
//                            split that saw no token, +inf = one with a NaN):
//                            a grid of S splits [B][n_query][Hq][S]; a balanced
//                            launch [slots][8, or 16 with several query tokens]
//                            with a slot for each (CTA, pair) that can meet
//   [.., +o)                 fp32 o, each split's normalised output: the same
//                            places, D numbers each
//   [.., +pairs)             int2 (first slot, splits) of each pair: balanced
//                            launches that a second launch combines
struct DecodeArgs {
    const void *q;                   // bf16 [B][Hq][D]
    const float *k_scale, *v_scale;  // [Hkv] (unused for bf16 cache)
    const int32_t *block_table;      // [B][max_pages]
    const int32_t *seq_lens;         // [B]
    const uint8_t *abort_flags;      // [B] or null
    void *out;                       // [B][Hq][D]
    unsigned int *counters;
    float *ws_lse;
    float *ws_o;
    int32_t batch, num_q_heads, num_kv_heads, group, page_size, num_pages;
    int32_t max_pages_per_seq, split_tokens, max_splits;
    const void *k_new, *v_new;       // fused append: bf16 [B][Hkv][D] new token, else null
    void *k_cache, *v_cache;         // fused append: the caches the token is written to
    int32_t cluster;                 // 0: combine through memory; else the splits of a
                                     // (request, KV head) form one cluster of max_splits CTAs
    const uint32_t *expected_tags;   // in-launch tag check (kvq_decode_step): [B][max_pages],
    const uint32_t *page_tags;       // [num_pages] and the flags written, [B]; else null and
    uint8_t *abort_out;              // abort_flags (if any) is read instead
    int32_t n_query;                 // new query tokens per request (q, out: [B][n_query][Hq][D])
    int32_t row_blocks;              // CTAs per (split, request, KV head): ceil(n_query * g / 16), or 1
                                     // with one query token or in the tensor-memory kernels
    float qk_scale_log2;             // softmax_scale * log2(e)
    uint64_t copy_wait_ns;           // a consumer's limit on one copy wait (0: give up at once)
    bool out_fp32, bf16_cache;
};

// What the windowed and block-scaled builds take beside it.  Apart, so that the
// other builds' launches carry no more than they read (with it, 528 bytes of
// parameters instead of 472: a step of 512 tokens 12.9 us instead of 13.1,
// 8 x 8 x 8,193 tokens over bf16 53.9 instead of 54.4).
struct ViewArgs : DecodeArgs {
    int32_t window, num_sinks;       // last positions a query sees (0: all) and
                                     // first positions that stay visible
    int32_t resident_ctas;           // balanced launch: CTAs that share the batch's units evenly; 0:
                                     // a grid of splits of split_tokens
    int32_t balanced_ctas;           // its grid: resident_ctas times the most waves there can be
    int32_t unit_shift;              // log2 of a unit's tokens (a multiple of the page size)
    int32_t min_split_units;
    int32_t pair_cost;               // units' worth of time that a border between two pairs costs
    const int8_t *k_exp, *v_exp;     // block-scaled cache: [num_pages][Hkv][page_size / 16]
    int2 *ws_pairs;                  // balanced launch: each pair's first workspace slot and splits
    bool combine_apart;              // launch_combine_rows combines the splits
};

// What a call over shared prefixes takes beside it.
struct PrefixArgs : ViewArgs {
    const int32_t *prefix_of, *prefix_lens;  // [B]
    // partials of the shared pages (kvq_prefix.cu)
    float *pre_lse;                          // a place per (CTA, row)
    float4 *pre_o;                           // 32 of each place
    int4 *pre_rec;                           // [B][n][Hq]: place of the first part; the CTAs that have one, negative
                                             // if each has two; how far apart those are
    uint8_t *kinds;                          // [B]: kSharedPart, kOwnPart
    int32_t *own_takers;                     // CTAs of the own pages' kernel that have work; 0: not known yet
    int32_t pre_ctas;
};
constexpr int kSharedPart = 1, kOwnPart = 2;   // a request has parts of shared pages, of its own
constexpr int kPrefixRows = 256;     // most rows of a CTA's job over shared pages
// Over the shared pages (box heights of k_map and v_map: prefix_box_tokens),
// over the requests' own pages past them, and the parts of both joined.
cudaError_t launch_prefix_rows(const PrefixArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                               cudaStream_t stream);
cudaError_t launch_decode_own(const PrefixArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                              cudaStream_t stream);
cudaError_t launch_decode_own_blocks(const PrefixArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                                     cudaStream_t stream);
cudaError_t launch_combine_prefix(const PrefixArgs &a, cudaStream_t stream);
cudaError_t read_prefix_error(uint32_t *bits, bool clear);
cudaError_t read_own_error(uint32_t *bits, bool clear);
cudaError_t read_own_blocks_error(uint32_t *bits, bool clear);
// Tokens of a copy of the shared pages.  A bf16 cache is read through a map of
// [rows][128] values, 64 of a row at a time.
inline int prefix_box_tokens(int page_size, bool bf16_cache)
{
    const int most = bf16_cache ? 64 : kChunkTokens;
    return page_size < most ? page_size : most;
}

// Default limit of a wait on a bulk copy in the decode kernel: about one
// second.  The drain that follows a timeout always waits this long.
constexpr uint64_t kCopyWaitLimitNs = 1000000000ull;
// The limit decode launches use for a consumer's copy waits: the default
// unless the diagnostics entry point changed it.
uint64_t decode_copy_wait_ns();

// Split kernel, the combine fused into its epilogue but for combine_apart.  The
// tensor maps describe the K and V caches as 2-D [rows][128 bytes] tensors with
// 128-byte swizzle.
cudaError_t launch_decode(const DecodeArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                          cudaStream_t stream);
// The same kernel's builds with a window (any cache of launch_decode) and for
// the block-scaled cache (a window or none); the plan is made for the pages
// that visible_pages says a request can show.
cudaError_t launch_decode_window(const ViewArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                                 cudaStream_t stream);
cudaError_t launch_decode_blocks(const ViewArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                                 cudaStream_t stream);
// The combine as a launch of its own.
cudaError_t launch_combine_rows(const ViewArgs &a, cudaStream_t stream);
cudaError_t read_window_error(uint32_t *bits, bool clear);
cudaError_t read_blocks_error(uint32_t *bits, bool clear);
// The planner's queries for these builds (as decode_ctas_per_sm and
// decode_cluster_capacity below).
int decode_view_ctas_per_sm(bool bf16_cache, bool multi);
int decode_view_cluster_capacity(int n, bool bf16_cache, bool multi);
// Resident decode CTAs per SM for the cache type (occupancy of the kernel;
// multi: the multi-token build, 16 query rows per CTA).
int decode_ctas_per_sm(bool bf16_cache, bool multi = false);
// How many clusters of n split CTAs can be resident at once on the current
// device (0 if clusters of n cannot be used).
int decode_cluster_capacity(int n, bool bf16_cache, bool multi = false);
// Query rows one CTA of the multi-token build serves, and the most splits of
// one of its requests.
constexpr int kMultiRowsPerCta = 16;
constexpr int kMultiMaxSplitsPerRequest = 512;

// Multi-token decode over an FP8 cache on the 5th-generation tensor cores
// (tcgen05, accumulators and the A operands in tensor memory): one CTA per
// (split, KV head, request) takes all n_query * g <= 128 query rows; the
// splits merge through the workspace (never a cluster).  Split sizes are
// multiples of kUmmaTileTokens.
constexpr int kUmmaTileTokens = 64;
// Query rows per KV head (n_query * g) from which multi-token decode over an
// FP8 cache takes that kernel; fewer rows take the mma.sync build, which
// converts K and V per 16 rows but has no tensor-memory pipeline to fill.
constexpr int kUmmaMinRows = 64;
inline bool use_umma(bool bf16_cache, int n_query, int group)
{
    return !bf16_cache && n_query > 1 && n_query * group >= kUmmaMinRows;
}
cudaError_t launch_decode_umma(const DecodeArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                               cudaStream_t stream);
// Resident CTAs per SM of that kernel (bf16 output; at most 2: tensor memory).
int decode_umma_ctas_per_sm();
cudaError_t read_umma_error(uint32_t *bits, bool clear);
// Its builds with a window, and for the block-scaled cache (a.k_exp set).
cudaError_t launch_decode_umma_view(const ViewArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                                    cudaStream_t stream);
cudaError_t read_umma_view_error(uint32_t *bits, bool clear);
// Where a windowed or block-scaled multi-token call over an FP8 cache takes it.
// The mma.sync build converts every tile once per 16 rows and costs what its
// row blocks cost; up to 64 rows cost the tensor-memory kernel the same, but
// it has a pipeline to fill.  8 requests x 8 KV heads x 8,193 tokens, 32, 40,
// 64 and 128 rows: 50, 50, 52 and 58 us against 53, 75, 106 and 191.
// From 33 rows the cache bytes that the tables allow times rows decide: at
// 0.94e9 (8 x 8 x 2,000 tokens 40 rows, 4 x 8 x 2,000 64 rows) the two are even,
// at 0.2e9 to 0.6e9 it is 0 to 3 us behind, at 3e9 22 us against 42.  With 17
// to 32 rows, two row blocks, it gains later (1 x 8 x 30,000 tokens, 24 rows,
// 1.5e9: 26 us against 37) and only where the tables allow less cache than the
// mma.sync build shares out evenly (16 x 8 x 1,000..16,000 tokens: 102 with 40
// rows here, 94 with 32 there).
constexpr int kUmmaViewMinRows = 17, kUmmaViewManyRows = 33;
constexpr double kUmmaViewMinWork = 0.9e9, kUmmaViewMinWorkFew = 1.4e9;
// (bytes from which the planner shares a call out evenly)
constexpr int64_t kBalancedMinBytes = 256 << 20;
inline bool use_umma_view(bool bf16_cache, int n_query, int group, int64_t batch, int64_t num_kv_heads,
                          int64_t max_tokens)
{
    const int64_t rows = static_cast<int64_t>(n_query) * group;
    if (bf16_cache || n_query == 1 || rows < kUmmaViewMinRows)
        return false;
    const double bytes = 256.0 * static_cast<double>(batch * num_kv_heads) * static_cast<double>(max_tokens);
    if (rows >= kUmmaViewManyRows)
        return bytes * static_cast<double>(rows) >= kUmmaViewMinWork;
    return bytes * static_cast<double>(rows) >= kUmmaViewMinWorkFew && bytes < static_cast<double>(kBalancedMinBytes);
}

// Box height (in 128-byte rows) of one bulk copy for a page size.
inline int tma_box_rows(int page_size, bool bf16_cache)
{
    int tok = page_size < kChunkTokens ? page_size : kChunkTokens;
    return bf16_cache ? 2 * tok : tok;
}

cudaError_t read_device_error(uint32_t *bits, bool clear);

#ifdef KVQ_PHASE_STAMPS
// Instrumented build only: the %globaltimer stamps of the last decode launch
// ([CTA][8] points) and of the last tag-check + append launch ([CTA][2]).
cudaError_t read_decode_stamps(unsigned long long *host, size_t count);
cudaError_t read_check_stamps(unsigned long long *host, size_t count);
cudaError_t read_tag_stamps(unsigned long long *host, size_t count);   // tag check alone, [CTA][2]
#endif

// SMs of the current device, queried once per device.  A host with no usable
// device (the planner's host-only queries) plans for a 152-SM GB300.
int device_sm_count();

} // namespace kvq
