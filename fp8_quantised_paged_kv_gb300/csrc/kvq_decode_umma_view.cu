// kvq_decode_umma_view.cu -- attention of many query rows on the 5th-generation
// tensor cores, with a window and sinks or over the block-scaled cache.
//
// The mathematics, the tiles of 64 tokens and the layouts are those of
// kvq_decode_umma.cu, and the window and the exponents mean what they mean in
// kvq_decode_split.cuh: a shortened context without the pages that no query
// sees, ek on the scores, ev in the softmax's exponent with 2^-ev undone in
// the sum.  A tile has four blocks of 16, the columns of one tensor-memory
// load.  P is kept 2^7 times larger (2^15 at most with the stale maximum's
// 2^8), so f16 cuts weights at 2^-32 of the largest.
//
// The jobs are kvq_decode_umma.cu's as well, but where one of them set the pace:
//   - with bf16 output two softmax groups of four warps take the even and the
//     odd tiles, each with a maximum, a sum and an accumulator of its own, so
//     that one group's exponentials run while the other waits for its scores
//     or for tensor memory.  The groups' results merge at the end as the
//     copies of a row do.  Two threads per row on every tile were slower: what
//     a tile costs whatever its size was paid twice.  With fp32 output P has
//     a second f16 term, whose columns take the place of the second
//     accumulator: one group;
//   - two warps issue S = Q K^T, of the even and the odd tiles;
//   - the converters look at V rows to zero only in the tiles that have some.
//     Eight converting warps, K and V apart, were slower (fewer registers for
//     the softmax, more warps on the same shared memory);
//   - the query rows are on their way while the exponents are read;
//   - the splits are combined by a launch of its own.
// 2 x 8 x 30,000 tokens, 128 rows: 49 us in nine splits (80 with the jobs
// as there, 60 before the combine of its own); 8 x 60,000, 64 rows: 42 (58).
// What bounds it: a tile takes 0.6 us an SM (64 rows) to 0.65, converters and
// softmax each at work for three quarters of it; the copies alone take 0.36.
#include "kvq_decode_umma.cuh"
#include "kvq_view.cuh"

namespace kvq {
namespace {

// The jobs of a build's warps.
template <bool kPrecise>
struct Jobs {
    static constexpr int kGroups = kPrecise ? 1 : 2;       // softmax groups: four warps, one per lane quarter
    static constexpr int kConv = 4 * kGroups;              // first of four converting warps
    static constexpr int kCopy = kConv + 4;                // copies of K's and V's rows
    static constexpr int kIssueS = kCopy + 1;              // two warps: even and odd tiles
    static constexpr int kIssueO = kIssueS + 2;
    static constexpr int kThreads = 32 * (kIssueO + 1);
    static constexpr int kOperands = kPrecise ? 2 : 4;     // operand buffers in flight
    static constexpr int kSoftThreads = 128 * kGroups;
};

// Shared memory: the rings of K and V rows as e4m3, the operand buffers (K as
// f16, [64 tokens][64 dims] twice, V alike), barriers and tables.
constexpr int kStageBytes = 2 * kTile * 128;               // K then V rows of one tile
constexpr int kOffOps = kStages * kStageBytes;
constexpr int kViewData = kOffOps + 4 * kKVBytes;
// With fp32 output O goes out of tensor memory every kFlushTiles tiles into
// fp32 sums that round, kept where two of the operand buffers would be (128
// rows x 512 bytes, 16-byte chunks xor-swizzled by the row): the tensor core
// cuts what it adds to a large accumulator, always towards zero, which came to
// 1.4e-6 of the output over 78 tiles (8.7e-7 so, 128 rows; 7.2e-7 and 5.0e-7
// with 64).
constexpr int kFlushTiles = 16;
constexpr int kOffSums = kOffOps + 2 * kKVBytes;
static_assert(kOffSums + 128 * kHeadDim * 4 <= kViewData, "the sums fit in two operand buffers");
static_assert(2 * 128 * (kMergeStride + 3) * 4 <= kViewData, "the merge buffer fits in the idle ring and buffers");
constexpr int kMaxBars = 2 * kStages + 2 * 4 + 3 * 2 + 1 + 3;   // see the barrier map in the kernel

constexpr int view_smem_bytes()
{
    return 1024 /* alignment slack */ + kViewData + kMaxBars * 8 + 16 /* tmem slot */ + kMaxPageList * 4 +
           2 * (8192 / kBlockTokens) /* exponents of the split's blocks */;
}
static_assert(view_smem_bytes() <= 232448, "one CTA fits an SM");

// Tensor-memory columns (lane m = row slot m): Q as f16 pairs, two score
// buffers, an accumulator per group, and two P buffers as f16 pairs.  With
// fp32 output the second accumulator's columns hold the P buffers' low parts.
constexpr uint32_t kTcQ = 0, kTcS = 64, kTcO = 192, kTcPlo = 320, kTcP = 448;
constexpr float kLift = 7.f;                               // log2 of what P, the sum and O are larger by

// kTpc: tokens of a tile each copy of the rows takes: 32 for up to 64 rows
// (two copies fill the 128 M slots), 64 for 65 .. 128 rows (one copy).
template <bool kPrecise, int kTpc, bool kBlocks>
__global__ void __launch_bounds__(Jobs<kPrecise>::kThreads, 1)
decode_rows_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                   const ViewArgs a)
{
    using J = Jobs<kPrecise>;
    constexpr int kThreads = J::kThreads, kKV = J::kOperands, kGroups = J::kGroups;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    // barriers: copy landed, stage free (per ring stage); operands
    // converted, operands read (per operand buffer); scores ready, scores read, P
    // written (per score / P buffer); Q staged; the issuing lanes' final drains
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + kViewData);
    uint64_t *landed = bars, *empty = landed + kStages;
    uint64_t *conv = empty + kStages, *pv_done = conv + kKV;
    uint64_t *s_full = pv_done + kKV, *s_free = s_full + 2, *p_full = s_free + 2;
    uint64_t *q_ready = p_full + 2, *drain = q_ready + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kMaxBars);
    int32_t *page_list = reinterpret_cast<int32_t *>(tmem_slot + 4);
    [[maybe_unused]] uint16_t *blk_exp = reinterpret_cast<uint16_t *>(page_list + kMaxPageList);
    __shared__ int s_abort;
    __shared__ int s_qexp[128];                            // the rows' q_row_exponent
    __shared__ int s_landed;                               // tiles whose copies a converter saw land

    const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = a.group, R = a.n_query * g, ps = a.page_size;
    const int ps_shift = __ffs(ps) - 1;                    // ps is 16, 32, 64 or 128
    constexpr int Rp = 2 * kTpc;                           // M slots per copy of the rows
    const int first_page = static_cast<int>(static_cast<int64_t>(split) * a.split_tokens / ps);
    const int span_left = a.max_pages_per_seq - first_page;
    const int span = a.split_tokens / ps < span_left ? a.split_tokens / ps : span_left;
    const int32_t *bt = a.block_table + static_cast<int64_t>(b) * a.max_pages_per_seq + first_page;

    // Launched as a programmatic dependent of the previous kernel on the
    // stream: nothing is read from global memory before the wait returns.
    if (tid == 0) {
        prefetch_tensor_map(&k_map);
        prefetch_tensor_map(&v_map);
    }
    grid_dependency_wait();

    constexpr int kIdsPerThread = (kMaxPageList + kThreads - 1) / kThreads;
    int32_t ids[kIdsPerThread];
    if (a.window == 0) {
#pragma unroll
        for (int k = 0; k < kIdsPerThread; ++k) {
            const int i = tid + k * kThreads;
            ids[k] = i < span ? __ldg(bt + i) : -1;
        }
    }
    const int64_t real_len = a.seq_lens[b];
    const bool aborted_req = a.abort_flags != nullptr && a.abort_flags[b] != 0;
    const int64_t cap = static_cast<int64_t>(a.max_pages_per_seq) * ps;
    const bool zero_request = aborted_req || real_len <= 0 || real_len > cap;
    // Window: from here on `len` and every position count the shortened
    // context (shown_context).
    int64_t len = real_len;
    int64_t win0 = 0;                                      // where the first query's window starts
    if (a.window > 0) {
        const Shown shown = shown_context(a, real_len, ps_shift);
        len = shown.len;
        win0 = shown.win0;
        // only entries of pages with a token of the shortened context are read
#pragma unroll
        for (int k = 0; k < kIdsPerThread; ++k) {
            const int i = tid + k * kThreads;
            const int64_t v = static_cast<int64_t>(first_page) + i;
            const bool held = !zero_request && i < a.split_tokens / ps && (v << ps_shift) < len;
            ids[k] = held ? __ldg(bt + i + (v < shown.sink_pages ? 0 : shown.hole)) : -1;
        }
    }
    const int nsplit = zero_request ? 1 : static_cast<int>((len + a.split_tokens - 1) / a.split_tokens);
    if (split >= nsplit)
        return;
    if (zero_request) {                                    // split 0 writes the zeros
        for (int i = tid; i < R * kHeadDim; i += kThreads)
            store_row_value(a.out, row_id(a, b, kvh, i / kHeadDim) * kHeadDim + i % kHeadDim, 0.f, a.out_fp32);
        return;
    }

    const int64_t t0 = static_cast<int64_t>(split) * a.split_tokens;
    const int64_t t1 = min(len, t0 + a.split_tokens);
    const int n_pages = static_cast<int>((t1 - 1) / ps) - first_page + 1;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kIdsPerThread; ++k) {
        const int i = tid + k * kThreads;
        if (i < n_pages) {
            bad |= (ids[k] < 0 || ids[k] >= a.num_pages);
            page_list[i] = ids[k];
        }
    }
    if (tid == 0) {
        s_abort = 0;
        s_landed = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&landed[i], 1);
            mbar_init(&empty[i], 4);
        }
        for (int i = 0; i < kKV; ++i) {
            mbar_init(&conv[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], 4);
            mbar_init(&p_full[i], 4);
        }
        mbar_init(q_ready, 4);
        for (int i = 0; i < 3; ++i)
            mbar_init(&drain[i], 1);
        fence_mbar_init();
    }
    bad = __syncthreads_or(bad);

    auto publish_invalid = [&]() {                         // the request's rows get zeros
        if (nsplit == 1) {
            for (int i = tid; i < R * kHeadDim; i += kThreads)
                store_row_value(a.out, row_id(a, b, kvh, i / kHeadDim) * kHeadDim + i % kHeadDim, 0.f,
                                a.out_fp32);
        } else if (tid < R) {
            a.ws_lse[row_id(a, b, kvh, tid) * a.max_splits + split] = __uint_as_float(0x7FC00000u);
        }
    };

    const int n_tiles = static_cast<int>((t1 - t0 + kTile - 1) / kTile);
    volatile int *abort_flag = &s_abort;
    // softmax thread (group gr, slot m): copy m / Rp of local row m % Rp
    const int gr = tid >> 7, m = tid & 127;
    const int copy = m / Rp, r = m % Rp;
    const bool row_valid = tid < J::kSoftThreads && r < R;
    float m_used = -INFINITY, l_sum = 0.f;
    // kPrecise: this thread's row of the sums, and what they are behind m_used by
    [[maybe_unused]] float4 *sums = reinterpret_cast<float4 *>(sm + kOffSums) + m * (kHeadDim / 4);
    [[maybe_unused]] float sums_mul = 1.f;
    int issued = 0;                                        // copying warp's lane 0: tiles whose copies it issued

    if (bad) {
        publish_invalid();
    } else {
        // the row's bf16 pairs, on their way while the exponents are read
        uint32_t qw[kHeadDim / 2];
        if (row_valid && gr == 0) {
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) +
                                                               row_id(a, b, kvh, r) * kHeadDim);
#pragma unroll
            for (int i = 0; i < kHeadDim / 8; ++i) {
                const uint4 v = __ldg(src + i);
                qw[4 * i] = v.x; qw[4 * i + 1] = v.y; qw[4 * i + 2] = v.z; qw[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kHeadDim / 2; ++i)
                qw[i] = 0u;
        }
        if (warp == 0)
            tmem_alloc(tmem_slot, kTmemCols);
        if constexpr (kBlocks) {
            // the exponents of the split's blocks (ek in the low byte, ev in
            // the high one); a block past the split's end has none
            const int bpp_shift = ps_shift - 4;            // blocks per page: ps / 16
            for (int i = tid; i < n_tiles * (kTile / kBlockTokens); i += kThreads) {
                uint16_t e = 0;
                if (t0 + static_cast<int64_t>(i) * kBlockTokens < t1) {
                    const int64_t at =
                        ((static_cast<int64_t>(page_list[i >> bpp_shift]) * a.num_kv_heads + kvh) << bpp_shift) +
                        (i & ((1 << bpp_shift) - 1));
                    const int ek = max(static_cast<int>(__ldcg(a.k_exp + at)), kReadKeyExpMin);
                    const int ev = max(static_cast<int>(__ldcg(a.v_exp + at)), kReadValueExpMin);
                    e = static_cast<uint16_t>((ek & 0xFF) | (min(ev, kReadValueExpMax) << 8));
                }
                blk_exp[i] = e;
            }
        }
        tmem_fence_before_sync();
        __syncthreads();
        tmem_fence_after_sync();
        const uint32_t tmem = *tmem_slot;

        if (warp == J::kCopy) {
            // ------------------------------------------------ copies of K's and V's rows
            const int box_tok = ps < kChunkTokens ? ps : kChunkTokens;
            const int parts = kTile / box_tok;             // 2 or 4 copies per tensor
            const uint64_t policy = l2_policy_evict_first();
            for (int j = 0; j < n_tiles; ++j) {
                const int st = j % kStages;
                if (j >= kStages && !__all_sync(0xFFFFFFFFu, wait_or_abort(&empty[st], ((j / kStages) - 1) & 1,
                                                                           kCopyWaitLimitNs, abort_flag, 4u)))
                    break;
                const int64_t tok = t0 + static_cast<int64_t>(j) * kTile;
                const int64_t left = t1 - tok;
                const int np = static_cast<int>(left >= kTile ? parts : (left + box_tok - 1) / box_tok);
                if (lane == 0)
                    mbar_arrive_expect_tx(&landed[st], static_cast<uint32_t>(2 * np * box_tok * 128));
                __syncwarp();
                if (lane < 2 * np) {                       // lanes 0 .. np - 1: K parts, np .. 2 np - 1: V parts
                    const bool is_v = lane >= np;
                    const int part = is_v ? lane - np : lane;
                    const int64_t ptok = tok + part * box_tok;
                    const int32_t page = page_list[static_cast<int>(ptok >> ps_shift) - first_page];
                    const int32_t y = static_cast<int32_t>((static_cast<int64_t>(page) * a.num_kv_heads + kvh) * ps +
                                                           (ptok & (ps - 1)));
                    tma_load_2d(sm + st * kStageBytes + (is_v ? kTile * 128 : 0) + part * box_tok * 128,
                                is_v ? static_cast<const void *>(&v_map) : static_cast<const void *>(&k_map), 0, y,
                                &landed[st], policy);
                }
                issued = j + 1;
            }
        } else if (warp >= J::kConv && warp < J::kCopy) {
            // ------------------------------------------------ e4m3 -> f16 (exact)
            const int ct = tid - 32 * J::kConv;            // 0 .. 127
            const int c = ct & 7;                          // 16-byte chunk (16 dims) of an e4m3 row
            // this thread's chunk of row t goes to an operand's chunks 2 c, 2 c + 1
            auto convert = [&](uint8_t *to, const uint4 (&x)[4]) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int t = (ct >> 3) + 16 * k;
                    const uint32_t base = static_cast<uint32_t>((c >> 2) * 8192);
                    const uint32_t o0 = base + sw128_chunk(t, 2 * (c & 3));
                    const uint32_t o1 = base + sw128_chunk(t, 2 * (c & 3) + 1);
                    // the two slices share banks: lanes with c >= 4 store their
                    // two 16-byte chunks in the other order, so a store's 8
                    // lanes hit 8 bank groups (the words are picked before
                    // they are converted)
                    const bool swap = c >= 4;
                    const uint32_t a0 = swap ? x[k].z : x[k].x, a1 = swap ? x[k].w : x[k].y;
                    const uint32_t b0 = swap ? x[k].x : x[k].z, b1 = swap ? x[k].y : x[k].w;
                    *reinterpret_cast<uint4 *>(to + (swap ? o1 : o0)) =
                        make_uint4(lo16_e4m3x2_to_f16x2(a0), hi16_e4m3x2_to_f16x2(a0),
                                   lo16_e4m3x2_to_f16x2(a1), hi16_e4m3x2_to_f16x2(a1));
                    *reinterpret_cast<uint4 *>(to + (swap ? o0 : o1)) =
                        make_uint4(lo16_e4m3x2_to_f16x2(b0), hi16_e4m3x2_to_f16x2(b0),
                                   lo16_e4m3x2_to_f16x2(b1), hi16_e4m3x2_to_f16x2(b1));
                }
            };
            // tiles [hide0, hide1) and the last hold V rows to zero: past the
            // split, or seen by no query
            const int hide0 = static_cast<int>(max(min(a.num_sinks - t0, static_cast<int64_t>(kTile) * n_tiles),
                                                   static_cast<int64_t>(0)) / kTile);
            const int hide1 = static_cast<int>((max(min(win0 - t0, static_cast<int64_t>(kTile) * n_tiles),
                                                    static_cast<int64_t>(0)) + kTile - 1) / kTile);
            int st = 0, landed_par = 0, seen = 0;
            for (int j = 0; j < n_tiles; ++j) {
                const int kb = j % kKV;
                // every lane polls; the warp goes on or gives up as one
                if (!__all_sync(0xFFFFFFFFu, wait_or_abort(&landed[st], landed_par, a.copy_wait_ns, abort_flag, 1u)))
                    break;
                seen = j + 1;
                // operand buffer kb is free once O += P V of tile j - kKV is done
                if (j >= kKV && !__all_sync(0xFFFFFFFFu, wait_or_abort(&pv_done[kb], ((j - kKV) / kKV) & 1,
                                                                       kCopyWaitLimitNs, abort_flag, 4u)))
                    break;
                const uint8_t *from = sm + st * kStageBytes;
                uint8_t *to = sm + kOffOps + kb * kKVBytes;
                uint4 xk[4], xv[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {              // every load of the tile first
                    const int t = (ct >> 3) + 16 * k;
                    const uint32_t src = static_cast<uint32_t>(t * 128 + ((c ^ (t & 7)) << 4));
                    xk[k] = *reinterpret_cast<const uint4 *>(from + src);
                    xv[k] = *reinterpret_cast<const uint4 *>(from + kTile * 128 + src);
                }
                if (j == n_tiles - 1 || (j >= hide0 && j < hide1)) {
                    const int64_t tok0 = t0 + static_cast<int64_t>(j) * kTile;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int64_t at = tok0 + (ct >> 3) + 16 * k;
                        if (at >= t1 || (at >= a.num_sinks && at < win0))
                            xv[k] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                convert(to, xk);
                convert(to + kKVBytes / 2, xv);
                fence_proxy_async_smem();                  // the writes, for the tensor core;
                __syncwarp();                              // the ring reads, for the next copy
                if (lane == 0) {
                    mbar_arrive(&conv[kb]);
                    mbar_arrive(&empty[st]);
                }
                if (++st == kStages) {
                    st = 0;
                    landed_par ^= 1;
                }
            }
            if (lane == 0)
                atomicMax(&s_landed, seen);
        } else if (warp == J::kIssueS || warp == J::kIssueS + 1) {
            // ------------------------------------------------ S = Q K^T of the even or odd tiles
            // A tcgen05.mma holds its issuing thread for 100 to 125 cycles at
            // these shapes; several issuing warps complete as many times more.
            if (lane == 0) {
                // descriptor of the first operand buffer's K; a k step or
                // another buffer adds its byte offset / 16 to the start field
                const uint64_t dk = umma_desc(smem_addr(sm + kOffOps), 0, 1024);
                const int sb = warp - J::kIssueS;
                bool ok = wait_or_abort(q_ready, 0, kCopyWaitLimitNs, abort_flag, 4u);
                for (int js = sb; ok && js < n_tiles; js += 2) {
                    // the score buffer is free once the softmax has read the
                    // scores of tile js - 2
                    if (js >= 2 && !wait_or_abort(&s_free[sb], ((js - 2) >> 1) & 1, kCopyWaitLimitNs, abort_flag, 4u))
                        break;
                    if (!wait_or_abort(&conv[js % kKV], (js / kKV) & 1, kCopyWaitLimitNs, abort_flag, 4u))
                        break;
                    tmem_fence_after_sync();
                    const uint64_t dkb = dk + static_cast<uint64_t>(((js % kKV) * kKVBytes) >> 4);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)         // Q: 8 columns (16 dims) per k step
                        umma_f16_ts(tmem + kTcS + 64u * sb, tmem + kTcQ + 8u * kk,
                                    dkb + static_cast<uint64_t>(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), kIdescS,
                                    kk > 0);
                    umma_commit(&s_full[sb]);
                }
                // nothing this lane issued may still run when the CTA moves on
                umma_commit(&drain[sb]);
                if (!mbar_wait_bounded(&drain[sb], 0, kCopyWaitLimitNs))
                    atomicOr(&g_umma_error, 4u);
            }
            __syncwarp();
        } else if (warp == J::kIssueO) {
            // ------------------------------------------------ O += P V, into the group's accumulator
            if (lane == 0) {
                const uint64_t dv = umma_desc(smem_addr(sm + kOffOps + kKVBytes / 2), 8192, 1024);
                for (int jp = 0; jp < n_tiles; ++jp) {
                    // P of tile jp written (so its scores, hence its K and V
                    // operands, are complete too)
                    const int pb = jp & 1, kb = jp % kKV;
                    if (!wait_or_abort(&p_full[pb], (jp >> 1) & 1, kCopyWaitLimitNs, abort_flag, 4u))
                        break;
                    tmem_fence_after_sync();
                    const uint64_t dvb = dv + static_cast<uint64_t>((kb * kKVBytes) >> 4);
                    const uint32_t o = tmem + kTcO + 128u * (jp % kGroups);
                    const bool onto = kPrecise ? jp % kFlushTiles != 0 : jp >= kGroups;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)         // P: 8 columns (16 tokens) per k step
                        umma_f16_ts(o, tmem + kTcP + 32u * pb + 8u * kk, dvb + static_cast<uint64_t>(kk * 128),
                                    kIdescPV, onto || kk > 0);
                    if constexpr (kPrecise) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_f16_ts(o, tmem + kTcPlo + 32u * pb + 8u * kk,
                                        dvb + static_cast<uint64_t>(kk * 128), kIdescPV, true);
                    }
                    umma_commit(&pv_done[kb]);
                }
                umma_commit(&drain[2]);
                if (!mbar_wait_bounded(&drain[2], 0, kCopyWaitLimitNs))
                    atomicOr(&g_umma_error, 4u);
            }
            __syncwarp();
        } else {
            // ------------------------------------------------ softmax
            const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
            float mul;                                     // score multiplier (log2 domain)
            // Positions below lim are visible.  A slot without a row sees them all:
            // its results go nowhere, and its warp needs no masks for it (8 x 8 x
            // 8,193 tokens, 24 and 40 rows: 53.5 and 53.4 us with them,
            // 49.5 and 50.3 without).
            int64_t lim = t1;
            {
                int e;
                if (gr == 0) {
                    uint32_t mx = 0;
#pragma unroll
                    for (int i = 0; i < kHeadDim / 2; ++i)
                        mx = max(mx, max(qw[i] & 0x7FFFu, (qw[i] >> 16) & 0x7FFFu));
                    e = q_row_exponent(mx);
                    s_qexp[m] = e;
                    // row m of Q as f16 pairs (dims 2c, 2c + 1 in column c)
                    const float q_mul = __int_as_float((127 + e) << 23);
#pragma unroll
                    for (int c0 = 0; c0 < kHeadDim / 2; c0 += 16) {
                        uint32_t h[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 f = bf16x2_to_f32x2(qw[c0 + i]);
                            h[i] = f32x2_to_f16x2(f.x * q_mul, f.y * q_mul);
                        }
                        tmem_st16(tmem + lane_base + kTcQ + c0, h);
                    }
                    tmem_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(q_ready);
                } else {
                    // a wait that gives up raises the abort flag, which ends
                    // this warp's first wait for scores
                    wait_or_abort(q_ready, 0, kCopyWaitLimitNs, abort_flag, 4u);
                    __syncwarp();
                    e = s_qexp[m];
                }
                mul = a.qk_scale_log2 * (kBlocks ? 1.f : a.k_scale[kvh]) * __int_as_float((127 - e) << 23);
                if (row_valid) {
                    const int64_t vis = len - a.n_query + 1 + r / g;
                    lim = vis < t1 ? vis : t1;
                }
            }
            // window: this row sees no position of [num_sinks, win)
            const int64_t win = a.window > 0 && row_valid ? win0 + r / g : 0;
            const int my0 = copy * kTpc;                   // this thread's tokens in a tile (its warp's)
            // Row m of a P buffer is one thread's alone: its columns outside the
            // copy's tokens are zeroed once here and never written again.
            if constexpr (kTpc < kTile) {
                uint32_t zero[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    zero[i] = 0u;
#pragma unroll
                for (int c0 = 0; c0 < 64 / kGroups; c0 += 16) {
                    tmem_st16(tmem + lane_base + kTcP + 32u * gr + c0, zero);
                    if constexpr (kPrecise)
                        tmem_st16(tmem + lane_base + kTcPlo + c0, zero);
                }
            }
            const uint32_t ocol = tmem + lane_base + kTcO + 128u * gr;
            for (int j = gr; j < n_tiles; j += kGroups) {
                const int sb = j & 1;                      // score and P buffer
                if (!__all_sync(0xFFFFFFFFu,
                                wait_or_abort(&s_full[sb], (j >> 1) & 1, kCopyWaitLimitNs, abort_flag, 4u)))
                    break;
                tmem_fence_after_sync();
                // this row's visible tokens of the tile: [my0, hi)
                const int64_t vl = lim - (t0 + static_cast<int64_t>(j) * kTile);
                const int hi = vl <= my0 ? my0 : (vl >= my0 + kTpc ? my0 + kTpc : static_cast<int>(vl));
                const uint32_t scol = tmem + lane_base + kTcS + 64u * sb + static_cast<uint32_t>(my0);
                float p[kTpc];
                uint64_t mul2 = f2_pack(mul, mul);
                // masked columns of the window: [hole_lo, hole_hi)
                const int64_t at0 = t0 + static_cast<int64_t>(j) * kTile;
                const int hole_lo = static_cast<int>(min(max(a.num_sinks - at0, static_cast<int64_t>(0)),
                                                         static_cast<int64_t>(kTile)));
                const int hole_hi = static_cast<int>(min(max(win - at0, static_cast<int64_t>(0)),
                                                         static_cast<int64_t>(kTile)));
                const bool no_hole = hole_hi <= max(hole_lo, my0) || hole_lo >= my0 + kTpc;
                // block q of this copy's columns: ek into mul2, ev into ev2
                [[maybe_unused]] uint64_t ev2 = 0;
                auto block = [&](int q) {
                    if constexpr (kBlocks) {
                        const int e = static_cast<int16_t>(blk_exp[4 * j + my0 / kBlockTokens + q]);
                        const float mk = mul * __int_as_float((127 + static_cast<int8_t>(e & 0xFF)) << 23);
                        const float ev = static_cast<float>(e >> 8);
                        mul2 = f2_pack(mk, mk);
                        ev2 = f2_pack(ev, ev);
                    }
                };
                auto scaled = [&](uint32_t s0, uint32_t s1, float &x0, float &x1) {
                    const uint64_t s = f2_pack(__uint_as_float(s0), __uint_as_float(s1));
                    if constexpr (kBlocks)
                        f2_unpack(f2_fma(s, mul2, ev2), x0, x1);
                    else
                        f2_unpack(f2_mul(s, mul2), x0, x1);
                };
                if (__all_sync(0xFFFFFFFFu, hi == my0 + kTpc && no_hole)) {   // every column visible: no masks
#pragma unroll
                    for (int q = 0; q < kTpc / 16; ++q) {
                        uint32_t sv[16];
                        tmem_ld16(scol + 16u * q, sv);
                        block(q);
#pragma unroll
                        for (int i = 0; i < 16; i += 2)
                            scaled(sv[i], sv[i + 1], p[16 * q + i], p[16 * q + i + 1]);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < kTpc / 16; ++q) {
                        uint32_t sv[16];
                        tmem_ld16(scol + 16u * q, sv);
                        block(q);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float x0, x1;
                            scaled(sv[i], sv[i + 1], x0, x1);
                            const int c = my0 + 16 * q + i;
                            const bool keep0 = c < hi && !(c >= hole_lo && c < hole_hi);
                            const bool keep1 = c + 1 < hi && !(c + 1 >= hole_lo && c + 1 < hole_hi);
                            p[16 * q + i] = keep0 ? x0 : -INFINITY;
                            p[16 * q + i + 1] = keep1 ? x1 : -INFINITY;
                        }
                    }
                }
                // the scores are in registers: the buffer can take tile j + 2
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&s_free[sb]);
                float mxa[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < kTpc; ++i)
                    mxa[i & 3] = fmaxf(mxa[i & 3], p[i]);
                const float mx = fmaxf(fmaxf(mxa[0], mxa[1]), fmaxf(mxa[2], mxa[3]));
                const bool raise = row_valid && mx > m_used + kRaiseThreshold;   // raise the running maximum
                const float alpha = raise ? (m_used == -INFINITY ? 0.f : fast_exp2(m_used - mx)) : 1.f;
                // O holds earlier tiles of row m: rescale it once O += P V of
                // the group's last tile is done (warp-wide loads and stores: the other
                // lanes multiply by 1)
                const bool flush = kPrecise && j > 0 && j % kFlushTiles == 0;
                const bool rescale = raise && m_used != -INFINITY && j >= kGroups && !flush;
                if constexpr (kPrecise) {
                    if (flush) {                           // O += P V starts from zero with this tile
                        if (!__all_sync(0xFFFFFFFFu, wait_or_abort(&pv_done[(j - 1) % kKV], ((j - 1) / kKV) & 1,
                                                                   kCopyWaitLimitNs, abort_flag, 4u)))
                            break;
                        tmem_fence_after_sync();
#pragma unroll 1
                        for (int cc = 0; cc < 8; ++cc) {
                            uint32_t o[16];
                            tmem_ld16(ocol + 16 * cc, o);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float4 &at = sums[(4 * cc + i) ^ (m & 7)];
                                float4 v = j == kFlushTiles ? make_float4(0.f, 0.f, 0.f, 0.f) : at;
                                v.x = fmaf(v.x, sums_mul, __uint_as_float(o[4 * i]));
                                v.y = fmaf(v.y, sums_mul, __uint_as_float(o[4 * i + 1]));
                                v.z = fmaf(v.z, sums_mul, __uint_as_float(o[4 * i + 2]));
                                v.w = fmaf(v.w, sums_mul, __uint_as_float(o[4 * i + 3]));
                                at = v;
                            }
                        }
                        sums_mul = 1.f;
                    }
                    if (raise)
                        sums_mul *= alpha;
                }
                if (__any_sync(0xFFFFFFFFu, rescale)) {
                    if (!__all_sync(0xFFFFFFFFu, wait_or_abort(&pv_done[(j - kGroups) % kKV],
                                                               ((j - kGroups) / kKV) & 1, kCopyWaitLimitNs, abort_flag, 4u)))
                        break;
                    tmem_fence_after_sync();
                    const float f = rescale ? alpha : 1.f;
#pragma unroll 1
                    for (int cc = 0; cc < 8; ++cc) {
                        uint32_t o[16];
                        const uint32_t addr = ocol + 16 * cc;
                        tmem_ld16(addr, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st16(addr, o);
                    }
                }
                if (raise) {
                    l_sum *= alpha;
                    m_used = mx;
                }
                const float base = (m_used == -INFINITY ? 0.f : m_used) - kLift;
                const uint64_t nb2 = f2_pack(-base, -base);
                [[maybe_unused]] float block_sum = 0.f;
                uint64_t sa2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
                for (int i = 0; i < kTpc; i += 2) {
                    float x0, x1;
                    f2_unpack(f2_add(f2_pack(p[i], p[i + 1]), nb2), x0, x1);
                    p[i] = fast_exp2(x0);
                    p[i + 1] = fast_exp2(x1);
                    sa2[(i >> 1) & 1] = f2_add(sa2[(i >> 1) & 1], f2_pack(p[i], p[i + 1]));
                    if (kBlocks && (i + 2) % kBlockTokens == 0) {          // a block's weights, times 2^-ev
                        const int e = static_cast<int16_t>(blk_exp[4 * j + (my0 + i) / kBlockTokens]) >> 8;
                        float s0, s1, s2, s3;
                        f2_unpack(sa2[0], s0, s1);
                        f2_unpack(sa2[1], s2, s3);
                        block_sum = fmaf((s0 + s1) + (s2 + s3), __int_as_float((127 - e) << 23), block_sum);
                        sa2[0] = sa2[1] = f2_pack(0.f, 0.f);
                    }
                }
                if constexpr (kBlocks) {
                    l_sum += block_sum;
                } else {
                    float s0, s1, s2, s3;
                    f2_unpack(sa2[0], s0, s1);
                    f2_unpack(sa2[1], s2, s3);
                    l_sum += (s0 + s1) + (s2 + s3);
                }
                // P buffer sb is free once O += P V of tile j - 2 is done
                if (j >= 2 && !__all_sync(0xFFFFFFFFu, wait_or_abort(&pv_done[(j - 2) % kKV], ((j - 2) / kKV) & 1,
                                                                     kCopyWaitLimitNs, abort_flag, 4u)))
                    break;
                // row m of P over the copy's tokens, as f16 pairs
                const uint32_t pcol = tmem + lane_base + kTcP + 32u * sb + static_cast<uint32_t>(my0 / 2);
                const uint32_t lcol = tmem + lane_base + kTcPlo + 32u * sb + static_cast<uint32_t>(my0 / 2);
#pragma unroll
                for (int q = 0; q < kTpc / 16; ++q) {
                    uint32_t h[8];
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        h[t] = f32x2_to_f16x2(p[16 * q + 2 * t], p[16 * q + 2 * t + 1]);
                    tmem_st8(pcol + 8u * q, h);
                    if constexpr (kPrecise) {              // what the f16 rounding of P dropped
                        uint32_t l[8];
#pragma unroll
                        for (int t = 0; t < 8; ++t) {
                            const float2 hf = f16x2_to_f32x2(h[t]);
                            l[t] = f32x2_to_f16x2(p[16 * q + 2 * t] - hf.x, p[16 * q + 2 * t + 1] - hf.y);
                        }
                        tmem_st8(lcol + 8u * q, l);
                    }
                }
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_full[sb]);
            }
            // the last tile's O += P V
            if (!*abort_flag)
                wait_or_abort(&pv_done[(n_tiles - 1) % kKV], ((n_tiles - 1) / kKV) & 1, kCopyWaitLimitNs,
                              abort_flag, 4u);
            __syncwarp();
            tmem_fence_after_sync();
        }
        tmem_fence_before_sync();
        __syncthreads();                                   // every role has finished or given up
        tmem_fence_after_sync();
        const bool failed = s_abort != 0;
        if (failed) {
            // Drain the copies still in flight (issued, not seen landed) with
            // the full limit, so that none lands in shared memory after the
            // CTA has moved on.  Tile t's copy is phase t / kStages of stage
            // t % kStages.
            if (warp == J::kCopy && lane == 0) {
                bool drained = true;
                for (int t = s_landed; t < issued; ++t)
                    drained &= mbar_wait_bounded(&landed[t % kStages], (t / kStages) & 1, kCopyWaitLimitNs);
                if (!drained)
                    atomicOr(&g_umma_error, 2u);
            }
            publish_invalid();
        }

        // ------------------------------------------ merge the parts of each row
        // (groups' halves and copies: part i of row r is slot r + i Rp)
        float *buf = reinterpret_cast<float *>(sm);                      // [128 kGroups][kMergeStride]
        float *sm_m = buf + J::kSoftThreads * kMergeStride;
        float *sm_l = sm_m + J::kSoftThreads;
        float *sm_lse = sm_l + J::kSoftThreads;
        constexpr int kParts = J::kSoftThreads / Rp;
        if (!failed && tid < J::kSoftThreads) {
            sm_m[tid] = m_used;
            sm_l[tid] = l_sum;
            named_barrier_sync(1, J::kSoftThreads);
            float wgt = 0.f;
            if (row_valid) {
                float M = -INFINITY;
#pragma unroll
                for (int i = 0; i < kParts; ++i)
                    M = fmaxf(M, sm_m[Rp * i + r]);
                float L = 0.f;
#pragma unroll
                for (int i = 0; i < kParts; ++i) {         // a NaN sum stays one
                    const float mi = sm_m[Rp * i + r];
                    L += (mi != -INFINITY ? fast_exp2(mi - M) : 0.f) * sm_l[Rp * i + r];
                }
                const float vs = kBlocks ? 1.f : a.v_scale[kvh];
                if (L != 0.f)
                    wgt = (m_used != -INFINITY ? fast_exp2(m_used - M) : L == L ? 0.f : L) * vs / L;
                if (tid < Rp)
                    sm_lse[r] = L == 0.f ? -INFINITY : L == L ? M + __log2f(L) - kLift : INFINITY;
            }
            // row m of O, weighted, into the merge buffer (a part that saw no
            // token writes zeros)
            __syncwarp();
            const uint32_t ocol = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + kTcO + 128u * gr;
#pragma unroll
            for (int cc = 0; cc < 8; ++cc) {
                uint32_t o[16];
                tmem_ld16(ocol + 16 * cc, o);
                if constexpr (kPrecise) {
                    if (n_tiles > kFlushTiles) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 v = sums[(4 * cc + i) ^ (m & 7)];
                            o[4 * i] = __float_as_uint(fmaf(v.x, sums_mul, __uint_as_float(o[4 * i])));
                            o[4 * i + 1] = __float_as_uint(fmaf(v.y, sums_mul, __uint_as_float(o[4 * i + 1])));
                            o[4 * i + 2] = __float_as_uint(fmaf(v.z, sums_mul, __uint_as_float(o[4 * i + 2])));
                            o[4 * i + 3] = __float_as_uint(fmaf(v.w, sums_mul, __uint_as_float(o[4 * i + 3])));
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 v = wgt != 0.f
                                         ? make_float4(__uint_as_float(o[i]) * wgt, __uint_as_float(o[i + 1]) * wgt,
                                                       __uint_as_float(o[i + 2]) * wgt, __uint_as_float(o[i + 3]) * wgt)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
                    *reinterpret_cast<float4 *>(buf + tid * kMergeStride + 16 * cc + i) = v;
                }
            }
            tmem_fence_before_sync();
            named_barrier_sync(1, J::kSoftThreads);
            // the parts' sum of each (row, 4 dims) item
            for (int it = tid; it < R * 32; it += J::kSoftThreads) {
                const int rr = it >> 5, d4 = 4 * (it & 31);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    const float4 x = *reinterpret_cast<const float4 *>(buf + (Rp * i + rr) * kMergeStride + d4);
                    v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
                }
                const int64_t id = row_id(a, b, kvh, rr);
                if (nsplit == 1)
                    store_row_value4(a.out, id * kHeadDim + d4, v, a.out_fp32);
                else
                    *reinterpret_cast<float4 *>(a.ws_o + (id * a.max_splits + split) * kHeadDim + d4) = v;
            }
            if (nsplit > 1 && tid < R)
                a.ws_lse[row_id(a, b, kvh, tid) * a.max_splits + split] = sm_lse[tid];
        }
        tmem_fence_before_sync();
        __syncthreads();
        if (warp == 0) {
            tmem_fence_after_sync();
            tmem_dealloc(tmem, kTmemCols);
        }
    }
}

template <bool kPrecise, int kTpc, bool kBlocks>
cudaError_t configure_rows(int dev)
{
    static int configured[64] = {0};
    if (dev >= 0 && dev < 64 && configured[dev])
        return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(decode_rows_kernel<kPrecise, kTpc, kBlocks>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, view_smem_bytes());
    if (e == cudaSuccess && dev >= 0 && dev < 64)
        configured[dev] = 1;
    return e;
}

template <bool kPrecise, int kTpc, bool kBlocks>
cudaError_t launch_rows(const ViewArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                        cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    e = configure_rows<kPrecise, kTpc, kBlocks>(dev);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.max_splits), static_cast<unsigned>(a.num_kv_heads),
                       static_cast<unsigned>(a.batch));
    cfg.blockDim = dim3(Jobs<kPrecise>::kThreads);
    cfg.dynamicSmemBytes = view_smem_bytes();
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, decode_rows_kernel<kPrecise, kTpc, kBlocks>, k_map, v_map, a);
    if (e != cudaSuccess)
        return e;
    return cudaGetLastError();
}

template <bool kBlocks>
cudaError_t launch_rows_build(const ViewArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                              cudaStream_t stream)
{
    if (a.batch == 0)
        return cudaSuccess;
    const int rows = a.n_query * a.group;
    if (rows < 17 || rows > 128)
        return cudaErrorInvalidValue;                      // the planner sends no others here
    const cudaError_t e = rows > 64 ? a.out_fp32 ? launch_rows<true, 64, kBlocks>(a, k_map, v_map, stream)
                                                 : launch_rows<false, 64, kBlocks>(a, k_map, v_map, stream)
                          : a.out_fp32 ? launch_rows<true, 32, kBlocks>(a, k_map, v_map, stream)
                                       : launch_rows<false, 32, kBlocks>(a, k_map, v_map, stream);
    return e != cudaSuccess || a.max_splits == 1 ? e : launch_combine_rows(a, stream);
}

} // namespace

cudaError_t launch_decode_umma_view(const ViewArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                                    cudaStream_t stream)
{
    return a.k_exp != nullptr ? launch_rows_build<true>(a, k_map, v_map, stream)
                              : launch_rows_build<false>(a, k_map, v_map, stream);
}

cudaError_t read_umma_view_error(uint32_t *bits, bool clear) { return read_umma_error_word(bits, clear); }

} // namespace kvq
