// kvq_append_blocks.cu -- quantise-on-append into the block-scaled cache: e4m3
// codes with one power-of-two exponent per block of 16 consecutive positions
// and KV head, K and V apart.
//
// Mathematics.  A code c in a block of exponent e stands for c * 2^e.  The
// block's need is the least e with amax <= 448 * 2^e over its new tokens
// (NaN passed over, 0 needs the least exponent), held in [-48, 48].  A block
// whose first position is among the new tokens starts over with e = need;
// otherwise e = max(e_old, need), and where that grew the earlier rows' codes
// become e4m3(c * 2^(e_old - e)).  Powers of two make this cheap and mild: the
// scaling is exact in fp32, e4m3's relative precision does not depend on where
// in its normal range a value lies, so a power of two loses nothing against a
// scale of amax / 448 but part of one step at the subnormal end, and moving a
// code to a larger exponent is exact until it turns subnormal.
//
// Split.  One warp per (request, block, K|V, KV head): a row of 256 bytes is 16
// lanes x 16 bytes, so the block's 16 new rows are eight 16-byte loads per
// lane, all issued before the first is used, the maximum stays in registers
// and every row is read once.  Rows leave as 8 codes per lane.  The old rows
// are read only where the exponent grew.
//
// Work items are numbered by offset / 16 + 2 * request, which leaves each
// request room for the blocks that its new tokens can touch (n new tokens
// touch at most (n + 14) / 16 + 1) without a prefix sum; a CTA finds its
// request by testing 256 requests at a time.
#include "kvq_rowops.cuh"

namespace kvq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRowsPerLoad = 32 / kThreadsPerRow;          // a warp covers two rows per load
constexpr int kLoads = kBlockTokens / kRowsPerLoad;        // 8

__device__ __forceinline__ int64_t request_offset(const AppendBlocksArgs &a, int64_t r)
{
    return a.token_offsets ? static_cast<int64_t>(__ldg(a.token_offsets + r))
                           : r * (a.num_tokens / a.batch);
}

// First work item of request r; also the item count's bound for r = batch.
__device__ __forceinline__ int64_t first_item(const AppendBlocksArgs &a, int64_t r)
{
    return request_offset(a, r) / kBlockTokens + 2 * r;
}

// The last request whose first item is not past `item` (0 if none is), by the
// whole block: one round of tests per 256-fold of the batch.
__device__ int64_t find_request(const AppendBlocksArgs &a, int64_t item)
{
    int64_t lo = 0, count = a.batch;                       // the answer lies in [lo, lo + count)
    while (count > 1) {
        const int64_t step = (count + kThreads - 1) / kThreads;
        const int64_t at = lo + threadIdx.x * step;
        const bool reached = threadIdx.x * step < count && first_item(a, at) <= item;
        const int passed = __syncthreads_count(reached);
        const int64_t skip = passed > 0 ? (passed - 1) * step : 0;
        lo += skip;
        count = min(step, count - skip);
    }
    return lo;
}

// Largest magnitude (bf16 bits) of a word's two elements, NaN as 0.
__device__ __forceinline__ uint32_t amax2(uint32_t w)
{
    const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
    return max(lo > 0x7F80u ? 0u : lo, hi > 0x7F80u ? 0u : hi);
}

// Least e in range with m <= 448 * 2^e, for the bf16 bits of m >= 0:
// 448 = 1.75 * 2^8, and 1.75 is the significand field 96 of 128.
__device__ __forceinline__ int block_exponent(uint32_t m)
{
    const int e = static_cast<int>(m >> 7) - 127 - 8 + ((m & 127u) > 96u ? 1 : 0);
    return m == 0 ? kBlockExpMin : max(kBlockExpMin, min(kBlockExpMax, e));
}

__device__ __forceinline__ uint32_t scale4_e4m3(uint32_t w0, uint32_t w1, float mul)
{
    const float2 p0 = bf16x2_to_f32x2(w0), p1 = bf16x2_to_f32x2(w1);
    return static_cast<uint32_t>(f32x2_to_e4m3x2(p0.x * mul, p0.y * mul)) |
           (static_cast<uint32_t>(f32x2_to_e4m3x2(p1.x * mul, p1.y * mul)) << 16);
}

__device__ __forceinline__ uint32_t rescale4_e4m3(uint32_t codes, float mul)
{
    const float2 p0 = f16x2_to_f32x2(lo16_e4m3x2_to_f16x2(codes)), p1 = f16x2_to_f32x2(hi16_e4m3x2_to_f16x2(codes));
    return static_cast<uint32_t>(f32x2_to_e4m3x2(p0.x * mul, p0.y * mul)) |
           (static_cast<uint32_t>(f32x2_to_e4m3x2(p1.x * mul, p1.y * mul)) << 16);
}

__global__ void __launch_bounds__(kThreads) append_blocks_kernel(const AppendBlocksArgs a)
{
    grid_launch_dependents();              // a dependent decode launch may begin now
    const int64_t item = blockIdx.x;
    int64_t r, local;
    if (a.token_offsets == nullptr) {      // equal counts: the same number of items each
        const int64_t n = a.num_tokens / a.batch, per = (n + kBlockTokens - 2) / kBlockTokens + 1;
        r = item / per;
        local = item % per;
    } else {
        r = find_request(a, item);
        local = item - first_item(a, r);
    }
    const int unit = blockIdx.y * kWarps + threadIdx.x / 32;
    if (unit >= 2 * a.num_kv_heads)
        return;
    const bool is_v = unit >= a.num_kv_heads;
    const int h = is_v ? unit - a.num_kv_heads : unit;
    const int lane = threadIdx.x % 32, part = lane % kThreadsPerRow, half = lane / kThreadsPerRow;

    // the request's new tokens: rows off .. off + n - 1, positions start .. len - 1
    const int64_t off = request_offset(a, r), n = request_offset(a, r + 1) - off;
    const int64_t len = __ldg(a.seq_lens + r), start = len - n;
    const bool aborted = a.abort_flags != nullptr && __ldg(a.abort_flags + r) != 0;
    if (aborted || n <= 0 || off < 0 || off + n > a.num_tokens || start < 0 ||
        len > static_cast<int64_t>(a.max_pages_per_seq) * a.page_size)
        return;
    const int64_t block = start / kBlockTokens + local, pos0 = block * kBlockTokens;
    if (local < 0 || pos0 >= len)
        return;
    const int lo = static_cast<int>(max(start - pos0, static_cast<int64_t>(0)));     // new rows of the block
    const int hi = static_cast<int>(min(len - pos0, static_cast<int64_t>(kBlockTokens)));
    const int32_t page = __ldg(a.block_table + r * a.max_pages_per_seq + pos0 / a.page_size);

    const uint16_t *src = static_cast<const uint16_t *>(is_v ? a.v_new : a.k_new) + h * kHeadDim + part * 8;
    uint4 x[kLoads];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int row = i * kRowsPerLoad + half;
        x[i] = make_uint4(0, 0, 0, 0);
        if (row >= lo && row < hi)
            x[i] = __ldg(reinterpret_cast<const uint4 *>(src + (off + pos0 + row - start) * a.num_kv_heads * kHeadDim));
    }
    if (page < 0 || page >= a.num_pages)
        return;
    const int sub = static_cast<int>(pos0 % a.page_size) / kBlockTokens, per_page = a.page_size / kBlockTokens;
    int8_t *exp = (is_v ? a.v_exp : a.k_exp) + (static_cast<int64_t>(page) * a.num_kv_heads + h) * per_page + sub;
    const int e_old = lo > 0 ? *exp : kBlockExpMin;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        m = max(max(m, max(amax2(x[i].x), amax2(x[i].y))), max(amax2(x[i].z), amax2(x[i].w)));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    const int need = block_exponent(m);
    const int e = lo > 0 ? max(e_old, need) : need;

    uint8_t *dst = static_cast<uint8_t *>(is_v ? a.v_cache : a.k_cache) +
                   ((static_cast<int64_t>(page) * a.num_kv_heads + h) * a.page_size + sub * kBlockTokens) * kHeadDim +
                   part * 8;
    if (lo > 0 && e > e_old) {                             // the earlier rows move to the new exponent
        const int d = e - e_old;
        const float mul = d > 126 ? 0.f : __int_as_float((127 - d) << 23);
        uint2 c[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int row = i * kRowsPerLoad + half;
            if (row < lo)
                c[i] = *reinterpret_cast<const uint2 *>(dst + row * kHeadDim);
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int row = i * kRowsPerLoad + half;
            if (row < lo)
                *reinterpret_cast<uint2 *>(dst + row * kHeadDim) =
                    make_uint2(rescale4_e4m3(c[i].x, mul), rescale4_e4m3(c[i].y, mul));
        }
    }
    // 2^-e: e can be a stored exponent of up to 127, and 2^-127 is subnormal
    const float mul = __int_as_float(e < 127 ? (127 - e) << 23 : 0x00400000);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int row = i * kRowsPerLoad + half;
        if (row >= lo && row < hi)
            *reinterpret_cast<uint2 *>(dst + row * kHeadDim) =
                make_uint2(scale4_e4m3(x[i].x, x[i].y, mul), scale4_e4m3(x[i].z, x[i].w, mul));
    }
    if (lane == 0)
        *exp = static_cast<int8_t>(e);
}

} // namespace

cudaError_t launch_append_blocks(const AppendBlocksArgs &a, cudaStream_t stream)
{
    if (a.batch == 0 || a.num_tokens == 0)
        return cudaSuccess;
    int64_t items;
    if (a.token_offsets == nullptr) {
        const int64_t n = a.num_tokens / a.batch;
        items = a.batch * ((n + kBlockTokens - 2) / kBlockTokens + 1);
    } else {
        items = a.num_tokens / kBlockTokens + 2 * static_cast<int64_t>(a.batch);
    }
    if (items > 0x7FFFFFFF)
        return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(items), static_cast<unsigned>((2 * a.num_kv_heads + kWarps - 1) / kWarps));
    append_blocks_kernel<<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

} // namespace kvq
