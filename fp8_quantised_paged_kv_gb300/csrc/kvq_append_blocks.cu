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
// are read only where the exponent grew.  Bound: HBM once there are some
// thousand tokens (58,637 tokens x 8 heads, 360 MB: 53.3 us, the measured copy
// rate), three rounds of dependent loads below (64 requests x 1 token: 2.5
// us).  What counts is how many rows are under way: the maximum goes over
// bf16 pairs, so that no fp32 copy of a row lives beside it, and 64 registers
// let four CTAs fit on an SM (fp32 maxima, 128 registers and two CTAs: 81 us).
// Variants that gave each warp several blocks, with and without the next
// block's loads issued early, took 56.6 to 60.6 us.
//
// Work items are numbered by offset / (16 x blocks per item) + 2 * request,
// which leaves each request room for the blocks that its new tokens can touch
// (n new tokens touch at most (n + 14) / 16 + 1) without a prefix sum; a CTA
// finds its request by testing 256 requests at a time.  (Offsets that descend
// break the numbering: blocks are then passed over, but each item still works
// by its request's own offsets.)  An item is one block,
// or with one or two KV heads as many as fill the CTA's eight warps (64,390
// tokens of one head: 11.0 us against 16.2).
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
// (n tokens of which n / (16 G) = q remainder b touch at most G q + G + 1
// blocks: q + 2 items of G blocks.)
__device__ __forceinline__ int64_t first_item(const AppendBlocksArgs &a, int64_t r, int shift)
{
    return (request_offset(a, r) >> (4 + shift)) + 2 * r;
}

// Items of a request with n new tokens, wherever they start.
__host__ __device__ inline int64_t items_per_request(int64_t n, int shift)
{
    return (((n + kBlockTokens - 2) / kBlockTokens) >> shift) + 1;
}

// The last request whose first item is not past `item` (0 if none is), by the
// whole block: one round of tests per 256-fold of the batch.
__device__ int64_t find_request(const AppendBlocksArgs &a, int64_t item, int shift)
{
    int64_t lo = 0, count = a.batch;                       // the answer lies in [lo, lo + count)
    while (count > 1) {
        const int64_t step = (count + kThreads - 1) / kThreads;
        const int64_t at = lo + threadIdx.x * step;
        const bool reached = threadIdx.x * step < count && first_item(a, at, shift) <= item;
        const int passed = __syncthreads_count(reached);
        const int64_t skip = passed > 0 ? (passed - 1) * step : 0;
        lo += skip;
        count = min(step, count - skip);
    }
    return lo;
}

// The larger of m's and |w|'s bf16 elements, pair by pair (m holds no NaN and
// no sign; a NaN in w is passed over).
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %2;\n\tmax.bf16x2 %0, %1, t;\n\t}" : "=r"(r) : "r"(m), "r"(w));
    return r;
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

// kShift: log2 of the blocks per work item.
template <int kShift>
__global__ void __launch_bounds__(kThreads, 4) append_blocks_kernel(const AppendBlocksArgs a)
{
    grid_launch_dependents();              // a dependent decode launch may begin now
    const int64_t item = blockIdx.x;
    int64_t r, local;                      // the request, and the warp's block among those it writes
    if (a.token_offsets == nullptr) {      // equal counts: the same number of items each
        const int64_t per = items_per_request(a.num_tokens / a.batch, kShift);
        r = item / per;
        local = (item % per) << kShift;
    } else {
        r = find_request(a, item, kShift);
        local = (item - first_item(a, r, kShift)) << kShift;
    }
    const int units = 2 * a.num_kv_heads, warp = threadIdx.x / 32;
    const int unit = kShift > 0 ? warp % units : static_cast<int>(blockIdx.y) * kWarps + warp;
    if (kShift > 0)
        local += warp / units;
    if (unit >= units)
        return;
    const bool is_v = unit >= a.num_kv_heads;
    const int h = is_v ? unit - a.num_kv_heads : unit;
    const int lane = threadIdx.x % 32, part = lane % kThreadsPerRow, half = lane / kThreadsPerRow;

    // the request's new tokens: rows off .. off + n - 1, positions start .. len - 1
    const int64_t off = request_offset(a, r), n = request_offset(a, r + 1) - off;
    const int64_t len = __ldg(a.seq_lens + r), start = len - n;
    const bool aborted = a.abort_flags != nullptr && __ldg(a.abort_flags + r) != 0;
    if (aborted || n <= 0 || off < 0 || off + n > a.num_tokens || start < 0 ||
        len > static_cast<int64_t>(a.max_pages_per_seq) * a.page_size || local < 0)
        return;
    const int64_t block = start / kBlockTokens + local, pos0 = block * kBlockTokens;
    if (pos0 >= len)
        return;
    const int lo = static_cast<int>(max(start - pos0, static_cast<int64_t>(0)));     // new rows of the block
    const int hi = static_cast<int>(min(len - pos0, static_cast<int64_t>(kBlockTokens)));
    const int ps_shift = __ffs(a.page_size) - 1, bpp_shift = ps_shift - 4;           // blocks per page: page_size / 16
    const int32_t page = __ldg(a.block_table + r * a.max_pages_per_seq + (block >> bpp_shift));

    // bytes from one token's row to the next, and this lane's part of row `half`
    const uint32_t row_step = static_cast<uint32_t>(a.num_kv_heads) * kHeadDim * 2;
    const uint8_t *src = static_cast<const uint8_t *>(is_v ? a.v_new : a.k_new) +
                         (off - start + pos0 + half) * row_step + h * kHeadDim * 2 + part * 16;
    uint4 x[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int row = i * kRowsPerLoad + half;
        x[i] = make_uint4(0, 0, 0, 0);
        if (row >= lo && row < hi)
            x[i] = __ldg(reinterpret_cast<const uint4 *>(src));
        src += kRowsPerLoad * row_step;
    }
    if (page < 0 || page >= a.num_pages)
        return;
    const int sub = static_cast<int>(block & ((1 << bpp_shift) - 1));
    const int64_t tile = static_cast<int64_t>(page) * a.num_kv_heads + h;
    int8_t *exp = (is_v ? a.v_exp : a.k_exp) + (tile << bpp_shift) + sub;
    const int e_old = lo > 0 ? *exp : kBlockExpMin;
    uint32_t m2 = 0;                                       // largest magnitudes of even and odd dims
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        m2 = amax2(amax2(amax2(amax2(m2, x[i].x), x[i].y), x[i].z), x[i].w);
    const int need = block_exponent(__reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16)));
    const int e = lo > 0 ? max(e_old, need) : need;

    uint8_t *dst = static_cast<uint8_t *>(is_v ? a.v_cache : a.k_cache) +
                   ((tile << ps_shift) + sub * kBlockTokens) * kHeadDim + part * 8;
    if (lo > 0 && e > e_old) {                             // the earlier rows move to the new exponent
        const int d = e - e_old;
        const float mul = d > 126 ? 0.f : __int_as_float((127 - d) << 23);
        constexpr int kOld = 4;                            // rows per lane and trip
#pragma unroll 1
        for (int i0 = 0; i0 < kLoads; i0 += kOld) {
            uint2 c[kOld];
#pragma unroll
            for (int i = 0; i < kOld; ++i) {
                const int row = (i0 + i) * kRowsPerLoad + half;
                if (row < lo)
                    c[i] = *reinterpret_cast<const uint2 *>(dst + row * kHeadDim);
            }
#pragma unroll
            for (int i = 0; i < kOld; ++i) {
                const int row = (i0 + i) * kRowsPerLoad + half;
                if (row < lo)
                    *reinterpret_cast<uint2 *>(dst + row * kHeadDim) =
                        make_uint2(rescale4_e4m3(c[i].x, mul), rescale4_e4m3(c[i].y, mul));
            }
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

template <int kShift>
cudaError_t launch(const AppendBlocksArgs &a, cudaStream_t stream)
{
    const int64_t items = a.token_offsets == nullptr
                              ? a.batch * items_per_request(a.num_tokens / a.batch, kShift)
                              : (a.num_tokens >> (4 + kShift)) + 2 * static_cast<int64_t>(a.batch);
    if (items > 0x7FFFFFFF)
        return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(items),
                    kShift > 0 ? 1u : static_cast<unsigned>((2 * a.num_kv_heads + kWarps - 1) / kWarps));
    append_blocks_kernel<kShift><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_append_blocks(const AppendBlocksArgs &a, cudaStream_t stream)
{
    if (a.batch == 0 || a.num_tokens == 0)
        return cudaSuccess;
    return a.num_kv_heads == 1 ? launch<2>(a, stream) : a.num_kv_heads == 2 ? launch<1>(a, stream) : launch<0>(a, stream);
}

} // namespace kvq
