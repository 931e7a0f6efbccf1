// kvq_copy_pages.cu -- pages copied inside every cache of a pool in one launch
// (a fork's own copy of a shared last page, pages moved to close gaps).
//
// Nothing but traffic: each listed page is read once and written once.  A CTA
// copies up to 16 KB of one page of one cache: 128 threads with eight 16-byte
// loads in flight each before the first store, so the SM's loads cover HBM's
// latency without shared memory.  (On 8,002 pages of 64 KB this form takes
// 153 to 154 us, 6.83 TB/s read and written, as a plain device copy of the same
// bytes does, 152 us; bulk copies through a shared-memory ring 159 to 197 us, one
// 16-byte load per thread 190 to 202 us.)  The exponents' pages (a few bytes) go by
// words of the largest size that divides them and their array's address.
#include "kvq_ptx.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kThreads = 128;
constexpr int kLoads = 8;
constexpr int kStrip = kThreads * 16;                      // 2,048 bytes: every page is a multiple
constexpr int kPiece = kStrip * kLoads;                    // 16 KB per CTA

__device__ __forceinline__ uint4 ld_stream(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

constexpr int kSmallPerThread = 8;                         // bytes or words of an exponent array per thread

template <typename Word>
__device__ __forceinline__ void copy_small(uint8_t *base, const CopyPagesArgs &a, int64_t worker, int64_t workers)
{
    Word *w = reinterpret_cast<Word *>(base);
    const int64_t words = a.exp_page_bytes / static_cast<int64_t>(sizeof(Word));
    for (int64_t i = worker; i < words * a.num_listed; i += workers) {
        const int64_t pair = i / words, at = i % words;
        const int64_t s = __ldg(a.src_pages + pair), d = __ldg(a.dst_pages + pair);
        if (s >= 0 && s < a.num_pages && d >= 0 && d < a.num_pages)
            w[d * words + at] = w[s * words + at];
    }
}

// Row y of the grid: `extra` of the exponents' blocks (small_blocks for each
// exponent array; first, so that their dependent loads hide behind the
// pages'), then the num_listed pages of cache y, `pieces` blocks each.
__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const __grid_constant__ CopyPagesArgs a,
                                                                uint32_t pieces, uint32_t small_blocks,
                                                                uint32_t extra)
{
    grid_launch_dependents();              // a dependent decode launch may begin now
    if (blockIdx.x < extra) {
        const uint32_t block = blockIdx.y * extra + blockIdx.x, array = block / small_blocks;
        if (array >= static_cast<uint32_t>(a.num_exps))
            return;
        uint8_t *base = static_cast<uint8_t *>(a.arrays[a.num_caches + array]);
        const int64_t worker = static_cast<int64_t>(block - array * small_blocks) * kThreads + threadIdx.x;
        const int64_t workers = static_cast<int64_t>(small_blocks) * kThreads;
        const uintptr_t unit = reinterpret_cast<uintptr_t>(base) | static_cast<uintptr_t>(a.exp_page_bytes);
        if (unit % 16 == 0)
            copy_small<uint4>(base, a, worker, workers);
        else if (unit % 4 == 0)
            copy_small<uint32_t>(base, a, worker, workers);
        else
            copy_small<uint8_t>(base, a, worker, workers);
        return;
    }
    uint8_t *base = static_cast<uint8_t *>(a.arrays[blockIdx.y]);
    const uint32_t pair = (blockIdx.x - extra) / pieces, piece = (blockIdx.x - extra) - pair * pieces;
    const int64_t s = __ldg(a.src_pages + pair), d = __ldg(a.dst_pages + pair);
    if (s < 0 || s >= a.num_pages || d < 0 || d >= a.num_pages || s == d)
        return;
    const int64_t at = static_cast<int64_t>(piece) * kPiece + threadIdx.x * 16;
    const uint8_t *src = base + s * a.cache_page_bytes + at;
    uint8_t *dst = base + d * a.cache_page_bytes + at;
    uint4 v[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        if (at + i * kStrip < a.cache_page_bytes)
            v[i] = ld_stream(reinterpret_cast<const uint4 *>(src + i * kStrip));
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
        if (at + i * kStrip < a.cache_page_bytes)
            __stcs(reinterpret_cast<uint4 *>(dst + i * kStrip), v[i]);
}

} // namespace

cudaError_t launch_copy_pages(const CopyPagesArgs &a, cudaStream_t stream)
{
    if (a.num_listed == 0 || a.num_caches + a.num_exps == 0)
        return cudaSuccess;
    const int64_t pieces = (a.cache_page_bytes + kPiece - 1) / kPiece;
    const int64_t per_cache = a.num_caches > 0 ? pieces * a.num_listed : 0;
    const int64_t small_blocks = (a.exp_page_bytes * a.num_listed + kThreads * kSmallPerThread - 1) /
                                 (kThreads * kSmallPerThread);
    const int64_t rows = a.num_caches > 0 ? a.num_caches : 1;
    const int64_t extra = (small_blocks * a.num_exps + rows - 1) / rows;
    if (per_cache + extra > 0x7FFFFFFF || extra * rows > 0x7FFFFFFF)
        return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(per_cache + extra), static_cast<unsigned>(rows));
    copy_pages_kernel<<<grid, kThreads, 0, stream>>>(a, static_cast<uint32_t>(pieces),
                                                     static_cast<uint32_t>(small_blocks), static_cast<uint32_t>(extra));
    return cudaGetLastError();
}

} // namespace kvq
