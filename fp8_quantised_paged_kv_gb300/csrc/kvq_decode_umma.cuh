// kvq_decode_umma.cuh -- what the two tensor-memory decode kernels share: the
// tile, its tensor-core instructions, the scaling of the query rows, bounded
// waits and the error word (one for each file that includes this).
#pragma once

#include <cfloat>

#include <cuda_bf16.h>

#include "kvq_internal.h"
#include "kvq_ptx.cuh"
#include "kvq_umma.cuh"

namespace kvq {
namespace {

// Sticky error word of this build of the kernel (read together with the other
// decode kernels' words).  Bit 0: a bulk-copy wait timed out.  Bit 1: the drain that
// follows also gave up.  Bit 2: a tensor-core completion wait timed out.
__device__ unsigned int g_umma_error = 0;

constexpr int kTile = 64;                                 // tokens per tile
constexpr int kStages = 5;                                // e4m3 ring
constexpr int kKVBytes = 32768;                           // a tile's operands: K and V as f16
constexpr int kMergeStride = 132;                         // floats per row of the merge buffer
constexpr int kMaxPageList = 8192 / 16 + 8;
constexpr uint32_t kTmemCols = 512;
constexpr float kRaiseThreshold = 8.f;

constexpr uint32_t kIdescS = umma_idesc_f16(128, kTile, false);
constexpr uint32_t kIdescPV = umma_idesc_f16(128, 128, true);

__device__ __forceinline__ void store_row_value(void *out, int64_t idx, float v, bool fp32)
{
    if (fp32)
        static_cast<float *>(out)[idx] = v;
    else
        static_cast<__nv_bfloat16 *>(out)[idx] = __float2bfloat16_rn(v);
}

// Four consecutive values (idx a multiple of 4).
__device__ __forceinline__ void store_row_value4(void *out, int64_t idx, float4 v, bool fp32)
{
    if (fp32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + idx) = v;
    } else {
        uint2 h;
        h.x = f32x2_to_bf16x2(v.x, v.y);
        h.y = f32x2_to_bf16x2(v.z, v.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(out) + idx) = h;
    }
}

// Exponent e putting the largest |q| of a row (bf16 bits, sign cleared) in
// [2^14, 2^15) (capped at 100; a zero row keeps 0): the row is multiplied by
// 2^e before it becomes f16 and its scores by 2^-e, so no element overflows
// f16 and every element within 2^28 of the row's largest keeps its bits.
__device__ __forceinline__ int q_row_exponent(uint32_t mx)
{
    if (mx == 0)
        return 0;
    const int field = static_cast<int>(mx >> 7);
    const int e_floor = field != 0 ? field - 127 : (31 - __clz(static_cast<int>(mx))) - 133;
    const int e = 14 - e_floor;
    return e > 100 ? 100 : e;
}

// Global row (in [B][n][Hq]) of local row r of (request b, KV head kvh).
__device__ __forceinline__ int64_t row_id(const DecodeArgs &a, int b, int kvh, int r)
{
    return (static_cast<int64_t>(b) * a.n_query + r / a.group) * a.num_q_heads + kvh * a.group + r % a.group;
}

// Wait for phase `parity` of `bar`, suspended in hardware between looks
// (at most 200 us at a time).  Gives up when another warp has given up (the
// CTA's abort flag), or after limit_ns (0: at once, without looking), in
// which case it raises the abort flag and sets `bit` in the error word.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, uint64_t limit_ns,
                                              volatile int *abort_flag, unsigned bit)
{
    if (limit_ns != 0) {
        if (mbar_try_wait(bar, parity))                    // already complete: no clock read
            return true;
        const uint64_t start = global_timer_ns();
        for (uint32_t i = 0; i < (1u << 24); ++i) {
            if (mbar_try_wait_sleep(bar, parity, 200000u))
                return true;
            if (*abort_flag)
                return false;
            if (global_timer_ns() - start > limit_ns)
                break;
        }
    }
    *abort_flag = 1;
    atomicOr(&g_umma_error, bit);
    return false;
}

// Read (and, if asked, reset) this build's error word.
cudaError_t read_umma_error_word(uint32_t *bits, bool clear)
{
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_umma_error, sizeof v);
    if (e != cudaSuccess)
        return e;
    if (bits)
        *bits = v;
    if (clear) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_umma_error, &zero, sizeof zero);
    }
    return e;
}

} // namespace
} // namespace kvq
