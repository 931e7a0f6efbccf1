// kvq_combine_rows.cu -- the combine of the splits as a launch of its own behind
// a windowed or block-scaled attention: out = sum_s w_s o_s / sum_s w_s with
// w_s = 2^(lse_s - max lse), for every row of the output.
#include <cuda_bf16.h>

#include "kvq_ptx.cuh"
#include "kvq_view.cuh"

namespace kvq {
namespace {

__device__ __forceinline__ void store_row4(void *out, int64_t idx, float4 v, bool fp32)
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

// A warp takes one row, a lane four dims of it and the lse of one split, with a
// round of kRound splits' partials in flight.  By the last CTA of each (request,
// KV head) to finish it took 14 us on 128 rows in 9 splits and 17 on 8 rows in
// 96, while the other SMs waited; here the launch, 2 to 3 us, is most of it (1
// x 60,000 tokens, single: 22.4 us in 48 splits, 15.9 in 67; 4 query tokens
// 32.3, 21.3).  A NaN sum (a split with lse +inf) makes the row NaN.
constexpr int kCombineWarps = 4;
__global__ void __launch_bounds__(32 * kCombineWarps)
combine_rows_kernel(const ViewArgs a)
{
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kCombineWarps + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    const int64_t rows_per_request = static_cast<int64_t>(a.n_query) * a.num_q_heads;
    grid_dependency_wait();
    if (row >= a.batch * rows_per_request)
        return;
    const int b = static_cast<int>(row / rows_per_request);
    const int64_t real = a.seq_lens[b];
    const bool aborted = a.abort_flags != nullptr && a.abort_flags[b] != 0;
    if (aborted || real <= 0 || real > static_cast<int64_t>(a.max_pages_per_seq) * a.page_size) {
        store_row4(a.out, row * kHeadDim + 4 * lane, make_float4(0.f, 0.f, 0.f, 0.f), a.out_fp32);
        return;
    }
    const int64_t len = shown_context(a, real, __ffs(a.page_size) - 1).len;
    int nsplit = static_cast<int>((len + a.split_tokens - 1) / a.split_tokens);
    // partial of split s: at + s * step
    int64_t at = row * a.max_splits;
    int step = 1;
    if (a.resident_ctas > 0) {
        const int per = a.n_query > 1 ? kMultiRowsPerCta : kMaxGroup;      // rows of a slot
        const int i = static_cast<int>(row % rows_per_request) / a.num_q_heads, hq = static_cast<int>(row % a.num_q_heads);
        const int kvh = hq / a.group, r = i * a.group + hq % a.group;
        const int2 pair = __ldcg(a.ws_pairs + (static_cast<int64_t>(b) * a.num_kv_heads + kvh) * a.row_blocks + r / per);
        at = static_cast<int64_t>(pair.x) * per + r % per;
        step = per;
        nsplit = pair.y;
    }
    if (nsplit == 1)                                       // written already
        return;
    constexpr int kRound = 8;
    const float *lse = a.ws_lse + at;
    const float *part = a.ws_o + at * kHeadDim + 4 * lane;
    float w = lane < nsplit ? __ldcg(lse + static_cast<int64_t>(lane) * step) : -INFINITY;
    float M = 0.f, inv = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < nsplit; s0 += kRound) {
        float4 v[kRound];
#pragma unroll
        for (int k = 0; k < kRound; ++k)
            v[k] = s0 + k < nsplit
                       ? __ldcg(reinterpret_cast<const float4 *>(part + static_cast<int64_t>(s0 + k) * step * kHeadDim))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
        if (s0 == 0) {                                     // the largest lse, and the weights' sum
            M = w;
            bool bad = w != w;
            for (int c = 32; c < nsplit; c += 32) {
                const float y = c + lane < nsplit ? __ldcg(lse + static_cast<int64_t>(c + lane) * step) : -INFINITY;
                bad |= y != y;
                M = fmaxf(M, y);
            }
            bad = __any_sync(0xFFFFFFFFu, bad);
            for (int off = 16; off > 0; off >>= 1)
                M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
            float sum = 0.f;
            for (int c = 0; c < nsplit; c += 32) {
                const float y = c == 0 ? w : c + lane < nsplit ? __ldcg(lse + static_cast<int64_t>(c + lane) * step) : -INFINITY;
                sum += y == -INFINITY ? 0.f : fast_exp2(y - M);
            }
            for (int off = 16; off > 0; off >>= 1)
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
            inv = bad || sum == 0.f ? 0.f : 1.f / sum;     // NaN stays
        }
        if (s0 % 32 == 0) {                                // lane s: the weight of split s0 + s
            if (s0 > 0)
                w = s0 + lane < nsplit ? __ldcg(lse + static_cast<int64_t>(s0 + lane) * step) : -INFINITY;
            w = inv == 0.f || w == -INFINITY ? 0.f : fast_exp2(w - M) * inv;
        }
#pragma unroll
        for (int k = 0; k < kRound; ++k) {
            const float wk = __shfl_sync(0xFFFFFFFFu, w, (s0 + k) & 31);
            if (s0 + k < nsplit && wk != 0.f) {            // a split without weight may hold anything
                acc.x += wk * v[k].x;
                acc.y += wk * v[k].y;
                acc.z += wk * v[k].z;
                acc.w += wk * v[k].w;
            }
        }
    }
    store_row4(a.out, row * kHeadDim + 4 * lane, acc, a.out_fp32);
}

} // namespace

cudaError_t launch_combine_rows(const ViewArgs &a, cudaStream_t stream)
{
    const int64_t rows = static_cast<int64_t>(a.batch) * a.n_query * a.num_q_heads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((rows + kCombineWarps - 1) / kCombineWarps));
    cfg.blockDim = dim3(32 * kCombineWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, combine_rows_kernel, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace kvq
