// kvq_decode_window.cu -- the decode kernel's build behind a sliding window with sinks, over caches with one
// scale per KV head (or BF16).
#include "kvq_decode_split.cuh"

namespace kvq {

cudaError_t launch_decode_window(const ViewArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                                 cudaStream_t stream)
{
    const cudaError_t e = launch_build<true, false>(a, k_map, v_map, stream);
    return e != cudaSuccess || !a.combine_apart ? e : launch_combine_rows(a, stream);
}

int decode_view_cluster_capacity(int n, bool bf16_cache, bool multi)
{
    return cluster_capacity<true>(n, bf16_cache, multi);
}

// What the launch bounds and the shared memory of the windowed builds (the
// block-scaled ones among them) leave room for.
int decode_view_ctas_per_sm(bool bf16_cache, bool multi)
{
    constexpr int kSm = 233472, kReserved = 1024;
    const int bytes = multi ? (bf16_cache ? smem_bytes<true, true, true>() : smem_bytes<false, true, true>())
                            : (bf16_cache ? smem_bytes<true, false, true>() : smem_bytes<false, false, true>());
    const int by_smem = kSm / (bytes + kReserved), bound = min_ctas(multi, true);
    return by_smem < bound ? by_smem : bound;
}

cudaError_t read_window_error(uint32_t *bits, bool clear) { return read_error_word(bits, clear); }

} // namespace kvq
