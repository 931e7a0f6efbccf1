// kvq_decode.cu -- the decode kernel's build for caches with one scale per KV
// head (or BF16), every token visible, and the planner's occupancy queries.
#include "kvq_decode_split.cuh"

namespace kvq {
cudaError_t launch_decode(const DecodeArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                          cudaStream_t stream)
{
    return launch_build<false, false>(a, k_map, v_map, stream);
}

int decode_cluster_capacity(int n, bool bf16_cache, bool multi)
{
    return cluster_capacity<false>(n, bf16_cache, multi);
}

int decode_ctas_per_sm(bool bf16_cache, bool multi)
{
    // resident CTAs per SM as the shared-memory footprint and the launch
    // bounds allow (no device)
    const int by_smem = bf16_cache ? 233472 / (Tile<true>::kSmemBytes + 1024)
                                   : 233472 / (Tile<false>::kSmemBytes + 1024);
    const int bound = multi ? 2 : kCtasPerSm;
    const int fallback = by_smem < bound ? (by_smem > 0 ? by_smem : 1) : bound;
    static std::mutex mu;
    static std::map<std::tuple<int, bool, bool>, int> cache;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return fallback;
    }
    std::lock_guard<std::mutex> lock(mu);
    const auto key = std::make_tuple(dev, bf16_cache, multi);
    auto it = cache.find(key);
    if (it != cache.end())
        return it->second;
    int n = 0;
    cudaError_t e = cudaSuccess;
    if (multi) {
        e = bf16_cache ? configure<true, false, false, true>(dev) : configure<false, false, false, true>(dev);
        if (e == cudaSuccess)
            e = bf16_cache ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                                 &n, decode_split_kernel<true, false, false, true, false, false>, kThreads, Tile<true>::kSmemBytes)
                           : cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                                 &n, decode_split_kernel<false, false, false, true, false, false>, kThreads, Tile<false>::kSmemBytes);
    } else {
        e = bf16_cache ? configure<true, false, false>(dev) : configure<false, false, false>(dev);
        if (e == cudaSuccess)
            e = bf16_cache ? cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                                 &n, decode_split_kernel<true, false, false, false, false, false>, kThreads, Tile<true>::kSmemBytes)
                           : cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                                 &n, decode_split_kernel<false, false, false, false, false, false>, kThreads, Tile<false>::kSmemBytes);
    }
    if (e != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = fallback;
    }
    cache[key] = n;
    return n;
}

#ifdef KVQ_PHASE_STAMPS
cudaError_t read_decode_stamps(unsigned long long *host, size_t count)
{
    const size_t n = count < static_cast<size_t>(kStampCtas * kStampPoints) ? count
                                                                            : kStampCtas * kStampPoints;
    return cudaMemcpyFromSymbol(host, g_phase_stamps, n * sizeof(unsigned long long));
}
#endif

cudaError_t read_device_error(uint32_t *bits, bool clear) { return read_error_word(bits, clear); }

} // namespace kvq
