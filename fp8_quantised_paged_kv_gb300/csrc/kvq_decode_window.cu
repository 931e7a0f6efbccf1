// kvq_decode_window.cu -- the decode kernel's build behind a sliding window with sinks, over caches with one
// scale per KV head (or BF16).
#include "kvq_decode_split.cuh"

namespace kvq {

cudaError_t launch_decode_window(const DecodeArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                                 cudaStream_t stream)
{
    return launch_build<true, false>(a, k_map, v_map, stream);
}

cudaError_t read_window_error(uint32_t *bits, bool clear) { return read_error_word(bits, clear); }

} // namespace kvq
