// kvq_decode_blocks.cu -- the decode kernel's build over the block-scaled cache (a power-of-two exponent per 16
// tokens and KV head), with or without a window.
#include "kvq_decode_split.cuh"

namespace kvq {

cudaError_t launch_decode_blocks(const ViewArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                                 cudaStream_t stream)
{
    const cudaError_t e = launch_build<true, true>(a, k_map, v_map, stream);
    return e != cudaSuccess || !a.combine_apart ? e : launch_combine_rows(a, stream);
}

cudaError_t read_blocks_error(uint32_t *bits, bool clear) { return read_error_word(bits, clear); }

} // namespace kvq
