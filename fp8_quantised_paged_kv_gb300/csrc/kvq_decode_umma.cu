// kvq_decode_umma.cu -- the tensor-memory kernel's build for caches with one
// scale per KV head, every token visible.
#include "kvq_decode_umma.cuh"

namespace kvq {

cudaError_t launch_decode_umma(const DecodeArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                               cudaStream_t stream)
{
    return launch_umma_build<false, false>(a, k_map, v_map, stream);
}

int decode_umma_ctas_per_sm()
{
    return 1;                                              // its shared memory takes most of an SM
}

cudaError_t read_umma_error(uint32_t *bits, bool clear) { return read_umma_error_word(bits, clear); }

} // namespace kvq
