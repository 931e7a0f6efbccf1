// kvq_decode_umma_view.cu -- the tensor-memory kernel's builds with a window, and
// for the block-scaled cache (a window or none).
#include "kvq_decode_umma.cuh"

namespace kvq {

cudaError_t launch_decode_umma_view(const DecodeArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                                    cudaStream_t stream)
{
    return a.k_exp != nullptr ? launch_umma_build<true, true>(a, k_map, v_map, stream)
                              : launch_umma_build<true, false>(a, k_map, v_map, stream);
}

cudaError_t read_umma_view_error(uint32_t *bits, bool clear) { return read_umma_error_word(bits, clear); }

} // namespace kvq
