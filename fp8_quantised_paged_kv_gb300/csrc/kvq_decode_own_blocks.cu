// kvq_decode_own_blocks.cu -- the decode kernel's build past the pages that requests share, over the block-scaled
// cache.
#define KVQ_OWN_ROWS
#include "kvq_decode_split.cuh"

namespace kvq {

cudaError_t launch_decode_own_blocks(const PrefixArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                                     cudaStream_t stream)
{
    return a.n_query > 1 ? launch_variant<true, true, false, true>(a, k_map, v_map, stream)
                         : launch_variant<true, true, false, false>(a, k_map, v_map, stream);
}

cudaError_t read_own_blocks_error(uint32_t *bits, bool clear) { return read_error_word(bits, clear); }

} // namespace kvq
