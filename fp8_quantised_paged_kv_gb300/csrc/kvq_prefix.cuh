// kvq_prefix.cuh -- what a request of a call over shared prefixes shares.
#pragma once

#include "kvq_ptx.cuh"
#include "kvq_view.cuh"

namespace kvq {

// Tokens of request r's context that come from the pages of row prefix_of[r]: as many
// whole pages as all its query tokens see and the other row holds.  0: none,
// its own row has everything.  (Through L2: whatever wrote the numbers may
// have run on this SM beside this CTA.)
__device__ __forceinline__ int shared_tokens(const PrefixArgs &a, int r, int ps_shift)
{
    const int lead = __ldcg(a.prefix_of + r), want = __ldcg(a.prefix_lens + r);
    const int64_t cap = static_cast<int64_t>(a.max_pages_per_seq) << ps_shift;
    const int real = __ldcg(a.seq_lens + r);
    const bool aborted = a.abort_flags != nullptr && __ldcg(a.abort_flags + r) != 0;
    if (lead < 0 || lead >= a.batch || want <= 0 || real <= 0 || real > cap || aborted)
        return 0;
    const int held = __ldcg(a.seq_lens + lead);
    if (held > cap || (a.abort_flags != nullptr && __ldcg(a.abort_flags + lead) != 0))
        return 0;
    const int n = min(min(want, held), real - a.n_query + 1);
    return n > 0 ? n >> ps_shift << ps_shift : 0;
}

// The shortened context that the request's own row adds: what is past the
// shared pages.
__device__ __forceinline__ Shown own_context(const PrefixArgs &, int64_t real, int64_t shared, int ps_shift)
{
    return {real - shared, 0, shared >> ps_shift, 0};
}

// The other calls share nothing.
__device__ __forceinline__ int shared_tokens(const ViewArgs &, int, int) { return 0; }
__device__ __forceinline__ Shown own_context(const ViewArgs &a, int64_t real, int64_t, int ps_shift)
{
    return shown_context(a, real, ps_shift);
}

} // namespace kvq
