// kvq_view.cuh -- what a windowed call sees of a request's context.
#pragma once

#include "kvq_internal.h"

namespace kvq {

// The context a windowed call shows of a request of `real` tokens, without
// the hole between the sinks' pages and the page where the first query's
// window starts: its length, the sinks' pages, the hole's pages, and the
// window's start, which like every position counts the shortened context.
struct Shown {
    int64_t len, sink_pages, hole, win0;
};
__device__ __forceinline__ Shown shown_context(const ViewArgs &a, int64_t real, int ps_shift)
{
    Shown v = {real, 0, 0, 0};
    if (a.window > 0) {
        const int64_t start = real - a.n_query + 1 - a.window;
        const int64_t ps = static_cast<int64_t>(1) << ps_shift;
        v.sink_pages = (min(real, static_cast<int64_t>(a.num_sinks)) + ps - 1) >> ps_shift;
        v.hole = max((max(start, static_cast<int64_t>(0)) >> ps_shift) - v.sink_pages, static_cast<int64_t>(0));
        v.len = real - (v.hole << ps_shift);
        v.win0 = start - (v.hole << ps_shift);
    }
    return v;
}

} // namespace kvq
