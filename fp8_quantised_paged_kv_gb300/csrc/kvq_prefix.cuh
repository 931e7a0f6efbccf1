// kvq_prefix.cuh -- what a request of a call over shared prefixes shares.
#pragma once

#include "kvq_ptx.cuh"
#include "kvq_view.cuh"

namespace kvq {

// Load and store that order what this thread reads after, or wrote and saw
// before, at GPU scope.
__device__ __forceinline__ int ld_acquire_gpu(const int *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void st_release_gpu(int *p, int v)
{
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// What this thread has come to see in global memory, before bulk copies that
// it issues from here on.
__device__ __forceinline__ void fence_proxy_async_global()
{
    asm volatile("fence.proxy.async.global;" ::: "memory");
}

// What 64 tokens of a KV head cost, in 1/140 us of an SM, as measured in each
// build: shared ones up to 128 query rows; a request's own, in the mma.sync kernel,
// per 16 rows (0.36 us, over a bf16 cache 0.86).  A further request's rows cost
// 11/16 of their share of the former.  Shared ones over a bf16 cache with fp32 output take
// 1.47 us alone and count as 2.3, what they cost beside the own ones, whose copies
// they wait for: 18 batches of 12 to 128 requests behind 1 to 16 prompts of 2,000 to
// 14,000 tokens took 62.8 us so, in the geometric mean, and 67.8 with 1.47 (from 10 %
// less, 30 requests of two query tokens behind three prompts, to 20 % more).
struct Costs {
    int tile, join, own;
    __device__ __forceinline__ explicit Costs(const PrefixArgs &a)
    {
        tile = a.bf16_cache ? (a.out_fp32 ? 320 : 137)
               : a.k_exp != nullptr ? (a.out_fp32 ? 197 : 138) : (a.out_fp32 ? 185 : 128);
        join = (tile * min(a.n_query * a.group, 128) * 11 / 16 + 127) / 128;
        own = (a.bf16_cache ? 120 : 50) * a.row_blocks;
    }
};

// A request's tokens by where they come from: whole pages, in whole 64 tokens, of row
// prefix_of[r], as many as all its query tokens see and the other row holds, and its own row
// (both 0: its outputs are zeros).  The other row serves only where so many
// consecutive requests (up to eight are counted) name it that this costs less, by Costs, than
// each reading its own.  With one query token: over e4m3 three (block scales four from
// seven heads a group on), with fp32 output four (five from five heads on, and with block
// scales); over a bf16 cache two, with fp32 output three.
// `joins`: the request before it names the same row.  (Through L2: whatever wrote
// the numbers may have run on this SM beside this CTA.)
struct Tokens {
    int shared, own, lead;
    bool joins;
};
__device__ __forceinline__ Tokens tokens_of(const PrefixArgs &a, int r, int ps_shift)
{
    constexpr int kLook = 8;
    const int lead = __ldcg(a.prefix_of + r), want = __ldcg(a.prefix_lens + r);
    int before[kLook - 1], after[kLook - 1];
#pragma unroll
    for (int i = 0; i < kLook - 1; ++i) {
        before[i] = r - 1 - i >= 0 ? __ldcg(a.prefix_of + r - 1 - i) : -1;
        after[i] = r + 1 + i < a.batch ? __ldcg(a.prefix_of + r + 1 + i) : -1;
    }
    const int64_t cap = static_cast<int64_t>(a.max_pages_per_seq) << ps_shift;
    const int real = __ldcg(a.seq_lens + r);
    const bool aborted = a.abort_flags != nullptr && __ldcg(a.abort_flags + r) != 0;
    const bool joins = before[0] == lead;
    if (real <= 0 || real > cap || aborted)
        return {0, 0, -1, joins};
    if (lead < 0 || lead >= a.batch || want <= 0)
        return {0, real, -1, joins};
    int together = 1;
    bool left = true, right = true;
#pragma unroll
    for (int i = 0; i < kLook - 1; ++i) {
        left = left && before[i] == lead;
        right = right && after[i] == lead;
        together += left + right;
    }
    together = min(together, kLook);
    const Costs c(a);
    if (together * c.own <= c.tile + (together - 1) * c.join)
        return {0, real, -1, joins};
    const int held = __ldcg(a.seq_lens + lead);
    if (held > cap || (a.abort_flags != nullptr && __ldcg(a.abort_flags + lead) != 0))
        return {0, real, -1, joins};
    const int n = min(min(want, held), real - a.n_query + 1);
    const int whole = max(ps_shift, 6);                    // (of tiles, too: kvq_prefix.cu)
    const int shared = n > 0 ? n >> whole << whole : 0;
    return {shared, real - shared, shared > 0 ? lead : -1, joins};
}

// How the SMs are divided between the kernel over the shared pages and the one
// over the requests' own, which runs beside it: in proportion to an estimate of
// their work that both make from the lengths (384 tokens are added to each pair of
// request and KV head).
struct Work {
    long long shared, own;
    __device__ __forceinline__ void add(const PrefixArgs &a, const Tokens &t)
    {
        const Costs c(a);
        shared += static_cast<long long>((t.shared + 63) / 64) * a.num_kv_heads * (t.joins ? c.join : c.tile);
        if (t.own > 0)
            own += static_cast<long long>((t.own + 63) / 64 + 6) * a.num_kv_heads * c.own;
    }
    // SMs for the shared pages
    __device__ __forceinline__ int sms(int all) const
    {
        if (shared == 0 || own == 0)
            return shared == 0 ? 0 : all;
        const int few = max(all / 38, 1);                  // what either gets at least
        const double part = static_cast<double>(shared) / static_cast<double>(shared + own);
        return min(max(static_cast<int>(part * all + 0.5), few), max(all - few, 1));
    }
};

// What decode_split_kernel asks of a call: the shared tokens, counted into its
// work; the shortened context that the own row adds (past the shared pages,
// which are a hole); the SMs that are its own.  Calls without sharing have none
// of it.
__device__ __forceinline__ int shared_tokens(const PrefixArgs &a, int r, int ps_shift, Work &w)
{
    const Tokens t = tokens_of(a, r, ps_shift);
    w.add(a, t);
    if (blockIdx.x == 0)                                   // for the combine
        a.kinds[r] = static_cast<uint8_t>((t.shared > 0 ? kSharedPart : 0) | (t.own > 0 ? kOwnPart : 0));
    return t.shared;
}
__device__ __forceinline__ int shared_tokens(const ViewArgs &, int, int, Work &) { return 0; }
__device__ __forceinline__ Shown own_context(const PrefixArgs &, int64_t real, int64_t shared, int ps_shift)
{
    return {real - shared, 0, shared >> ps_shift, 0};
}
__device__ __forceinline__ Shown own_context(const ViewArgs &a, int64_t real, int64_t, int ps_shift)
{
    return shown_context(a, real, ps_shift);
}
__device__ __forceinline__ int own_ctas(const PrefixArgs &a, const Work &w)
{
    const int left = a.pre_ctas - w.sms(a.pre_ctas);
    const int ctas = left > 0 ? a.resident_ctas / a.pre_ctas * left : a.resident_ctas;
    if (blockIdx.x == 0 && threadIdx.x == 0)
        st_release_gpu(a.own_takers, ctas);
    return ctas;
}
__device__ __forceinline__ int own_ctas(const ViewArgs &a, const Work &) { return a.resident_ctas; }
// Whether CTA 0 has found out that this one has nothing to do: the CTAs that find
// room only when the shared pages are done leave at once.  (Acquires what was
// written before the call: decode_split_kernel.)
__device__ __forceinline__ bool nothing_left(const PrefixArgs &a)
{
    const int takers = ld_acquire_gpu(a.own_takers);
    return takers > 0 && static_cast<int>(blockIdx.x) >= takers;
}
__device__ __forceinline__ bool nothing_left(const ViewArgs &) { return false; }

} // namespace kvq
