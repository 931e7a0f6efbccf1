// kvq_tag_check.cu -- the separate batched KV-cache integrity pass.
//
// Every physical page carries a tag that changes whenever the page is
// reassigned; each request records the tag it expects for each of its
// pages; before decode reads the cache the check compares the two and aborts
// the request on any mismatch.  It runs as its own batched pass rather than
// inside the attention kernel, so no attention thread group races with it
// (blog post "Smaller, faster, safer", page-2 mirror section "KV Cache
// 完整性检查"; page-3 mirror section "一个不能出错的共享缓存").
//
// One CTA per request: its 512 threads take the ceil(L / page_size) entries
// the request uses, 4,096 per pass, issuing every block-table and
// expected-tag load of the pass before the live-tag gathers, so a pass costs
// two rounds of dependent loads; OR-reduce with __syncthreads_or; thread 0
// writes the flag (0 or 1).
#include "kvq_rowops.cuh"

namespace kvq {
namespace {

constexpr int kTagThreads = 512;

#ifdef KVQ_PHASE_STAMPS
// Instrumented build only: %globaltimer at entry (point 0) and when the flag
// is written (1) by thread 0 of every CTA of the last launch.
constexpr int kTagStampCtas = 4096;
__device__ unsigned long long g_tag_stamps[kTagStampCtas * 2];
__device__ __forceinline__ void tag_stamp(int point)
{
    if (threadIdx.x == 0 && blockIdx.x < kTagStampCtas)
        g_tag_stamps[blockIdx.x * 2 + point] = global_timer_ns();
}
#define KVQ_TAG_STAMP(p) tag_stamp(p)
#else
#define KVQ_TAG_STAMP(p) ((void)0)
#endif

__global__ void __launch_bounds__(kTagThreads) tag_check_kernel(TagCheckArgs a)
{
    KVQ_TAG_STAMP(0);
    grid_launch_dependents();              // a dependent decode launch may begin now
    const int64_t r = blockIdx.x;
    const bool bad = tag_check_request<8>(a.block_table, a.expected_tags, a.seq_lens, a.page_tags,
                                          a.max_pages_per_seq, a.page_size, a.num_pages, r);
    if (threadIdx.x == 0)
        a.abort_flags[r] = bad ? 1 : 0;
    KVQ_TAG_STAMP(1);
}

// The check of a request that holds only the pages a window shows: the entries
// of the sinks' pages, then those from the page where the window of the
// request's first new token starts.  The entries between are not read (their
// pages may have been given back).  The visible entries are numbered in one
// run, so a pass takes 2,048 of them whatever the hole; unlike the check of
// every entry it needs the length before its first table load (three rounds
// of dependent loads, and two more for each further pass).
constexpr int kWindowUnroll = 4;
__global__ void __launch_bounds__(kTagThreads) tag_check_window_kernel(const TagWindowArgs w)
{
    grid_launch_dependents();              // a dependent decode launch may begin now
    const TagCheckArgs &a = w.t;
    const int64_t r = blockIdx.x;
    const int32_t *bt = a.block_table + r * a.max_pages_per_seq;
    const uint32_t *exp = a.expected_tags + r * a.max_pages_per_seq;
    const int32_t seq = a.seq_lens[r];
    const int64_t len = seq > 0 ? seq : 0;
    int64_t used = (len + a.page_size - 1) / a.page_size;
    bool bad = used > a.max_pages_per_seq;
    if (bad)
        used = a.max_pages_per_seq;
    int64_t sink_pages = used, hole = 0;                   // window 0: every entry
    if (w.window > 0) {
        const int64_t w0 = max(len - w.num_query_tokens + 1 - w.window, static_cast<int64_t>(0));
        sink_pages = (min(len, static_cast<int64_t>(w.num_sinks)) + a.page_size - 1) / a.page_size;
        hole = max(w0 / a.page_size - sink_pages, static_cast<int64_t>(0));
    }
    const int64_t seen = used - hole;
    for (int64_t base = 0; base < seen; base += kTagThreads * kWindowUnroll) {
        int32_t p[kWindowUnroll];
        uint32_t want[kWindowUnroll], live[kWindowUnroll];
        bool look[kWindowUnroll];
#pragma unroll
        for (int k = 0; k < kWindowUnroll; ++k) {
            const int64_t v = base + k * kTagThreads + threadIdx.x;
            const int64_t i = v < sink_pages ? v : v + hole;
            look[k] = v < seen;
            p[k] = look[k] ? __ldg(bt + i) : 0;
            want[k] = look[k] ? __ldg(exp + i) : 0u;
        }
#pragma unroll
        for (int k = 0; k < kWindowUnroll; ++k)
            live[k] = look[k] && p[k] >= 0 && p[k] < a.num_pages ? __ldg(a.page_tags + p[k]) : 0u;
#pragma unroll
        for (int k = 0; k < kWindowUnroll; ++k)
            bad |= look[k] && (p[k] < 0 || p[k] >= a.num_pages || live[k] != want[k]);
    }
    const bool any = __syncthreads_or(bad) != 0;
    if (threadIdx.x == 0)
        a.abort_flags[r] = any ? 1 : 0;
}

} // namespace

cudaError_t launch_tag_check_window(const TagWindowArgs &a, cudaStream_t stream)
{
    if (a.t.batch == 0)
        return cudaSuccess;
    tag_check_window_kernel<<<static_cast<unsigned>(a.t.batch), kTagThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_tag_check(const TagCheckArgs &a, cudaStream_t stream)
{
    if (a.batch == 0)
        return cudaSuccess;
    tag_check_kernel<<<static_cast<unsigned>(a.batch), kTagThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

#ifdef KVQ_PHASE_STAMPS
cudaError_t read_tag_stamps(unsigned long long *host, size_t count)
{
    const size_t n = count < static_cast<size_t>(kTagStampCtas * 2) ? count : kTagStampCtas * 2;
    return cudaMemcpyFromSymbol(host, g_tag_stamps, n * sizeof(unsigned long long));
}
#endif

} // namespace kvq
