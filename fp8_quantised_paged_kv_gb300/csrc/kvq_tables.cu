// kvq_tables.cu -- page tables kept on the GPU: rows given pages and slots for
// new tokens (extend), rows that start on another row's pages (fork), and
// pages given back (trim).  No length, count or id reaches the host, so the
// calls can be captured with the step that uses the tables.
//
// The mathematics is a prefix sum over the requests in order.  With h_r pages
// held and d_r more wanted, request r takes places s_r = sum_{i < r} d_i up to
// s_r + d_r of the free list, counted from its top; a request whose places
// pass the list's end gets nothing, and because s does not descend, neither
// does any later one that wants a page.  A row whose partly filled last page has
// other holders wants none and gets nothing.  So who is served, and with which page,
// goes by the tables alone, not by the order in which CTAs run.
//
// What bounds them is latency: a step touches a few kilobytes, a batch of
// prompts a few megabytes (its slots).  Every CTA sums the wants of the
// requests before its own by itself, which is one trip to L2 for up to 256
// requests and spares a launch or a grid-wide wait.  Lengths and the list's
// count are changed in place, so the CTA that finishes last changes them, when
// nobody reads them any more; a call that one CTA can do has no such tail.
// Trim counts down with atomics, whose order does not matter to the counts,
// and marks pages without holders in a bitmap; the last CTA moves them to the
// list in ascending order.
#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kTrimThreads = 512;
// Entries or tokens of a thread whose loads are under way together: a row's loop
// is a chain of trips to L2 otherwise (60 rows of up to 1,711 entries forked,
// extended by a token and trimmed: 21.6 us one at a time).
constexpr int kBatch = 4;
constexpr int64_t kMaxTokens = 0x7FFFFFFF;             // that an int32 length holds, whatever the row's width

__device__ __forceinline__ int pages_of(int64_t tokens, int ps_shift)
{
    return static_cast<int>((tokens + (1 << ps_shift) - 1) >> ps_shift);
}

__device__ __forceinline__ int clamp_count(int count, int num_pages)
{
    return count < 0 ? 0 : count > num_pages ? num_pages : count;
}

// A page taken from place `place` of the free list, counted from its top: its
// tag changes and it has one holder.  (An id outside the pool, which no call of
// this file puts on the list, is handed out as it is.)
__device__ __forceinline__ int take_page(const PoolArgs &p, int count, int place, uint32_t &tag)
{
    const int page = __ldcg(p.free_pages + (count - 1 - place));
    tag = 0;
    if (page >= 0 && page < p.num_pages) {
        p.page_refs[page] = 1;
        if (p.page_tags != nullptr)
            p.page_tags[page] = tag = __ldcg(p.page_tags + page) + 1u;
    }
    return page;
}

// Inclusive sum over the block of one number per thread; *total their sum.
template <int kN, typename T>
__device__ __forceinline__ T block_scan(T v, T *total)
{
    __shared__ T s_warp[kN / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const T o = __shfl_up_sync(0xFFFFFFFFu, v, off);
        v += lane >= off ? o : 0;
    }
    __syncthreads();                         // an earlier scan's sums have been read
    if (lane == 31)
        s_warp[warp] = v;
    __syncthreads();
    T before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kN / 32; ++w) {
        before += w < warp ? s_warp[w] : 0;
        all += s_warp[w];
    }
    *total = all;
    return v + before;
}

// Whether this CTA is the last of the grid to arrive.  The others' writes are
// then visible to it; the counter is left at zero for the next call.
__device__ __forceinline__ bool last_to_arrive(unsigned int *counter, unsigned int ctas)
{
    __shared__ bool s_last;
    __syncthreads();
    if (ctas == 1)
        return true;
    if (threadIdx.x == 0) {
        s_last = atom_add_acq_rel_gpu(counter, 1u) == ctas - 1;
        if (s_last)
            *counter = 0;
    }
    __syncthreads();
    return s_last;
}

// What an extend wants for request r.
struct Want {
    int64_t old, n, off;                     // tokens held, new ones, the first one's place among the call's
    int have, need;                          // pages held, and more
    bool fits;
};
// tail: look whether the row may write its last, partly filled page.  One that
// other rows hold too (kvq_trim_tables can leave it so behind a fork) is not its
// own, and a slot in it would be one of theirs.  (Two more trips to L2 for such
// rows, for their entry and its holders.)
__device__ __forceinline__ Want want_of(const ExtendArgs &a, int r, int ps_shift, bool tail)
{
    Want w;
    w.old = __ldcg(a.seq_lens + r);
    if (a.token_offsets != nullptr) {
        w.off = __ldcg(a.token_offsets + r);
        w.n = static_cast<int64_t>(__ldcg(a.token_offsets + r + 1)) - w.off;
    } else {
        w.n = a.tokens_each;
        w.off = w.n * r;
    }
    w.fits = w.old >= 0 && w.n >= 0 && w.off >= 0 && w.off + w.n <= a.num_tokens &&
             w.old + w.n <= min(static_cast<int64_t>(a.max_pages_per_seq) << ps_shift, kMaxTokens);
    if (tail && w.fits && w.n > 0 && (w.old & ((1 << ps_shift) - 1)) != 0) {
        const int page = __ldcg(a.block_table + static_cast<int64_t>(r) * a.max_pages_per_seq + (w.old >> ps_shift));
        w.fits = page < 0 || page >= a.pool.num_pages || __ldcg(a.pool.page_refs + page) <= 1;
    }
    w.have = w.fits ? pages_of(w.old, ps_shift) : 0;
    w.need = w.fits ? pages_of(w.old + w.n, ps_shift) - w.have : 0;
    return w;
}

// CTA (x, y) serves requests [x m, (x + 1) m), part y of each one's tokens and
// pages; `team` threads work on a request.
__global__ void __launch_bounds__(kThreads) extend_kernel(const ExtendArgs a)
{
    struct Held {
        int64_t old, n, off;
        int have, need, start;
        bool ok;
    };
    __shared__ Held s_held[kThreads];
    grid_dependency_wait();
    grid_launch_dependents();
    const int ps_shift = __ffs(a.pool.page_size) - 1;
    const int count = clamp_count(__ldcg(a.pool.free_count), a.pool.num_pages);
    const int r0 = static_cast<int>(blockIdx.x) * a.per_cta;
    const int m = min(a.per_cta, a.batch - r0);
    // the wants before this CTA's requests, then each of its own, in 64 bits:
    // those that no pool could fill may add up to more than 31
    int64_t mine = 0, base, all;
    Want w = {};
    if (static_cast<int>(threadIdx.x) < m)
        w = want_of(a, r0 + threadIdx.x, ps_shift, true);
    for (int r = threadIdx.x; r < r0; r += kThreads)
        mine += want_of(a, r, ps_shift, true).need;
    block_scan<kThreads>(mine, &base);
    const int64_t upto = base + block_scan<kThreads>(static_cast<int64_t>(w.need), &all);
    if (static_cast<int>(threadIdx.x) < m) {
        const bool ok = w.fits && (w.need == 0 || upto <= count);
        s_held[threadIdx.x] = {w.old, w.n, w.off, w.have, w.need, ok ? static_cast<int>(upto) - w.need : 0, ok};
        if (blockIdx.y == 0)
            a.refused[r0 + threadIdx.x] = ok ? 0 : 1;
    }
    __syncthreads();
    const int teams = kThreads / a.team, team = static_cast<int>(threadIdx.x) / a.team;
    const int step = a.team * static_cast<int>(gridDim.y);
    const int first = static_cast<int>(threadIdx.x) % a.team + a.team * static_cast<int>(blockIdx.y);
    for (int i = team; i < m; i += teams) {
        const Held h = s_held[i];
        int32_t *row = a.block_table + static_cast<int64_t>(r0 + i) * a.max_pages_per_seq;
        uint32_t *tags = a.expected_tags == nullptr
                             ? nullptr : a.expected_tags + static_cast<int64_t>(r0 + i) * a.max_pages_per_seq;
        if (h.ok)
            for (int j = first; j < h.need; j += step) {
                uint32_t tag;
                row[h.have + j] = take_page(a.pool, count, h.start + j, tag);
                if (tags != nullptr)
                    tags[h.have + j] = tag;
            }
        if (a.slot_mapping == nullptr || h.n < 0 || h.off < 0 || h.off + h.n > a.num_tokens)
            continue;
        for (int64_t t0 = first; t0 < h.n; t0 += kBatch * step) {
            int page[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int64_t t = t0 + k * step;
                const int at = static_cast<int>((h.old + t) >> ps_shift);
                page[k] = -1;
                if (h.ok && t < h.n)
                    page[k] = at < h.have ? __ldcg(row + at)
                                          : __ldcg(a.pool.free_pages + (count - 1 - h.start - (at - h.have)));
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int64_t t = t0 + k * step;
                if (t < h.n)
                    a.slot_mapping[h.off + t] =
                        h.ok ? (static_cast<int64_t>(page[k]) << ps_shift) + ((h.old + t) & ((1 << ps_shift) - 1)) : -1;
            }
        }
    }
    // the lengths and the list's count, when no CTA reads them any more
    if (!last_to_arrive(a.pool.scratch, gridDim.x * gridDim.y))
        return;
    int taken = 0, total;
    for (int r = threadIdx.x; r < a.batch; r += kThreads) {
        const Want v = want_of(a, r, ps_shift, false);
        if (__ldcg(a.refused + r) == 0) {
            taken += v.need;
            a.seq_lens[r] = static_cast<int32_t>(v.old + v.n);
        }
    }
    block_scan<kThreads>(taken, &total);
    if (threadIdx.x == 0 && total > 0)
        *a.pool.free_count = count - total;
}

// What request r's fork wants; the parent is another row, which holds the tokens.
struct Fork {
    int parent, len;
    bool asked, fits, part;                  // part: a page of its own for the tokens past the whole pages
};
__device__ __forceinline__ Fork fork_of(const ForkArgs &a, int r, int ps_shift)
{
    Fork f;
    f.parent = __ldcg(a.parents + r);
    f.len = __ldcg(a.fork_lens + r);
    f.asked = f.parent >= 0;
    f.fits = f.asked && f.parent < a.batch && f.parent != r && __ldcg(a.seq_lens + r) == 0 && f.len >= 0;
    if (f.fits) {
        const int held = __ldcg(a.seq_lens + f.parent);
        f.fits = f.len <= held && held <= static_cast<int64_t>(a.max_pages_per_seq) << ps_shift;
    }
    f.part = f.fits && (f.len & ((1 << ps_shift) - 1)) != 0;
    return f;
}

__global__ void __launch_bounds__(kThreads) fork_kernel(const ForkArgs a)
{
    struct Held {
        int parent, len, place;
        bool ok, part;
    };
    __shared__ Held s_held[kThreads];
    grid_dependency_wait();
    grid_launch_dependents();
    const int ps_shift = __ffs(a.pool.page_size) - 1;
    const int count = clamp_count(__ldcg(a.pool.free_count), a.pool.num_pages);
    const int r0 = static_cast<int>(blockIdx.x) * a.per_cta;
    const int m = min(a.per_cta, a.batch - r0);
    int mine = 0;
    for (int r = threadIdx.x; r < r0; r += kThreads)
        mine += fork_of(a, r, ps_shift).part;
    int base, all;
    block_scan<kThreads>(mine, &base);
    Fork f = {};
    if (static_cast<int>(threadIdx.x) < m)
        f = fork_of(a, r0 + threadIdx.x, ps_shift);
    const int upto = base + block_scan<kThreads>(static_cast<int>(f.part), &all);
    if (static_cast<int>(threadIdx.x) < m) {
        const bool ok = f.fits && (!f.part || upto <= count);
        s_held[threadIdx.x] = {f.parent, f.len, upto - 1, ok, f.part};
        const int r = r0 + threadIdx.x;
        a.refused[r] = f.asked && !ok ? 1 : 0;
        if (!ok || !f.part)
            a.src_pages[r] = a.dst_pages[r] = -1;
    }
    __syncthreads();
    for (int i = 0; i < m; ++i) {
        const Held h = s_held[i];
        if (!h.ok)
            continue;
        const int64_t to = static_cast<int64_t>(r0 + i) * a.max_pages_per_seq;
        const int64_t from = static_cast<int64_t>(h.parent) * a.max_pages_per_seq;
        const int whole = h.len >> ps_shift;
        for (int j0 = threadIdx.x; j0 < whole; j0 += kBatch * kThreads) {
            int page[kBatch];
            uint32_t tag[kBatch] = {};
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int j = j0 + k * kThreads;
                page[k] = j < whole ? __ldcg(a.block_table + from + j) : -1;
                if (a.expected_tags != nullptr && j < whole)
                    tag[k] = __ldcg(a.expected_tags + from + j);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int j = j0 + k * kThreads;
                if (j >= whole)
                    break;
                a.block_table[to + j] = page[k];
                if (page[k] >= 0 && page[k] < a.pool.num_pages)
                    atomicAdd(a.pool.page_refs + page[k], 1);
                if (a.expected_tags != nullptr)
                    a.expected_tags[to + j] = tag[k];
            }
        }
        if (h.part && threadIdx.x == kThreads - 1) {
            uint32_t tag;
            const int page = take_page(a.pool, count, h.place, tag);
            a.block_table[to + whole] = page;
            if (a.expected_tags != nullptr)
                a.expected_tags[to + whole] = tag;
            a.src_pages[r0 + i] = __ldcg(a.block_table + from + whole);
            a.dst_pages[r0 + i] = page;
        }
    }
    if (!last_to_arrive(a.pool.scratch, gridDim.x))
        return;
    int taken = 0;
    for (int at = 0; at < a.batch; at += kThreads) {
        const int r = at + static_cast<int>(threadIdx.x);
        if (r < a.batch && __ldcg(a.parents + r) >= 0 && __ldcg(a.refused + r) == 0) {
            const int len = __ldcg(a.fork_lens + r);
            taken += (len & ((1 << ps_shift) - 1)) != 0;
            a.seq_lens[r] = len;
        }
    }
    int total;
    block_scan<kThreads>(taken, &total);
    if (threadIdx.x == 0 && total > 0)
        *a.pool.free_count = count - total;
}

// One CTA per row; scratch: the arrival counter, whether any page is marked,
// and from word 64 on the bitmap of pages that nobody holds any more.
__global__ void __launch_bounds__(kTrimThreads) trim_kernel(const TrimArgs a)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int ps_shift = __ffs(a.pool.page_size) - 1;
    uint32_t *marked = a.pool.scratch + 1, *bitmap = a.pool.scratch + kPoolBitmapWord;
    const int64_t r = blockIdx.x;
    const int64_t cap = static_cast<int64_t>(a.max_pages_per_seq) << ps_shift;
    const int64_t held = min(static_cast<int64_t>(__ldcg(a.seq_lens + r)), cap);
    const int64_t keep = __ldcg(a.keep_lens + r);
    if (keep >= 0 && keep < held) {
        int32_t *row = a.block_table + r * a.max_pages_per_seq;
        const int end = pages_of(held, ps_shift);
        bool any = false;
        for (int j0 = pages_of(keep, ps_shift) + static_cast<int>(threadIdx.x); j0 < end; j0 += kBatch * kTrimThreads) {
            int page[kBatch], had[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                page[k] = j0 + k * kTrimThreads < end ? __ldcg(row + j0 + k * kTrimThreads) : -1;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                had[k] = 2;
                if (page[k] >= 0 && page[k] < a.pool.num_pages)
                    had[k] = atomicSub(a.pool.page_refs + page[k], 1);
                if (j0 + k * kTrimThreads < end)
                    row[j0 + k * kTrimThreads] = -1;
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (had[k] == 1) {
                    atomicOr(bitmap + (page[k] >> 5), 1u << (page[k] & 31));
                    any = true;
                } else if (had[k] <= 0) {    // free already: a row that named it more often than it held it
                    atomicAdd(a.pool.page_refs + page[k], 1);
                }
        }
        if (any)
            atomicOr(marked, 1u);
        __syncthreads();                     // every thread has read the length
        if (threadIdx.x == 0)
            a.seq_lens[r] = static_cast<int32_t>(keep);
    }
    if (!last_to_arrive(a.pool.scratch, gridDim.x))
        return;
    if (__ldcg(marked) == 0)
        return;
    // Marked pages, in ascending order, onto the list.  A pass takes four words of
    // the bitmap a thread; a warp then writes a word's pages at a time, a lane each
    // (a thread's own 128 places, one after the other, took 25 us for 65,000 pages).
    constexpr int kWords = 4 * kTrimThreads;
    __shared__ uint32_t s_bits[kWords];
    __shared__ int s_place[kWords];
    int count = clamp_count(__ldcg(a.pool.free_count), a.pool.num_pages);
    const int words = static_cast<int>((static_cast<int64_t>(a.pool.num_pages) + 31) / 32);
    for (int w0 = 0; w0 < words; w0 += kWords) {
        uint32_t bits[4];
        int n = 0;
        const int at = 4 * static_cast<int>(threadIdx.x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            bits[k] = w0 + at + k < words ? __ldcg(bitmap + w0 + at + k) : 0u;
            n += __popc(bits[k]);
        }
        int total;
        int place = count + block_scan<kTrimThreads>(n, &total) - n;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (bits[k] != 0)
                bitmap[w0 + at + k] = 0;
            s_bits[at + k] = bits[k];
            s_place[at + k] = place;
            place += __popc(bits[k]);
        }
        __syncthreads();
        if (total > 0) {
            const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
            for (int w = warp; w < min(kWords, words - w0); w += kTrimThreads / 32) {
                const uint32_t b = s_bits[w];
                const int to = s_place[w] + __popc(b & ((1u << lane) - 1u));
                if ((b >> lane & 1u) != 0 && to < a.pool.num_pages)
                    a.pool.free_pages[to] = 32 * (w0 + w) + lane;
            }
        }
        count += total;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        *marked = 0;
        *a.pool.free_count = clamp_count(count, a.pool.num_pages);
    }
}

template <typename Args>
cudaError_t launch_tables(void (*kernel)(Args), const Args &a, dim3 grid, int threads, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// Requests per CTA, at most a thread each, so that two CTAs per SM hold the batch.
int requests_per_cta(int batch)
{
    const int ctas = 2 * device_sm_count();
    const int per = (batch + ctas - 1) / ctas;
    return per < kThreads ? per : kThreads;
}

} // namespace

cudaError_t launch_extend_tables(ExtendArgs a, cudaStream_t stream)
{
    if (a.batch == 0)
        return cudaSuccess;
    const int64_t each = a.num_tokens / a.batch;
    // threads on a request: one in a decode step, a warp for a few tokens, else all
    a.team = each <= 2 ? 1 : each <= 64 ? 32 : kThreads;
    // what a single CTA does in one or two passes needs no arrival of others
    if (a.batch <= kThreads && static_cast<int64_t>(a.batch) * a.team <= 2 * kThreads)
        a.per_cta = a.batch;
    else
        a.per_cta = requests_per_cta(a.batch);
    const int x = (a.batch + a.per_cta - 1) / a.per_cta;
    int64_t parts = a.team < kThreads ? 1 : each / 1024;
    const int64_t room = 6 * device_sm_count() / x;
    parts = parts < room ? parts : room;
    return launch_tables(extend_kernel, a, dim3(static_cast<unsigned>(x), static_cast<unsigned>(parts > 1 ? parts : 1)),
                         kThreads, stream);
}

cudaError_t launch_fork_tables(ForkArgs a, cudaStream_t stream)
{
    if (a.batch == 0)
        return cudaSuccess;
    a.per_cta = requests_per_cta(a.batch);
    return launch_tables(fork_kernel, a, dim3(static_cast<unsigned>((a.batch + a.per_cta - 1) / a.per_cta)), kThreads,
                         stream);
}

cudaError_t launch_trim_tables(const TrimArgs &a, cudaStream_t stream)
{
    if (a.batch == 0)
        return cudaSuccess;
    return launch_tables(trim_kernel, a, dim3(static_cast<unsigned>(a.batch)), kTrimThreads, stream);
}

} // namespace kvq
