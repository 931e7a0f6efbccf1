// kvq_prefix.cu -- attention over pages that several requests share, once for
// all of them, on the 5th-generation tensor cores.
//
// Consecutive requests whose shared tokens come from one row of the table (a
// run) put the query rows of a KV head together: m requests of n tokens and g
// heads are m n g rows over the same K and V, and
//   s = q K^T,  o = sum_j 2^(s_j - M) V_j / l,  l = sum_j 2^(s_j - M)
// (scores in log2 units, M a running maximum) is a product of matrices again.
// What each request's own pages add, kvq_decode_own.cu computes;
// combine_prefix_kernel below joins the parts by their log-sum-exps.
//
// A CTA takes up to 256 rows, two tiles of 128, through a range of the run's
// pages, 64 tokens at a time.  Its warps have one job each: copies by TMA; over an
// FP8 cache the conversion of K and V to f16 (once for all rows); per row tile a
// thread that issues S = Q K^T and O += P V, and a softmax group of four warps, a row per thread, which reads S from tensor
// memory, and writes P over it.  One tile's exponentials run beside the other's
// products, and each group has the next tile's S while it works on one.  With
// up to 128 rows both groups serve the same rows on alternate token tiles, and
// their results are two parts.  Tensor memory is full: four S of 64 columns and
// two accumulators of 128; so Q is read from shared memory.
//
// Block scales mean what they mean in kvq_decode_split.cuh: ek on the scores,
// ev in the exponent with 2^-ev undone in l.  Over an FP8 cache P is kept 2^7
// larger, so that f16 cuts weights at 2^-32 of the largest; the maximum may lag
// by 2^8 before O is rescaled.  Over a bf16 cache P is bf16 and kept 2^-8 times
// as large, at most 1, so that large values do not overflow sums.
//
// How the work is shared out is decided on the device, as in
// kvq_decode_split.cuh: one line of places, run after run, KV head after KV
// head, row pair after row pair; CTA c takes an equal stretch of it.
#include "kvq_decode_umma.cuh"
#include "kvq_prefix.cuh"

namespace kvq {
namespace {

enum CacheKind { kFp8, kBlocksFp8, kBf16 };

constexpr int kTok = 64;                                   // tokens of a tile
constexpr int kHalfBytes = kTok * 256;                     // K or V of a tile, 16-bit
constexpr int kSliceBytes = kTok * 128;                    // 64 dims of it
constexpr int kQBytes = 128 * 256;                         // 128 rows as 16-bit values
constexpr int kRingStage = kTok * 128;                     // a stage of the e4m3 ring: K, or V, of a tile
// Two row tiles' Q leave room for eleven stages; with one tile the ring has
// the place of the second Q as well.
constexpr int kWideStages = 11, kNarrowStages = 15;
constexpr int kOffQ = 0, kOffQ2 = kQBytes;
constexpr int kOffRingNarrow = kOffQ2, kOffRingWide = kOffQ2 + kQBytes;
constexpr int kOffRingEnd = kOffRingWide + kWideStages * kRingStage;
static_assert(kOffRingNarrow + kNarrowStages * kRingStage == kOffRingEnd, "both rings end where the buffers start");
constexpr int kData = kOffRingEnd + 2 * 2 * kHalfBytes;
constexpr int kStageStride = 132;                          // floats of a row on its way out
static_assert(256 * kStageStride * 4 <= kData, "every row has room");

// The most that differs between the builds.
template <int kKind, bool kPrecise>
struct Build {
    static constexpr bool kConvert = kKind != kBf16, kBlocks = kKind == kBlocksFp8;
    // 16-bit terms of a weight: one for bf16 output (f16 2^-11; over a bf16 cache
    // bf16 2^-8, which puts 1.6e-3 of their norm on outputs whose own rounding is
    // 1.7e-3; the other builds round so too, kvq_decode_split_body.cuh); for fp32
    // output two of f16 (2^-22) or three of bf16 (2^-24)
    static constexpr int kTerms = !kPrecise ? 1 : kConvert ? 2 : 3;
    // S buffers per group, of 64 columns; three terms of P need the place of both
    static constexpr int kSBufs = kTerms == 3 ? 1 : 2;
    // Tiles whose K and V are in 16-bit buffers at a time, converted or as the
    // copies bring them.  An even number: with two groups on alternate tiles a
    // buffer is then one group's alone.
    static constexpr int kSlots = kConvert ? 2 : 4;
    static constexpr int kOffBufs = kConvert ? kOffRingEnd : kOffQ2 + kQBytes;
    static_assert(kOffBufs + 2 * kSlots * kHalfBytes <= kData);
    static constexpr int kCopy = kConvert ? 16 : 8;        // the copying warp; before it eight converting ones
    static constexpr int kIssue = kCopy + 1;               // two issuing warps, one per group
    // With converters whole warpgroups, which divide the launch's registers
    // (640 x 96) otherwise: 136 for the softmax, 72 for the converters, 56 for the rest.
    static constexpr int kThreads = kConvert ? 640 : 32 * (kIssue + 2);
    // places of a tile of tokens for one row tile (0.91 us against 1.20 for two over
    // e4m3, 0.99 against 1.60 with block scales, 0.98 against 1.03 over a bf16 cache;
    // fp32 output 1.21 against 1.82, 1.45 against 2.28, 1.47 against 2.61)
    static constexpr int kNarrowCost = kKind == kBf16 ? (kPrecise ? 4 : 7) : kKind == kFp8 ? 6 : 5;
    // and of a border between two jobs: 6 to 8 us (a place is 0.15 to 0.2 us, with three
    // terms 0.37; there 40 places took 1.3 % longer over the 18 batches at Costs)
    static constexpr int kBorderCost = kTerms == 3 ? 20 : 40;
    // fp32 output: tiles between O's ways out of tensor memory into fp32 sums that
    // round.  The tensor core cuts each addition to a large accumulator towards zero, 4
    // kTerms of them a tile: 11 tiles over a bf16 cache put 2.8e-6 on the outputs, 6 of them
    // 1.2e-6 to 1.5e-6, 4 of them 1.05e-6 (2 to 10 % slower); 8 over e4m3 1.1e-6 to 1.2e-6,
    // 16 1.4e-6 to 2.0e-6; 16 with block scales 0.4e-6 to 0.5e-6.
    static constexpr int kFlush = kKind == kBf16 ? 6 : kKind == kFp8 ? 8 : 16;
    static constexpr float kLift = kConvert ? 7.f : -8.f;  // log2 of what P, l and O are larger by
};

constexpr int kBlockReq = 128;                             // a run does not cross a multiple of it
constexpr int kMaxBlocks = 512;                            // of up to 65,535 requests
constexpr int kMinTiles = 4;                               // of a CTA's share, in wide tiles
constexpr int kWideCost = 8;                               // places of a tile of tokens for two row tiles

constexpr uint32_t kColS = 0, kColO = 256;                 // + 128 for the second group

// Column, from its S buffer's first, of term t of P for tokens 32 c .. 32 c + 31
// of a tile.  P is written over scores that have been read.
template <int kTerms>
__device__ __forceinline__ uint32_t p_column(int c, int t)
{
    if constexpr (kTerms < 3)
        return 32u * c + 16u * t;
    else
        return 48u * c + 16u * t;
}

struct Run {
    int first, count, lead, tiles;                         // requests, the row that is read, tiles of the longest part
    int len;                                               // its tokens
    int64_t start;                                         // first place
};

struct Bars {
    uint64_t wide_landed[kWideStages], wide_empty[kWideStages];
    uint64_t narrow_landed[kNarrowStages], narrow_empty[kNarrowStages];
    uint64_t full[8], free[8];                             // K and V of each slot (kBf16: full when the copies landed)
    uint64_t s_full[2][2], p_full[2][2];                   // of each group's S buffers
    uint64_t o_done[2], drain[2];
};

// A CTA's stretch of the line and where it is on it.
struct Walk {
    int64_t share, x, end, block_start;                    // block_start: first place of the block in s.runs
    int64_t total, block_total;
    int block, n_runs;
    // the job at hand: rows [row0, row0 + rows) of run (first, count), tokens [t0, t1)
    int first, lead, kvh, row0, rows, len, tile0, tile1;
    int run_rows, c0, nsplit;                              // rows of the run's KV head; first CTA of the job, and CTAs
    bool wide;
};

struct Shared {
    Bars bars;
    uint32_t tmem_slot;
    int abort, bad_from;                                   // bad_from: first token whose page is out of range
    int search, job_there;                                 // for the next job: what find_job found
    int skip;                                              // an earlier job met an error: nothing more is computed
    Walk w;
    Run runs[kBlockReq];
    int len[kBlockReq];                                    // shared tokens of each request of the block
};
static_assert(kData + 1024 + sizeof(Shared) <= 232448, "one CTA fits an SM");

// Scratch of the search, in Q's place.
struct Scratch {
    int lead[3][kBlockReq], most[3][kBlockReq];
    uint32_t cont[3][4];
    int heads[3][4];
    int64_t warp_sum[3][4];
    int64_t total[kMaxBlocks];
    unsigned long long work[2];
};
static_assert(sizeof(Scratch) <= kQBytes, "the scratch fits in Q's place");

// Instruction descriptor of kind::f16, 128 x n, fp32 accumulator.
template <bool kBf>
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn)
{
    return umma_idesc_f16(128, n, b_mn) | (kBf ? (1u << 7) | (1u << 10) : 0u);
}

// A score buffer: 64 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
                 "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
                 "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
                   "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
                   "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
                   "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
                   "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
                 : "r"(taddr)
                 : "memory");
}

// 16 columns stored; tmem_wait_put waits for all that this thread has stored.
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 "
                 "[%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                   "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_put() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One thread of a whole warp.  What it alone issues needs no vote over the
// operands, which a branch on the lane would cost the tensor-core instructions.
__device__ __forceinline__ bool elect_one()
{
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on != 0;
}

__device__ __forceinline__ void red_add_f32x4(float4 *at, float4 v)
{
    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1,%2,%3,%4};"
                 ::"l"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// Registers of this warpgroup's threads from here on.
template <int kRegs>
__device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// O of the rows that are `wanted`, out of tensor memory onto their sums (from
// zero, the first time).  Sums that are not behind the maximum are added to by
// reductions at L2, which nothing here waits for: a row's sums are its thread's alone.
__device__ __forceinline__ void flush_sums(uint32_t ocol, float4 *part, int rows, bool wanted, bool onto, float mul)
{
    const bool behind = __any_sync(0xFFFFFFFFu, wanted && onto && mul != 1.f);
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        uint32_t o[16];
        tmem_ld16(ocol + 16u * c, o);
        if (wanted)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float4 *at = part + (4 * c + k) * rows;
                float4 v = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                       __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
                if (onto && !behind) {
                    red_add_f32x4(at, v);
                    continue;
                }
                if (onto) {
                    const float4 u = __ldcg(at);
                    v = make_float4(fmaf(u.x, mul, v.x), fmaf(u.y, mul, v.y), fmaf(u.z, mul, v.z), fmaf(u.w, mul, v.w));
                }
                __stcg(at, v);
            }
    }
}

// The runs of a block of requests and their places on the line, worked out by
// the 128 threads of a team.  c.total[block]: all its places.  list: also the
// runs themselves and every request's shared tokens, into s.
template <int kNarrowCost, int kBorderCost>
__device__ __forceinline__ void find_runs(const PrefixArgs &a, Shared &s, Scratch &c, int team, int block, int ps_shift,
                                          bool list, Work *work = nullptr)
{
    const int i = threadIdx.x & 127, lane = threadIdx.x & 31, quarter = i >> 5;
    const uint32_t bar = 2 + team;
    const int r = block * kBlockReq + i;
    int lead = -1, len = 0;
    if (r < a.batch) {
        const Tokens t = tokens_of(a, r, ps_shift);
        len = t.shared;
        lead = t.lead;
        if (work != nullptr)
            work->add(a, t);
    }
    c.lead[team][i] = lead;
    c.most[team][i] = 0;
    named_barrier_sync(bar, 128);
    // whether request i goes on with the run of request i - 1
    const bool goes_on = i > 0 && len > 0 && c.lead[team][i - 1] == lead;
    const bool starts = len > 0 && !goes_on;
    const uint32_t cont = __ballot_sync(0xFFFFFFFFu, goes_on), heads = __ballot_sync(0xFFFFFFFFu, starts);
    if (lane == 0) {
        c.cont[team][quarter] = cont;
        c.heads[team][quarter] = __popc(heads);
    }
    named_barrier_sync(bar, 128);
    // the nearest request at or before i that starts a run or shares nothing,
    // and the nearest after i
    int head = i, next = kBlockReq;
    for (int k = quarter; k >= 0; --k) {
        uint32_t z = ~c.cont[team][k];
        if (k == quarter)
            z &= 0xFFFFFFFFu >> (31 - lane);
        if (z != 0) {
            head = 32 * k + 31 - __clz(z);
            break;
        }
    }
    for (int k = quarter; k < 4; ++k) {
        uint32_t z = ~c.cont[team][k];
        if (k == quarter)
            z &= lane == 31 ? 0u : 0xFFFFFFFFu << (lane + 1);
        if (z != 0) {
            next = 32 * k + __ffs(z) - 1;
            break;
        }
    }
    if (len > 0)
        atomicMax(&c.most[team][head], len);
    named_barrier_sync(bar, 128);
    int64_t places = 0;
    Run run = {};
    if (starts) {
        run.first = r;
        run.lead = lead;
        run.count = next - i;
        run.len = c.most[team][i];
        run.tiles = (run.len + kTok - 1) / kTok;
        const int rows = run.count * a.n_query * a.group, row_tiles = (rows + 127) / 128;
        places = static_cast<int64_t>(row_tiles / 2) * (kBorderCost + static_cast<int64_t>(kWideCost) * run.tiles) +
                 (row_tiles & 1) * (kBorderCost + static_cast<int64_t>(kNarrowCost) * run.tiles);
        places *= a.num_kv_heads;
    }
    int64_t upto = places;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xFFFFFFFFu, upto, off);
        upto += lane >= off ? o : 0;
    }
    if (lane == 31)
        c.warp_sum[team][quarter] = upto;
    named_barrier_sync(bar, 128);
    int64_t before = 0, all = 0;
    int number = __popc(heads & ((1u << lane) - 1u)), of = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        before += k < quarter ? c.warp_sum[team][k] : 0;
        all += c.warp_sum[team][k];
        number += k < quarter ? c.heads[team][k] : 0;
        of += c.heads[team][k];
    }
    if (i == 0)
        c.total[block] = all;
    if (list) {
        run.start = before + upto - places;
        if (starts)
            s.runs[number] = run;
        s.len[i] = len;
        if (i == 0) {
            s.w.n_runs = of;
            s.w.block = block;
            s.w.block_total = all;
        }
    }
}

// Quotient of numbers that are not negative, nearly always of 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0)
        return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The job at place x of the line, by one thread; moves x past what this CTA does
// of it.  False if that is nothing (x lies in the border).
template <int kNarrowCost, int kBorderCost>
__device__ __forceinline__ bool set_job(const PrefixArgs &a, Shared &s)
{
    Walk &w = s.w;
    int k = 0;
    // the run that holds x (places of the block before a run's start are the run before's)
    const int64_t at = w.x - w.block_start;
    int hi = w.n_runs - 1;
    while (k < hi) {
        const int mid = (k + hi + 1) / 2;
        if (s.runs[mid].start <= at)
            k = mid;
        else
            hi = mid - 1;
    }
    const Run run = s.runs[k];
    const int all_rows = run.count * a.n_query * a.group, row_tiles = (all_rows + 127) / 128;
    const int64_t wide = kBorderCost + static_cast<int64_t>(kWideCost) * run.tiles;
    const int64_t narrow = kBorderCost + static_cast<int64_t>(kNarrowCost) * run.tiles;
    const int64_t per_head = row_tiles / 2 * wide + (row_tiles & 1) * narrow;
    const int64_t in_run = at - run.start;
    const int kvh = static_cast<int>(quotient(in_run, per_head));
    const int64_t in_head = in_run - kvh * per_head;
    const int pair = static_cast<int>(min(quotient(in_head, wide), static_cast<int64_t>(row_tiles / 2)));
    w.wide = pair < row_tiles / 2;
    const int cost = w.wide ? kWideCost : kNarrowCost;     // (a share is longer: every CTA of a job has a tile)
    // places [job, job + size) of the line; tiles from `start` on
    const int64_t job = w.block_start + run.start + kvh * per_head + pair * wide, size = w.wide ? wide : narrow;
    const int64_t start = job + kBorderCost;
    const int64_t from = max(w.x - start, static_cast<int64_t>(0)), to = min(w.end - start, size - kBorderCost);
    w.x = min(w.end, job + size);
    // a tile is the CTA's in whose stretch its first place lies
    w.tile0 = static_cast<int>(quotient(from + cost - 1, cost));
    w.tile1 = to <= 0 ? 0 : static_cast<int>(quotient(to + cost - 1, cost));
    if (w.tile0 >= w.tile1)
        return false;
    const int64_t c0 = quotient(start, w.share), c1 = quotient(start + static_cast<int64_t>(run.tiles - 1) * cost, w.share);
    w.c0 = static_cast<int>(c0);
    w.nsplit = static_cast<int>(c1 - c0) + 1;
    w.run_rows = all_rows;
    w.first = run.first;
    w.kvh = kvh;
    w.row0 = 256 * pair;
    w.rows = min(all_rows - w.row0, w.wide ? 256 : 128);
    w.len = run.len;
    w.lead = run.lead;
    return true;
}

// The job at hand as a warp works it off.
struct Job {
    bool wide;
    int tile0, n_tiles, kvh, first, len;
    const int32_t *bt;                       // the row of the table that is read

    __device__ __forceinline__ Job(const PrefixArgs &a, const Shared &s)
        : wide(s.w.wide), tile0(s.w.tile0), n_tiles(s.w.tile1 - s.w.tile0), kvh(s.w.kvh), first(s.w.first), len(s.w.len),
          bt(a.block_table + static_cast<int64_t>(s.w.lead) * a.max_pages_per_seq)
    {
    }
    // of group gr: the first tile (of the job's), how far apart they are, and how many
    __device__ __forceinline__ int first_tile(int gr) const { return wide ? 0 : gr; }
    __device__ __forceinline__ int step() const { return wide ? 1 : 2; }
    __device__ __forceinline__ int tiles(int gr) const { return (n_tiles - first_tile(gr) + step() - 1) / step(); }
};

// What went through the rings, the buffers and the barriers in the jobs before:
// stages of either ring, tiles, tiles of the warp's group, jobs.
struct Done {
    uint32_t wide = 0, narrow = 0, tiles = 0, group = 0, jobs = 0;
    __device__ __forceinline__ void add(const Job &j, int gr)
    {
        (j.wide ? wide : narrow) += 2 * j.n_tiles;
        tiles += j.n_tiles;
        group += j.tiles(gr);
        ++jobs;
    }
};

// One block-wide barrier opens a job: its numbers are in s.  False: there is none.
// Another ends its work, by all but the results.
__device__ __forceinline__ bool open_job(const Shared &s)
{
    __syncthreads();
    return s.job_there;
}
__device__ __forceinline__ void end_job()
{
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
}

// The next job, found by the softmax warps.
template <int kNarrowCost, int kBorderCost>
__device__ __forceinline__ void find_job(const PrefixArgs &a, Shared &s, Scratch &scratch, int ps_shift)
{
    named_barrier_sync(1, 256);              // the last job's numbers have been read
    if (threadIdx.x >= 128)
        return;
    for (;;) {
        if (threadIdx.x == 0) {
            Walk &w = s.w;
            s.search = w.x >= w.end ? 0 : w.x >= w.block_start + w.block_total ? 2 : set_job<kNarrowCost, kBorderCost>(a, s) ? 1 : 3;
            s.bad_from = 0x7FFFFFFF;
            s.job_there = s.search == 1;
            // as the last job left it: a warp of the next one may raise the flag
            // before others have looked, and all have to meet at its barriers
            s.skip = s.abort;
        }
        named_barrier_sync(2, 128);
        const int found = s.search, block = s.w.block + 1;
        if (found < 2)
            return;
        named_barrier_sync(2, 128);          // everyone has read it
        if (found == 2) {
            if (threadIdx.x == 0)
                s.w.block_start += s.w.block_total;
            find_runs<kNarrowCost, kBorderCost>(a, s, scratch, 0, block, ps_shift, true);
            named_barrier_sync(2, 128);
        }
    }
}

// ------------------------------------------------------------------ Q, softmax, the rows' results

template <int kKind, bool kPrecise>
__device__ __forceinline__ void softmax_role(const PrefixArgs &a, Shared &s, uint8_t *sm, uint32_t tmem, int warp)
{
    using B = Build<kKind, kPrecise>;
    constexpr int kSBufs = B::kSBufs;
    constexpr bool kBlocks = B::kBlocks;
    Bars &bar = s.bars;
    Scratch &scratch = *reinterpret_cast<Scratch *>(sm + kOffQ);
    const int lane = threadIdx.x & 31, m = threadIdx.x & 127, gr = warp >> 2;
    const int ps_shift = __ffs(a.page_size) - 1;
    const int hkv = a.num_kv_heads, per_request = a.n_query * a.group;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t scol = tmem + lanes + kColS + 128u * gr, ocol = tmem + lanes + kColO + 128u * gr;
    volatile int *abort_flag = &s.abort;
    Done done;
    for (;;) {
        find_job<B::kNarrowCost, B::kBorderCost>(a, s, scratch, ps_shift);
        if (!open_job(s))
            return;
        const Walk &w = s.w;
        const Job job(a, s);
        const bool wide = job.wide;
        const int tile0 = job.tile0, tile1 = tile0 + job.n_tiles, kvh = job.kvh, first = job.first;
        const int step = job.step(), mine0 = job.first_tile(gr), mine = job.tiles(gr);
        const uint32_t group_done = done.group;
        const int32_t *bt = job.bt;
        const int tile_rows = wide ? min(128, w.rows - 128 * gr) : w.rows;             // of the group's row tile
        // place of the group's part: the job's, behind one of the same number per CTA
        const int64_t place0 = 2 * (static_cast<int64_t>(first) * per_request * hkv +
                                    static_cast<int64_t>(kvh) * w.run_rows + w.row0) +
                               gr * (wide ? 128 : w.rows);
        const int local = wide ? 128 * gr + m : m;
        const bool row_valid = m < tile_rows;
        int64_t id = 0;
        int lim = 0x7FFFFFFF;                              // tokens the row sees (a slot without a row: no masks)
        if (row_valid) {
            const int at = w.row0 + local, req = at / per_request, in = at - req * per_request;
            id = (static_cast<int64_t>(first + req) * a.n_query + in / a.group) * a.num_q_heads + kvh * a.group +
                 in % a.group;
            lim = s.len[first % kBlockReq + req];
        }
        float m_used = -INFINITY, l_sum = 0.f;
        // This row's sums so far (four dims of all the tile's rows side by side, in the
        // rows' places) are behind m_used by sums_mul.  With fp32 output O goes there
        // now and then.  Else, and then for good (`saved`), it goes there when the
        // row's tokens end before the others' do: the others' further values are not
        // the row's, and a NaN or an infinity among them, times its weights of 0, would be.
        float sums_mul = 1.f;
        bool saved = false;
        float4 *const sums = a.pre_o + (256ll * blockIdx.x + place0) * 32 + m;

        if (!s.skip) {
            const float kv_scale = B::kConvert && !kBlocks ? a.k_scale[kvh] : 1.f;
            const float signed_mul = a.qk_scale_log2 * kv_scale;
            // A warp's 32 rows, two at a time: 16 lanes read a row (a row per lane
            // touches 32 sectors a load: 4 us).  Over an FP8 cache a row is scaled by
            // the power of two that puts its largest element in [2^14, 2^15).
            // The scores' multiplier is not negative: a negative one turns q.
            uint4 qv[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int from = 2 * i + (lane >> 4);
                const int64_t at = __shfl_sync(0xFFFFFFFFu, row_valid ? id : -1, from);
                qv[i] = make_uint4(0u, 0u, 0u, 0u);
                if (at >= 0)
                    qv[i] = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + at * kHeadDim) +
                                   (lane & 15));
            }
            int e = 0;
            uint8_t *qs = sm + kOffQ + (wide ? gr : 0) * kQBytes + ((lane & 15) >> 3) * (kQBytes / 2);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int from = 2 * i + (lane >> 4), row = 32 * (warp & 3) + from;
                uint32_t h[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
                if constexpr (B::kConvert) {
                    uint32_t mx = 0;                       // of both halves
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx = __vmaxu2(mx, h[k] & 0x7FFF7FFFu);
                    mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
                    for (int off = 1; off < 16; off <<= 1)
                        mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
                    const int ei = q_row_exponent(mx), mine_e = __shfl_sync(0xFFFFFFFFu, ei, 16 * (lane & 1));
                    e = lane >> 1 == i ? mine_e : e;
                    const float q_mul = __int_as_float(((127 + ei) << 23) | (signed_mul < 0.f ? 0x80000000u : 0u));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = bf16x2_to_f32x2(h[k]);
                        h[k] = f32x2_to_f16x2(f.x * q_mul, f.y * q_mul);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[k] ^= signed_mul < 0.f ? 0x80008000u : 0u;
                }
                if (wide || gr == 0)
                    *reinterpret_cast<uint4 *>(qs + sw128_chunk(row, lane & 7)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
            const float mul = fabsf(signed_mul) * __int_as_float((127 - e) << 23);
            fence_proxy_async_smem();
            named_barrier_sync(5, 320);                // the softmax and the issuing warps

            // block-scaled: lane i has the exponents of the tile's block i,
            // fetched a tile ahead (ek in the low byte, ev in the high one)
            [[maybe_unused]] int exps = 0, exps_next = 0, page_next = -1;
            const int blk = lane * kBlockTokens;
            const auto page_at = [&](int tile) {
                const int tok = tile * kTok + blk;
                return lane < kTok / kBlockTokens && tile < tile1 && tok < w.len ? __ldcg(bt + (tok >> ps_shift)) : -1;
            };
            const auto exps_at = [&](int tile, int page) {
                if (page < 0 || page >= a.num_pages)
                    return 0;
                const int64_t at = ((static_cast<int64_t>(page) * hkv + kvh) << (ps_shift - 4)) +
                                   (((tile * kTok + blk) & (a.page_size - 1)) >> 4);
                const int ek = max(static_cast<int>(__ldcg(a.k_exp + at)), kReadKeyExpMin);
                const int ev = max(static_cast<int>(__ldcg(a.v_exp + at)), kReadValueExpMin);
                return (ek & 0xFF) | (min(ev, kReadValueExpMax) << 8);
            };
            if constexpr (kBlocks) {
                const int t = tile0 + mine0;
                exps_next = exps_at(t, page_at(t));
                page_next = page_at(t + step);
            }
            for (int i = 0; i < mine; ++i) {
                const int tile = tile0 + mine0 + i * step;
                const uint32_t gi = group_done + i, sb = gi % kSBufs;
                if constexpr (kBlocks) {
                    exps = exps_next;
                    exps_next = exps_at(tile + step, page_next);
                    page_next = page_at(tile + 2 * step);
                }
                if (!__all_sync(0xFFFFFFFFu, wait_or_abort(&bar.s_full[gr][sb], (gi / kSBufs) & 1, kCopyWaitLimitNs,
                                                           abort_flag, 4u)))
                    break;
                tmem_fence_after_sync();
                const uint32_t col = scol + 64u * sb;
                uint32_t sv[kTok];
                tmem_ld64(col, sv);
                const int vis = lim - tile * kTok;     // > 0: the row sees the tile
                // a row that has ended has scores of -inf, times 1: the multiplier may be 0
                const float row_mul = vis > 0 ? mul : 1.f;
                bool ending = false, save = false;
                if (!__all_sync(0xFFFFFFFFu, vis >= kTok)) {   // a row's tokens end between tiles
#pragma unroll
                    for (int k = 0; k < kTok; ++k)
                        sv[k] = vis > 0 ? sv[k] : 0xFF800000u;
                    ending = vis <= 0 && !saved && l_sum != 0.f;
                    save = __any_sync(0xFFFFFFFFu, ending);
                }
                // block q (16 columns) of the tile: its multiplier and its ev
                [[maybe_unused]] float mk[4], ev[4];
                if constexpr (kBlocks) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int x = __shfl_sync(0xFFFFFFFFu, exps, q);
                        mk[q] = row_mul * __int_as_float((127 + static_cast<int8_t>(x & 0xFF)) << 23);
                        ev[q] = static_cast<float>(x >> 8);
                    }
                }
                // ---- the tile's largest score
                float mx = -INFINITY;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 16 * q; k < 16 * q + 16; k += 4) {
                        top[0] = fmaxf(top[0], fmaxf(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1])));
                        top[1] = fmaxf(top[1], fmaxf(__uint_as_float(sv[k + 2]), __uint_as_float(sv[k + 3])));
                    }
                    const float t = fmaxf(top[0], top[1]);
                    if constexpr (kBlocks)
                        mx = t != -INFINITY ? fmaxf(mx, fmaf(t, mk[q], ev[q])) : mx;
                    else
                        mx = fmaxf(mx, t);
                }
                if constexpr (!kBlocks)
                    mx = mx == -INFINITY ? mx : mx * row_mul;
                const bool raise = row_valid && mx > m_used + kRaiseThreshold;
                const float alpha = raise ? (m_used == -INFINITY ? 0.f : fast_exp2(m_used - mx)) : 1.f;
                const bool flush = kPrecise && i > 0 && i % B::kFlush == 0;
                const bool rescale = raise && m_used != -INFINITY && i > 0 && !flush;
                const bool scale = __any_sync(0xFFFFFFFFu, rescale);
                if (scale || save || flush) {
                    // O holds the group's earlier tiles once O += P V of the last one is done
                    if (!__all_sync(0xFFFFFFFFu, wait_or_abort(&bar.o_done[gr], (gi - 1) & 1, kCopyWaitLimitNs,
                                                               abort_flag, 4u)))
                        break;
                    tmem_fence_after_sync();
                    if (save || flush) {
                        flush_sums(ocol, sums, tile_rows, row_valid && !saved && (flush || ending),
                                   kPrecise && i > B::kFlush, sums_mul);
                        sums_mul = flush || ending ? 1.f : sums_mul;
                        saved = saved || ending;
                    }
                    if (scale) {
                        const float f = rescale ? alpha : 1.f;
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            uint32_t o[16];
                            tmem_ld16(ocol + 16u * c, o);
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st16(ocol + 16u * c, o);
                        }
                    }
                }
                if (raise) {
                    sums_mul *= alpha;
                    l_sum *= alpha;
                    m_used = mx;
                }
                // ---- P = 2^(s - m_used + kLift), written over S
                const float base = (m_used == -INFINITY ? 0.f : m_used) - B::kLift;
                float sum = 0.f;
                uint64_t sum2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float p[32];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float mq = kBlocks ? mk[2 * c + q] : row_mul, off = kBlocks ? ev[2 * c + q] - base : -base;
                        const uint64_t mq2 = f2_pack(mq, mq), off2 = f2_pack(off, off);
#pragma unroll
                        for (int k = 16 * q; k < 16 * q + 16; k += 2) {
                            float x0, x1;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[32 * c + k]), __uint_as_float(sv[32 * c + k + 1])),
                                             mq2, off2), x0, x1);
                            p[k] = fast_exp2(x0);
                            p[k + 1] = fast_exp2(x1);
                            sum2[(k >> 1) & 1] = f2_add(sum2[(k >> 1) & 1], f2_pack(p[k], p[k + 1]));
                        }
                        if constexpr (kBlocks) {       // a block's weights, times 2^-ev
                            float s0, s1, s2, s3;
                            f2_unpack(sum2[0], s0, s1);
                            f2_unpack(sum2[1], s2, s3);
                            sum = fmaf((s0 + s1) + (s2 + s3),
                                       __int_as_float((127 - static_cast<int>(ev[2 * c + q])) << 23), sum);
                            sum2[0] = sum2[1] = f2_pack(0.f, 0.f);
                        }
                    }
                    // the terms of P, each what the rounding of those before it dropped
#pragma unroll
                    for (int t = 0; t < B::kTerms; ++t) {
                        uint32_t h[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            h[k] = B::kConvert ? f32x2_to_f16x2(p[2 * k], p[2 * k + 1])
                                               : f32x2_to_bf16x2(p[2 * k], p[2 * k + 1]);
                            if (t + 1 < B::kTerms) {
                                const float2 f = B::kConvert ? f16x2_to_f32x2(h[k]) : bf16x2_to_f32x2(h[k]);
                                p[2 * k] -= f.x;
                                p[2 * k + 1] -= f.y;
                            }
                        }
                        tmem_put16(col + p_column<B::kTerms>(c, t), h);
                    }
                }
                if constexpr (!kBlocks) {
                    float s0, s1, s2, s3;
                    f2_unpack(sum2[0], s0, s1);
                    f2_unpack(sum2[1], s2, s3);
                    sum = (s0 + s1) + (s2 + s3);
                }
                l_sum += sum;
                tmem_wait_put();
                tmem_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bar.p_full[gr][sb]);
            }
            // the last tile's O += P V
            if (mine > 0 && !*abort_flag)
                wait_or_abort(&bar.o_done[gr], (group_done + mine - 1) & 1, kCopyWaitLimitNs, abort_flag, 4u);
            __syncwarp();
        }
        end_job();
        const bool failed = s.abort != 0;
        {
            const int64_t place = 256ll * blockIdx.x + place0 + m;
            if (row_valid) {
                float lse = l_sum == 0.f ? -INFINITY : l_sum == l_sum ? m_used + __log2f(l_sum) - B::kLift : INFINITY;
                if (failed || lim > s.bad_from)            // the row gets zeros
                    lse = __uint_as_float(0x7FC00000u);
                a.pre_lse[place] = lse;
                if (w.c0 == static_cast<int>(blockIdx.x) && (wide || gr == 0))
                    a.pre_rec[id] = make_int4(static_cast<int>(256ll * w.c0 + place0) + m, wide ? w.nsplit : -w.nsplit,
                                              tile_rows, 0);
            }
            if (!failed && mine > 0) {
                // O, weighted, through shared memory (the operands' place), so that
                // a row's values leave as 512 bytes in a row
                const float vs = B::kConvert && !kBlocks ? a.v_scale[kvh] : 1.f;
                const float wgt = l_sum == 0.f ? 0.f : vs / l_sum;
                float *stage = reinterpret_cast<float *>(sm) + warp * 32 * kStageStride;
                const bool onto = saved || (kPrecise && mine > B::kFlush && row_valid);
#pragma unroll 1
                for (int c = 0; c < 8; c += 2) {
                    float4 u[8];                           // sums, a trip to L2 for two blocks
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        u[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (onto)
                            u[k] = __ldcg(sums + (4 * c + k) * tile_rows);
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t o[16];
                        tmem_ld16(ocol + 16u * (c + half), o);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float4 v = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                                   __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
                            if (onto) {
                                v = saved ? make_float4(0.f, 0.f, 0.f, 0.f) : v;
                                const float4 w = u[4 * half + k];
                                v = make_float4(fmaf(w.x, sums_mul, v.x), fmaf(w.y, sums_mul, v.y),
                                                fmaf(w.z, sums_mul, v.z), fmaf(w.w, sums_mul, v.w));
                            }
                            *reinterpret_cast<float4 *>(stage + lane * kStageStride + 16 * (c + half) + 4 * k) =
                                wgt != 0.f ? make_float4(v.x * wgt, v.y * wgt, v.z * wgt, v.w * wgt)
                                           : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                    }
                }
                named_barrier_sync(6 + gr, 128);           // the sums lie where the rows go
                __syncwarp();
                float4 *to = a.pre_o + (256ll * blockIdx.x + place0 + 32 * (warp & 3)) * 32 + lane;
                const int n = min(32, tile_rows - 32 * (warp & 3));
#pragma unroll 4
                for (int r = 0; r < n; ++r)
                    to[32 * r] = *reinterpret_cast<const float4 *>(stage + r * kStageStride + 4 * lane);
                fence_proxy_async_smem();                  // the reads, for the next job's copies
            }
        }
        tmem_fence_before_sync();
        done.add(job, gr);
    }
}

// ------------------------------------------------------------------ S = Q K^T and O += P V of one group

template <int kKind, bool kPrecise>
__device__ __forceinline__ void issue_role(const PrefixArgs &a, Shared &s, uint8_t *sm, uint32_t tmem, int gr)
{
    using B = Build<kKind, kPrecise>;
    constexpr int kSBufs = B::kSBufs, kSlots = B::kSlots;
    Bars &bar = s.bars;
    volatile int *abort_flag = &s.abort;
    Done done;
    while (open_job(s)) {
        const Job job(a, s);
        const bool wide = job.wide;
        const int step = job.step(), mine0 = job.first_tile(gr), mine = job.tiles(gr);
        const uint32_t group_done = done.group, tiles_done = done.tiles;
        if (!s.skip) {
            named_barrier_sync(5, 320);                    // Q is there
            tmem_fence_after_sync();
            if (elect_one()) {
                constexpr uint32_t idesc_s = idesc<!B::kConvert>(kTok, false), idesc_o = idesc<!B::kConvert>(128, true);
                const uint64_t dq = umma_desc(smem_addr(sm + kOffQ + (wide ? gr : 0) * kQBytes), 0, 1024);
                const uint64_t dk = umma_desc(smem_addr(sm + B::kOffBufs), 0, 1024);
                const uint64_t dv = umma_desc(smem_addr(sm + B::kOffBufs + kHalfBytes), kSliceBytes, 1024);
                const uint32_t scol = tmem + kColS + 128u * gr, ocol = tmem + kColO + 128u * gr;
                const uint64_t limit = B::kConvert ? kCopyWaitLimitNs : a.copy_wait_ns;
                const unsigned bit = B::kConvert ? 4u : 1u;
                // S of the group's tile i, into its S buffer
                const auto scores = [&](int i) {
                    const uint32_t gi = group_done + i, tile = tiles_done + mine0 + i * step, slot = tile % kSlots;
                    // P of the tile before was read from there
                    if (i >= kSBufs && !wait_or_abort(&bar.o_done[gr], (gi - kSBufs) & 1, kCopyWaitLimitNs, abort_flag, 4u))
                        return false;
                    if (!wait_or_abort(&bar.full[2 * slot], (tile / kSlots) & 1, limit, abort_flag, bit))
                        return false;
                    tmem_fence_after_sync();
                    const uint64_t kb = dk + ((slot * 2 * kHalfBytes) >> 4);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_f16(scol + 64u * (gi % kSBufs), dq + (((kk >> 2) * (kQBytes / 2) + (kk & 3) * 32) >> 4),
                                 kb + (((kk >> 2) * kSliceBytes + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
                    umma_commit(&bar.s_full[gr][gi % kSBufs]);
                    umma_commit(&bar.free[2 * slot]);
                    if (!wide)                         // the other group does not read it
                        umma_commit(&bar.free[2 * slot]);
                    return true;
                };
                bool ok = true;
                for (int i = 0; i < kSBufs && i < mine; ++i)
                    ok = ok && scores(i);
                for (int i = 0; ok && i < mine; ++i) {
                    const uint32_t gi = group_done + i, tile = tiles_done + mine0 + i * step, slot = tile % kSlots;
                    if (!wait_or_abort(&bar.full[2 * slot + 1], (tile / kSlots) & 1, limit, abort_flag, bit))
                        break;
                    if (!wait_or_abort(&bar.p_full[gr][gi % kSBufs], (gi / kSBufs) & 1, kCopyWaitLimitNs, abort_flag, 4u))
                        break;
                    tmem_fence_after_sync();
                    const uint64_t vb = dv + ((slot * 2 * kHalfBytes) >> 4);
                    const uint32_t pcol = scol + 64u * (gi % kSBufs);
                    const bool onto = kPrecise ? i % B::kFlush != 0 : i > 0;
#pragma unroll
                    for (int t = 0; t < B::kTerms; ++t)
#pragma unroll
                        for (int kk = 0; kk < kTok / 16; ++kk)
                            umma_f16_ts(ocol, pcol + p_column<B::kTerms>(kk >> 1, t) + 8u * (kk & 1),
                                        vb + static_cast<uint64_t>((kk * 2048) >> 4), idesc_o,
                                        onto || t > 0 || kk > 0);
                    umma_commit(&bar.o_done[gr]);
                    umma_commit(&bar.free[2 * slot + 1]);
                    if (!wide)
                        umma_commit(&bar.free[2 * slot + 1]);
                    ok = i + kSBufs >= mine || scores(i + kSBufs);
                }
                // nothing this lane issued may still run when the job ends
                umma_commit(&bar.drain[gr]);
                if (!mbar_wait_bounded(&bar.drain[gr], done.jobs & 1, kCopyWaitLimitNs))
                    atomicOr(&g_umma_error, 4u);
            }
            __syncwarp();
        }
        end_job();
        done.add(job, gr);
    }
}

// ------------------------------------------------------------------ copies of K's and V's rows

template <int kKind, bool kPrecise>
__device__ __forceinline__ void copy_role(const PrefixArgs &a, Shared &s, uint8_t *sm, const CUtensorMap &k_map,
                                          const CUtensorMap &v_map)
{
    using B = Build<kKind, kPrecise>;
    constexpr int kSlots = B::kSlots;
    Bars &bar = s.bars;
    const int lane = threadIdx.x & 31, hkv = a.num_kv_heads;
    const int ps_shift = __ffs(a.page_size) - 1;
    volatile int *abort_flag = &s.abort;
    Done done;
    while (open_job(s)) {
        const Job job(a, s);
        const bool wide = job.wide, failed_before = s.skip != 0;
        const int tile0 = job.tile0, tile1 = tile0 + job.n_tiles, kvh = job.kvh;
        const int32_t *bt = job.bt;
        const uint32_t wide_done = done.wide, narrow_done = done.narrow, tiles_done = done.tiles;
        uint32_t issued = 0;                               // stages or buffers in this job
        if (!failed_before) {
            const uint64_t policy = l2_policy_evict_normal();
            // boxes of a tile: one lane each; a box does not cross a page
            const int box = min(a.page_size, B::kConvert ? kChunkTokens : kTok), boxes = kTok / box;
            const int64_t outside = -256;              // rows no copy finds: zeros
            const auto page_at = [&](int tile) {
                const int tok = tile * kTok + lane * box;
                return lane < boxes && tile < tile1 && tok < job.len ? __ldcg(bt + (tok >> ps_shift)) : -1;
            };
            int page = page_at(tile0);
            bool ok = true;
            for (int tile = tile0; ok && tile < tile1; ++tile) {
                const int tok = tile * kTok + lane * box;
                const bool held = lane < boxes && tok < job.len, fine = held && page >= 0 && page < a.num_pages;
                if (held && !fine)
                    atomicMin(&s.bad_from, tok);
                const int y = static_cast<int>(
                    fine ? (static_cast<int64_t>(page) * hkv + kvh) * a.page_size + (tok & (a.page_size - 1)) : outside);
                page = page_at(tile + 1);
                const uint32_t t = tiles_done + (tile - tile0), slot = t % kSlots;
                for (int q = 0; ok && q < 2; ++q) {    // K, then V
                    const void *map = q ? static_cast<const void *>(&v_map) : static_cast<const void *>(&k_map);
                    if constexpr (B::kConvert) {
                        uint64_t *landed = wide ? bar.wide_landed : bar.narrow_landed;
                        uint64_t *empty = wide ? bar.wide_empty : bar.narrow_empty;
                        const uint32_t n = (wide ? wide_done : narrow_done) + issued;
                        const uint32_t st = wide ? n % kWideStages : n % kNarrowStages;
                        const uint32_t round = wide ? n / kWideStages : n / kNarrowStages;
                        if (round > 0)
                            ok = __all_sync(0xFFFFFFFFu, wait_or_abort(&empty[st], (round - 1) & 1, kCopyWaitLimitNs,
                                                                       abort_flag, 4u));
                        if (!ok)
                            break;
                        if (lane == 0)
                            mbar_arrive_expect_tx(&landed[st], kRingStage);
                        __syncwarp();
                        if (lane < boxes)
                            tma_load_2d(sm + (wide ? kOffRingWide : kOffRingNarrow) + st * kRingStage + lane * box * 128,
                                        map, 0, y, &landed[st], policy);
                    } else {
                        const uint32_t b = 2 * slot + q;
                        if (t >= kSlots)
                            ok = __all_sync(0xFFFFFFFFu, wait_or_abort(&bar.free[b], (t / kSlots - 1) & 1,
                                                                       kCopyWaitLimitNs, abort_flag, 4u));
                        if (!ok)
                            break;
                        if (lane == 0)
                            mbar_arrive_expect_tx(&bar.full[b], kHalfBytes);
                        __syncwarp();
                        if (lane < boxes)
#pragma unroll
                            for (int half = 0; half < 2; ++half)
                                tma_load_2d(sm + B::kOffBufs + b * kHalfBytes + half * kSliceBytes + lane * box * 128, map,
                                            64 * half, y, &bar.full[b], policy);
                    }
                    ++issued;
                }
            }
        }
        end_job();
        if (s.abort != 0 && !failed_before && lane == 0) {
            // none of the copies in flight may land after the CTA has moved on
            bool drained = true;
            if constexpr (B::kConvert) {
                const uint32_t n_st = wide ? kWideStages : kNarrowStages, all = (wide ? wide_done : narrow_done) + issued;
                uint64_t *landed = wide ? bar.wide_landed : bar.narrow_landed;
                for (uint32_t n = all - min(n_st, issued); n < all; ++n)
                    drained &= mbar_wait_bounded(&landed[n % n_st], (n / n_st) & 1, kCopyWaitLimitNs);
            } else {
                const uint32_t all = 2 * tiles_done + issued;
                for (uint32_t n = all - min(2u * kSlots, issued); n < all; ++n)
                    drained &= mbar_wait_bounded(&bar.full[n % (2 * kSlots)], (n / (2 * kSlots)) & 1, kCopyWaitLimitNs);
            }
            if (!drained)
                atomicOr(&g_umma_error, 2u);
        }
        __syncwarp();
        done.add(job, 0);
    }
}

// ------------------------------------------------------------------ e4m3 -> f16 (exact)

template <int kKind, bool kPrecise>
__device__ __forceinline__ void convert_role(const PrefixArgs &a, Shared &s, uint8_t *sm, int warp)
{
    using B = Build<kKind, kPrecise>;
    constexpr int kSlots = B::kSlots;
    Bars &bar = s.bars;
    const int tid = threadIdx.x, lane = tid & 31;
    volatile int *abort_flag = &s.abort;
    Done done;
    while (open_job(s)) {
        const Job job(a, s);
        const bool wide = job.wide;
        const int n_tiles = job.n_tiles;
        const uint32_t wide_done = done.wide, narrow_done = done.narrow, tiles_done = done.tiles;
        if (!s.skip) {
            // Warps 8 .. 11 convert K, 12 .. 15 V: what a warp waits for (the
            // copy, the buffer, its own stores) the others do not.
            const int ct = tid & 127, v = (warp - 8) >> 2;
            const int c = ct & 7;                      // 16-byte chunk (16 dims) of a row
            uint64_t *landed = wide ? bar.wide_landed : bar.narrow_landed;
            uint64_t *empty = wide ? bar.wide_empty : bar.narrow_empty;
            const uint8_t *ring = sm + (wide ? kOffRingWide : kOffRingNarrow);
            const uint32_t before = wide ? wide_done : narrow_done;
            // The next tile's rows are on their way while one's are
            // converted.  Every lane polls; the warp goes on or gives up as one.
            uint4 x[4], next[4];
            const auto landed_at = [&](int j) {
                const uint32_t n = before + 2 * j + v;
                const uint32_t st = wide ? n % kWideStages : n % kNarrowStages;
                const uint32_t round = wide ? n / kWideStages : n / kNarrowStages;
                if (!__all_sync(0xFFFFFFFFu, wait_or_abort(&landed[st], round & 1, a.copy_wait_ns, abort_flag, 1u)))
                    return false;
                const uint8_t *from = ring + st * kRingStage;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int t = (ct >> 3) + 16 * k;
                    next[k] = *reinterpret_cast<const uint4 *>(from + t * 128 + ((c ^ (t & 7)) << 4));
                }
                return true;
            };
            bool more = landed_at(0);
            for (int j = 0; more && j < n_tiles; ++j) {
                const uint32_t tile = tiles_done + j, b = 2 * (tile % kSlots) + v;
                uint8_t *to = sm + B::kOffBufs + b * kHalfBytes;
                const uint32_t n = before + 2 * j + v, st = wide ? n % kWideStages : n % kNarrowStages;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] = next[k];
                if (j + 1 < n_tiles)
                    more = landed_at(j + 1);
                if (tile >= kSlots && !__all_sync(0xFFFFFFFFu, wait_or_abort(&bar.free[b], (tile / kSlots - 1) & 1,
                                                                             kCopyWaitLimitNs, abort_flag, 4u)))
                    break;
                // chunk c of row t goes to the operand's chunks 2 c, 2 c + 1;
                // lanes with c >= 4 (the other slice, the same banks) store
                // theirs in the other order
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int t = (ct >> 3) + 16 * k;
                    const uint32_t slice = static_cast<uint32_t>((c >> 2) * kSliceBytes);
                    const uint32_t o0 = slice + sw128_chunk(t, 2 * (c & 3));
                    const uint32_t o1 = slice + sw128_chunk(t, 2 * (c & 3) + 1);
                    const bool swap = c >= 4;
                    const uint32_t a0 = swap ? x[k].z : x[k].x, a1 = swap ? x[k].w : x[k].y;
                    const uint32_t b0 = swap ? x[k].x : x[k].z, b1 = swap ? x[k].y : x[k].w;
                    *reinterpret_cast<uint4 *>(to + (swap ? o1 : o0)) =
                        make_uint4(lo16_e4m3x2_to_f16x2(a0), hi16_e4m3x2_to_f16x2(a0),
                                   lo16_e4m3x2_to_f16x2(a1), hi16_e4m3x2_to_f16x2(a1));
                    *reinterpret_cast<uint4 *>(to + (swap ? o0 : o1)) =
                        make_uint4(lo16_e4m3x2_to_f16x2(b0), hi16_e4m3x2_to_f16x2(b0),
                                   lo16_e4m3x2_to_f16x2(b1), hi16_e4m3x2_to_f16x2(b1));
                }
                fence_proxy_async_smem();              // the writes, for the tensor core;
                __syncwarp();                          // the ring reads, for the next copy
                if (lane == 0) {
                    mbar_arrive(&empty[st]);
                    mbar_arrive(&bar.full[b]);
                }
            }
        }
        end_job();
        done.add(job, 0);
    }
}

template <int kKind, bool kPrecise>
__global__ void __launch_bounds__(Build<kKind, kPrecise>::kThreads, 1)
prefix_rows_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                   const PrefixArgs a)
{
    using B = Build<kKind, kPrecise>;
    constexpr int kThreads = B::kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Shared &s = *reinterpret_cast<Shared *>(sm + kData);
    Scratch &scratch = *reinterpret_cast<Scratch *>(sm + kOffQ);
    Bars &bar = s.bars;
    const int tid = threadIdx.x;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // the same register for the whole warp
    const int ps_shift = __ffs(a.page_size) - 1;

    if (tid == 0) {
        prefetch_tensor_map(&k_map);
        prefetch_tensor_map(&v_map);
        for (int i = 0; i < kWideStages; ++i) {
            mbar_init(&bar.wide_landed[i], 1);
            mbar_init(&bar.wide_empty[i], 4);
        }
        for (int i = 0; i < kNarrowStages; ++i) {
            mbar_init(&bar.narrow_landed[i], 1);
            mbar_init(&bar.narrow_empty[i], 4);
        }
        for (int i = 0; i < 2 * B::kSlots; ++i) {
            mbar_init(&bar.full[i], B::kConvert ? 4 : 1);
            mbar_init(&bar.free[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            for (int k = 0; k < 2; ++k) {
                mbar_init(&bar.s_full[i][k], 1);
                mbar_init(&bar.p_full[i][k], 4);
            }
            mbar_init(&bar.o_done[i], 1);
            mbar_init(&bar.drain[i], 1);
        }
        fence_mbar_init();
        s.abort = 0;
        s.bad_from = 0x7FFFFFFF;
    }
    grid_dependency_wait();
    // The own pages' kernel may start beside this one: it reads nothing of it but
    // this zero, released behind what was written before the call (decode_split_kernel,
    // kSharing).  It may start as soon as one thread of each CTA has said so: the zero
    // comes before any thread of its CTA does.
    if (blockIdx.x == 0) {
        if (tid == 0) {
            st_release_gpu(a.own_takers, 0);
            __threadfence();
        }
        __syncthreads();
    }
    grid_launch_dependents();

    // ---------------------------------------------- this CTA's stretch of the line
    const int n_blocks = (a.batch + kBlockReq - 1) / kBlockReq;
    constexpr int kTeams = kThreads / 128 < 3 ? kThreads / 128 : 3;
    const int team = tid / 128;
    Work work = {0, 0};
    if (tid == 0)
        scratch.work[0] = scratch.work[1] = 0;
    __syncthreads();
    for (int b = team; team < kTeams && b < n_blocks; b += kTeams)
        find_runs<B::kNarrowCost, B::kBorderCost>(a, s, scratch, team, b, ps_shift, n_blocks == 1, &work);
    if (work.shared + work.own != 0) {
        atomicAdd(&scratch.work[0], static_cast<unsigned long long>(work.shared));
        atomicAdd(&scratch.work[1], static_cast<unsigned long long>(work.own));
    }
    __syncthreads();
    if (tid == 0) {
        Walk &w = s.w;
        w.total = 0;
        for (int b = 0; b < n_blocks; ++b)
            w.total += scratch.total[b];
        work = {static_cast<long long>(scratch.work[0]), static_cast<long long>(scratch.work[1])};
        const int ctas = max(work.sms(gridDim.x), 1);
        const int64_t even = quotient(w.total + ctas - 1, ctas);
        w.share = max(even, static_cast<int64_t>(kMinTiles * kWideCost));
        w.x = min(w.total, w.share * blockIdx.x);
        w.end = min(w.total, w.x + w.share);
        int b = 0;
        int64_t start = 0;
        if (w.x < w.end)
            while (w.x >= start + scratch.total[b])
                start += scratch.total[b++];
        w.block = b;
        w.block_start = start;
    }
    __syncthreads();
    if (s.w.x >= s.w.end)
        return;
    if (warp == 0)
        tmem_alloc(&s.tmem_slot, kTmemCols);
    if (n_blocks > 1 && tid < 128)                         // the runs of the block in which the stretch begins
        find_runs<B::kNarrowCost, B::kBorderCost>(a, s, scratch, 0, s.w.block, ps_shift, true);
    tmem_fence_before_sync();
    __syncthreads();
    tmem_fence_after_sync();
    const uint32_t tmem = s.tmem_slot;

    static_assert(!B::kConvert || 256 * 136 + 256 * 72 + 128 * 56 <= 640 * 96, "what the launch has");
    if (warp < 8) {
        if constexpr (B::kConvert)
            more_registers<136>();
        softmax_role<kKind, kPrecise>(a, s, sm, tmem, warp);
    } else if (B::kConvert && warp < B::kCopy) {
        if constexpr (B::kConvert) {
            fewer_registers<72>();
            convert_role<kKind, kPrecise>(a, s, sm, warp);
        }
    } else {
        if constexpr (B::kConvert)
            fewer_registers<56>();
        if (warp == B::kCopy)
            copy_role<kKind, kPrecise>(a, s, sm, k_map, v_map);
        else if (warp < B::kIssue + 2)
            issue_role<kKind, kPrecise>(a, s, sm, tmem, warp - B::kIssue);
        else                                               // fills the warpgroup
            while (open_job(s))
                end_job();
    }
    tmem_fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tmem_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ combine

// out = sum_s w_s o_s / sum_s w_s with w_s = 2^(lse_s - max lse), over the parts
// of the shared pages and of the row's own.  A lane has four dims of a row and
// the log-sum-exps of every 32nd part; eight parts' values are in flight at a time.
// Each trip to L2 depends on the one before (what parts there are, their
// log-sum-exps, their values), so the first two are made for the next row beside
// the third for this one.  Zeros where any part is invalid (lse NaN); a NaN sum
// (lse +inf) makes the row NaN.
//
// kTogether warps share a row and take its parts in turn: all four of a CTA while
// a CTA has no more than two rows, and so few trips to hide a row's behind (1,280
// rows of 40 parts: 15 us after the parts are there with one warp), else one.
constexpr int kCombineWarps = 4, kCombineCtas = 5;         // resident per SM
struct Parts {
    int4 rec;                                // of the shared pages: as in PrefixArgs
    int64_t own_at;                          // place of the first own part's log-sum-exp
    int np, nt;                              // parts of the shared pages, and all
    float lse0, lse1;                        // of parts `lane` and lane + 32
};
template <int kTogether>
__global__ void __launch_bounds__(32 * kCombineWarps, kCombineCtas)
combine_prefix_kernel(const PrefixArgs a)
{
    __shared__ float4 s_sum[kTogether][32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    constexpr int kRows = kCombineWarps / kTogether;       // of a CTA at a time
    static_assert(kTogether == 1 || kRows == 1, "a CTA's warps work together or alone");
    const int64_t per_request = static_cast<int64_t>(a.n_query) * a.num_q_heads, rows = a.batch * per_request;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    const int per = a.n_query > 1 ? kMultiRowsPerCta : kMaxGroup;
    grid_dependency_wait();
    const auto place = [&](const Parts &p, int q) -> int64_t {     // of part q < np
        return static_cast<int64_t>(p.rec.x) + (p.rec.y < 0 ? 256ll * (q >> 1) + (q & 1) * p.rec.z : 256ll * q);
    };
    const auto lse_of = [&](const Parts &p, int q) {
        return q < p.np ? __ldcg(a.pre_lse + place(p, q))
                        : __ldcg(a.ws_lse + p.own_at + static_cast<int64_t>(q - p.np) * per);
    };
    const auto parts_of = [&](int64_t row) {
        Parts p = {};
        if (row < rows) {
            const int b = static_cast<int>(row / per_request), in = static_cast<int>(row - b * per_request);
            const int hq = in % a.num_q_heads, kvh = hq / a.group, r = in / a.num_q_heads * a.group + hq % a.group;
            const int kind = __ldcg(a.kinds + b);
            p.rec = __ldcg(a.pre_rec + row);
            const int2 pair =
                __ldcg(a.ws_pairs + (static_cast<int64_t>(b) * a.num_kv_heads + kvh) * a.row_blocks + r / per);
            p.np = !(kind & kSharedPart) ? 0 : p.rec.y < 0 ? -2 * p.rec.y : p.rec.y;
            p.nt = p.np + (kind & kOwnPart ? pair.y : 0);
            p.own_at = static_cast<int64_t>(pair.x) * per + r % per;
        }
        return p;
    };
    const auto fetch_lse = [&](Parts &p) {
        p.lse0 = lane < p.nt ? lse_of(p, lane) : -INFINITY;
        p.lse1 = lane + 32 < p.nt ? lse_of(p, lane + 32) : -INFINITY;
    };
    int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + warp / kTogether;
    Parts p = parts_of(row);
    fetch_lse(p);
    for (; row < rows; row += step) {
        Parts next = parts_of(row + step);
        float M = fmaxf(p.lse0, p.lse1);
        bool bad = p.lse0 != p.lse0 || p.lse1 != p.lse1;
        for (int q = lane + 64; q < p.nt; q += 32) {
            const float y = lse_of(p, q);
            bad |= y != y;
            M = fmaxf(M, y);
        }
        bad = __any_sync(0xFFFFFFFFu, bad);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
        const auto weight = [&](float y) { return y == -INFINITY ? 0.f : fast_exp2(y - M); };
        float sum = weight(p.lse0) + weight(p.lse1);
        for (int q = lane + 64; q < p.nt; q += 32)
            sum += weight(lse_of(p, q));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
        const float inv = bad || sum == 0.f ? 0.f : 1.f / sum;       // NaN stays
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q0 = 0; q0 < p.nt; q0 += 8 * kTogether) {
            float4 v[8];
            float wk[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int q = q0 + kTogether * k + warp % kTogether;
                float y = __shfl_sync(0xFFFFFFFFu, q < 32 ? p.lse0 : p.lse1, q % 32);
                if (q >= 64)
                    y = q < p.nt ? lse_of(p, q) : -INFINITY;
                wk[k] = q < p.nt && inv != 0.f ? weight(y) * inv : 0.f;
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (wk[k] != 0.f)                          // a part without weight may hold anything
                    v[k] = __ldcg((q < p.np ? a.pre_o + place(p, q) * 32
                                            : reinterpret_cast<const float4 *>(a.ws_o) +
                                                  (p.own_at + static_cast<int64_t>(q - p.np) * per) * 32) + lane);
            }
            if (q0 == 0)
                fetch_lse(next);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (wk[k] != 0.f) {
                    acc.x += wk[k] * v[k].x;
                    acc.y += wk[k] * v[k].y;
                    acc.z += wk[k] * v[k].z;
                    acc.w += wk[k] * v[k].w;
                }
        }
        if (p.nt == 0)
            fetch_lse(next);
        if constexpr (kTogether > 1) {
            s_sum[warp][lane] = acc;
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int w = 1; w < kTogether; ++w) {
                    const float4 u = s_sum[w][lane];
                    acc.x += u.x; acc.y += u.y; acc.z += u.z; acc.w += u.w;
                }
            }
            __syncthreads();
        }
        if (kTogether == 1 || warp == 0)
            store_row_value4(a.out, row * kHeadDim + 4 * lane, acc, a.out_fp32);
        p = next;
    }
}

cudaLaunchConfig_t dependent(dim3 grid, int threads, size_t smem, cudaStream_t stream, cudaLaunchAttribute (&attr)[1])
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <int kKind, bool kPrecise>
cudaError_t launch_rows(const PrefixArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map, cudaStream_t stream)
{
    constexpr int kBytes = 1024 + kData + static_cast<int>(sizeof(Shared));
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(prefix_rows_kernel<kKind, kPrecise>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
        if (e != cudaSuccess)
            return e;
        if (dev >= 0 && dev < 64)
            configured[dev] = 1;
    }
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg =
        dependent(dim3(static_cast<unsigned>(a.pre_ctas)), Build<kKind, kPrecise>::kThreads, kBytes, stream, attr);
    e = cudaLaunchKernelEx(&cfg, prefix_rows_kernel<kKind, kPrecise>, k_map, v_map, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace

cudaError_t launch_prefix_rows(const PrefixArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map,
                               cudaStream_t stream)
{
    if (a.bf16_cache)
        return a.out_fp32 ? launch_rows<kBf16, true>(a, k_map, v_map, stream)
                          : launch_rows<kBf16, false>(a, k_map, v_map, stream);
    if (a.k_exp != nullptr)
        return a.out_fp32 ? launch_rows<kBlocksFp8, true>(a, k_map, v_map, stream)
                          : launch_rows<kBlocksFp8, false>(a, k_map, v_map, stream);
    return a.out_fp32 ? launch_rows<kFp8, true>(a, k_map, v_map, stream)
                      : launch_rows<kFp8, false>(a, k_map, v_map, stream);
}

cudaError_t launch_combine_prefix(const PrefixArgs &a, cudaStream_t stream)
{
    const int64_t rows = static_cast<int64_t>(a.batch) * a.n_query * a.num_q_heads;
    const int64_t most = kCombineCtas * device_sm_count();
    const bool alone = rows > 2 * most;
    const int64_t ctas = alone ? (rows + kCombineWarps - 1) / kCombineWarps : rows;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg =
        dependent(dim3(static_cast<unsigned>(ctas < most ? ctas : most)), 32 * kCombineWarps, 0, stream, attr);
    const cudaError_t e = alone ? cudaLaunchKernelEx(&cfg, combine_prefix_kernel<1>, a)
                                : cudaLaunchKernelEx(&cfg, combine_prefix_kernel<kCombineWarps>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t read_prefix_error(uint32_t *bits, bool clear) { return read_umma_error_word(bits, clear); }

} // namespace kvq
