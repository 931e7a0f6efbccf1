// kvq_decode_split_body.cuh -- the statements that work off one split (not a
// header: kvq_decode_split.cuh includes it inside two functions).
//
// In the plain cluster builds they stand in the kernel itself, in the others
// in a function (inlined), which a balanced launch calls once per border of
// its share.  The compiler's registers go by that, and each form is measured
// faster where it stands: as a function the plain cluster builds took 58.6
// us instead of 57.8 (8 x 8 x 8,193 tokens, 4 query tokens); in the kernel the
// plain grids took 122.8 instead of 119.8 (bf16, 16 x 8 x 1,000..16,000 tokens,
// 2 query tokens) and 113.0 instead of 111.7 (64 x 8 x 1,000..8,000, fp32
// output), the block-scaled builds 13.9 instead of 13.2 (64 x 8 x 100..300) and
// 31.7 instead of 30.8 (8 x 8 x 8,193, 2 query tokens).
//
// In scope: k_map, v_map, a (ArgsOf<kWindow>) and the build's template
// parameters; with a window job (the split) and first (no split of this CTA
// came before).
    using T = BuildTile<kBf16Cache, kWindow>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + T::kRingBytes);
    int32_t *page_list = reinterpret_cast<int32_t *>(full + kWarps * T::kStages);
    uint32_t *tag_live = reinterpret_cast<uint32_t *>(page_list + kMaxPageList);   // kvq_decode_step:
    uint32_t *tag_want = tag_live + kMaxPageList;                                  // the split's tags
    uint8_t *new_tok = reinterpret_cast<uint8_t *>(tag_want + kMaxPageList);       // [K row][V row]
    // windowed builds, in the place of the tags (kExpBytes, kQFragBytes)
    [[maybe_unused]] uint16_t *blk_exp = reinterpret_cast<uint16_t *>(page_list + kMaxPageList);
    [[maybe_unused]] uint2 *q_frag =
        reinterpret_cast<uint2 *>(reinterpret_cast<uint8_t *>(page_list + kMaxPageList) + kExpBytes);
    constexpr bool kSmemQ = smem_q(kMulti, kWindow);
    __shared__ int s_failed;
    __shared__ int s_stale;                                // kvq_decode_step: a page of this split failed

    // The builds without a window always run the split that their place in
    // the grid names.
    const int split = kWindow ? job.split : static_cast<int>(blockIdx.x);
    const int b = kWindow ? job.b : static_cast<int>(blockIdx.z);
    // with several query tokens, blockIdx.y = KV head x row blocks
    const int line = static_cast<int>(blockIdx.y);
    const int kvh = kWindow ? job.kvh : kMulti ? line / a.row_blocks : line;
    const int rb = kWindow ? job.rb : kMulti ? line % a.row_blocks : 0;
    const int split_tokens = kWindow ? job.span : a.split_tokens;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int gq = lane >> 2, tq = lane & 3;
    const int g = a.group, ps = a.page_size;
    const int ps_shift = __ffs(ps) - 1;                  // ps is 16, 32, 64 or 128
    Rows<kMulti, kWindow> R;
    R.b = b;
    R.kvh = kvh;
    R.row0 = rb * rows_per_cta(kMulti);
    R.nrows = kMulti ? min(rows_per_cta(true), a.n_query * g - R.row0) : g;
    R.slot = kWindow ? (static_cast<int64_t>(b) * a.num_kv_heads + kvh) * (kMulti ? a.row_blocks : 1) + rb
                     : static_cast<int64_t>(b) * gridDim.y + line;
    R.base = job.base;
    if constexpr (kWindow) {
        __shared__ int64_t s_ids[rows_per_cta(kMulti)];
        if (threadIdx.x < R.nrows)
            s_ids[threadIdx.x] = R.id(a, threadIdx.x);
        R.ids = s_ids;
    }

    const int first_page = kWindow ? static_cast<int>(job.t0 >> ps_shift)
                                   : static_cast<int>(static_cast<int64_t>(split) * a.split_tokens / ps);
    const int span_left = a.max_pages_per_seq - first_page;
    const int span = split_tokens / ps < span_left ? split_tokens / ps : span_left;
    const int32_t *bt = a.block_table + static_cast<int64_t>(b) * a.max_pages_per_seq + first_page;
    const int lines_per_tok = kBf16Cache ? 2 : 1;

    if constexpr (!kWindow && kCluster)                    // here, for the registers' sake again
        start_dependent(k_map, v_map);

    // A lane's part of query row nt * 8 + gq: dims 32 tq .. 32 tq + 31.  The
    // single-token windowed builds fetch it here, beside the first table
    // entries (0.3 us sooner under way); only what follows the first copies
    // uses it.
    constexpr bool kEarlyQ = kWindow && !kMulti;
    constexpr int kNT = rows_per_cta(kMulti) / kMaxGroup;   // mma n-tiles of query rows per warp
    constexpr int kRowsT = rows_per_cta(kMulti);
    uint32_t q_raw[kNT][16];
    auto load_q = [&](int nt) {
        uint32_t (&w)[16] = q_raw[nt];
        if (nt * kMaxGroup + gq < R.nrows) {
            const uint4 *src = reinterpret_cast<const uint4 *>(
                static_cast<const uint16_t *>(a.q) + (R.id(a, nt * kMaxGroup + gq) * kHeadDim + 32 * tq));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = read_input(src + i);
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                w[i] = 0;
        }
    };

    // The block-table entries this split can use depend only on the split
    // index, so they are loaded together with the request's length.
    constexpr int kIdsPerThread = (kMaxPageList + kThreads - 1) / kThreads;
    int32_t ids[kIdsPerThread];
    bool every = true;                                     // no window
    if constexpr (kWindow)
        every = !kSharing && a.window == 0;
    if (every) {
#pragma unroll
        for (int k = 0; k < kIdsPerThread; ++k) {
            const int i = threadIdx.x + k * kThreads;
            ids[k] = i < span ? __ldg(bt + i) : -1;
        }
    }
    const int64_t real_len = kWindow && job.real >= 0 ? job.real : a.seq_lens[b];
    if constexpr (kEarlyQ)
        load_q(0);
    // kvq_decode_step: each split checks the tags of its own pages (together
    // the request's used entries) while it streams them, and publishes a
    // failure with its partial; the CTA that sees every split's partial
    // writes the flag and, if the request passed, its new token
    // (finish_here, or finish_step in the workspace form).  A request
    // without tokens to check is decided here.
    const bool step_check = !kWindow && a.expected_tags != nullptr;
    const bool reporter = step_check && split == 0 && kvh == 0 && threadIdx.x == 0;
    const bool aborted = !step_check && a.abort_flags != nullptr && read_plain(a.abort_flags + b) != 0;
    const int64_t cap = static_cast<int64_t>(a.max_pages_per_seq) * ps;
    const bool zero_request = aborted || real_len <= 0 || real_len > cap;
    // Window: from here on `len` and every position count the shortened
    // context (shown_context).
    int64_t len = real_len;
    [[maybe_unused]] int64_t win0 = 0;                     // where the first query's window starts
    if constexpr (kWindow) {
        if (kSharing || a.window > 0) {
            const Shown shown = own_context(a, real_len, job.shared, ps_shift);
            len = shown.len;
            win0 = shown.win0;
            // only entries of pages with a token of the shortened context are read
#pragma unroll
            for (int k = 0; k < kIdsPerThread; ++k) {
                const int i = threadIdx.x + k * kThreads;
                const int64_t v = static_cast<int64_t>(first_page) + i;
                const bool held = !zero_request && i < split_tokens / ps && (v << ps_shift) < len;
                ids[k] = held ? read_input(bt + i + (v < shown.sink_pages ? 0 : shown.hole)) : -1;
            }
        }
    }
    if (reporter && zero_request)                          // the check's verdict without a look:
        a.abort_out[b] = real_len > cap ? 1 : 0;                // too long fails, empty passes
    const int nsplit = zero_request ? 1
                       : kWindow && job.nsplit > 0
                           ? job.nsplit
                           : static_cast<int>((len + a.split_tokens - 1) / a.split_tokens);
    float *part = reinterpret_cast<float *>(smem) + scratch_offset(kMulti);   // cluster partial
    // kvq_decode_step: the split that finishes the step of a request with
    // tokens in the cluster form and when there is one split -- the last
    // split, which holds the new token (the workspace form's combine
    // finishes in whichever split arrives last)
    const int finisher = step_check && !zero_request ? nsplit - 1 : -1;
    if constexpr (kCluster) {
        if (zero_request || split >= nsplit) {             // no tokens: weight 0
            cluster_finish<kMulti, kWindow>(a, R, kPartialEmpty, part, finisher);
            return;
        }
    }
    if (split >= nsplit)
        return;

    if (zero_request) {                                    // split 0 writes the zeros
        for (int i = threadIdx.x; i < R.nrows * kHeadDim; i += kThreads)
            store_out(a.out, R.id(a, i / kHeadDim) * kHeadDim + i % kHeadDim, 0.f, a.out_fp32);
        return;
    }

    const int64_t t0 = kWindow ? job.t0 : static_cast<int64_t>(split) * a.split_tokens;
    const int64_t t1 = min(len, t0 + (kWindow ? split_tokens : a.split_tokens));
    // page ids of this split (t0 is a multiple of the page size)
    const int n_pages = static_cast<int>((t1 - 1) / ps) - first_page + 1;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kIdsPerThread; ++k) {
        const int i = threadIdx.x + k * kThreads;
        if (i < n_pages) {
            bad |= (ids[k] < 0 || ids[k] >= a.num_pages);
            page_list[i] = ids[k];
        }
    }
    if (threadIdx.x == 0) {
        s_failed = 0;
        s_stale = 0;
        for (int i = 0; i < kWarps * T::kStages; ++i) {
            if (kWindow && !first)
                mbar_inval(&full[i]);
            mbar_init(&full[i], 1);
        }
        fence_mbar_init();
    }
    bad = __syncthreads_or(bad);

    // Fused append (kvq_decode_attn_append): the split holding token len - 1
    // writes that token's codes for KV head kvh into the cache now (when its
    // page id is valid, as kvq_append would) and patches them into its tile
    // when the chunk's copy lands, so its own attention uses them without
    // reading them back.
    int it_new = -1;
    using NewRow = std::conditional_t<kBf16Cache, uint2, uint32_t>;   // a lane's part of the row
    NewRow new_k{}, new_v{};
    int64_t new_row = -1;                                  // cache row of the new token
    if (!kWindow && a.k_new != nullptr && split == nsplit - 1) {
        const int64_t tpos = len - 1;
        const int c_last = static_cast<int>((tpos - t0) / kChunkTokens);
        const int32_t page = page_list[static_cast<int>(tpos / ps) - first_page];
        if (warp == c_last % kWarps && page >= 0 && page < a.num_pages) {
            it_new = c_last / kWarps;
            const int64_t src = (static_cast<int64_t>(b) * a.num_kv_heads + kvh) * kHeadDim + 4 * lane;
            const uint2 xk = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.k_new) + src);
            const uint2 xv = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.v_new) + src);
            new_row = (static_cast<int64_t>(page) * a.num_kv_heads + kvh) * ps + tpos % ps;
            if constexpr (kBf16Cache) {
                new_k = xk;
                new_v = xv;
            } else {
                new_k = encode4_e4m3(xk.x, xk.y, a.k_scale[kvh]);
                new_v = encode4_e4m3(xv.x, xv.y, a.v_scale[kvh]);
            }
            if (step_check) {                              // kept for the end of the step
                reinterpret_cast<NewRow *>(new_tok)[lane] = new_k;
                reinterpret_cast<NewRow *>(new_tok + T::kRowBytes)[lane] = new_v;
            }
        }
    }
    // kvq_decode_step, on the split that holds the new token (the request's
    // last split) once the request's verdict is known: KV head 0 reports
    // it, and a request that passed gets the staged row written.
    auto finish_here = [&](bool stale) {
        if (kvh == 0 && threadIdx.x == 0)
            a.abort_out[b] = stale ? 1 : 0;
        const int64_t tpos = len - 1;
        const int32_t page = page_list[static_cast<int>(tpos / ps) - first_page];
        if (stale || threadIdx.x >= 32 || page < 0 || page >= a.num_pages)
            return;
        const int64_t row = (static_cast<int64_t>(page) * a.num_kv_heads + kvh) * ps + tpos % ps;
        const int ln = threadIdx.x;
        *reinterpret_cast<NewRow *>(static_cast<uint8_t *>(a.k_cache) + row * T::kRowBytes + sizeof(NewRow) * ln) =
            reinterpret_cast<const NewRow *>(new_tok)[ln];
        *reinterpret_cast<NewRow *>(static_cast<uint8_t *>(a.v_cache) + row * T::kRowBytes + sizeof(NewRow) * ln) =
            reinterpret_cast<const NewRow *>(new_tok + T::kRowBytes)[ln];
    };
    auto write_new = [&]() {
        if (new_row < 0)
            return;
        if constexpr (kBf16Cache) {
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.k_cache) + new_row * 256 + 8 * lane) = new_k;
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.v_cache) + new_row * 256 + 8 * lane) = new_v;
        } else {
            *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.k_cache) + new_row * 128 + 4 * lane) = new_k;
            *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.v_cache) + new_row * 128 + 4 * lane) = new_v;
        }
    };
    if (!step_check)                                       // kvq_decode_step: finish_step writes it
        write_new();

    if (bad) {                                             // for kvq_decode_step a failed check
        if constexpr (kCluster) {
            cluster_finish<kMulti, kWindow>(a, R, step_check ? kPartialStale : kPartialInvalid, part, finisher);
            if (split == finisher)                         // this split failed: so did the request
                finish_here(true);
        } else
            drop_split<kMulti, kWindow>(a, R, split, nsplit, reinterpret_cast<float *>(smem),
                       step_check ? kLseStale : kLseInvalid);
        return;
    }

    // ---------------------------------------------------------------- setup
    const int n_chunks = static_cast<int>((t1 - t0 + kChunkTokens - 1) / kChunkTokens);
    const int my_chunks = n_chunks > warp ? (n_chunks - warp + kWarps - 1) / kWarps : 0;
    uint8_t *ring = smem + warp * T::kStages * T::kStageBytes;
    uint64_t *my_full = full + warp * T::kStages;
    const int box_tok = ps < kChunkTokens ? ps : kChunkTokens;
    const int parts = kChunkTokens / box_tok;                       // 1 or 2 copies per tensor
    const uint32_t part_bytes = static_cast<uint32_t>(box_tok * T::kRowBytes);
    // evict-first unless other row blocks of the split read the same pages
    auto make_policy = [&]() {
        return kMulti && a.row_blocks > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
    };
    uint64_t policy = 0;
    if constexpr (!kWindow)
        policy = make_policy();


    // Issue the copies of this warp's local chunk `it`: the whole warp, one
    // copy per lane (lanes 0 .. np - 1 the K parts, np .. 2 np - 1 the V
    // parts), which issues them about twice as fast as one lane in turn.
    auto issue = [&](int it) {
        const int c = warp + it * kWarps;
        const int64_t tok = t0 + static_cast<int64_t>(c) * kChunkTokens;
        const int st = it % T::kStages;
        const int64_t left = t1 - tok;
        const int np = left >= kChunkTokens ? parts : static_cast<int>((left + box_tok - 1) / box_tok);
        if (lane == 0)
            mbar_arrive_expect_tx(&my_full[st], 2u * part_bytes * np);
        __syncwarp();
        if (lane < 2 * np) {
            const int part = lane < np ? lane : lane - np;
            const int64_t ptok = tok + part * box_tok;
            const int32_t page = page_list[static_cast<int>(ptok >> ps_shift) - first_page];
            const int64_t row = (static_cast<int64_t>(page) * a.num_kv_heads + kvh) * ps + (ptok & (ps - 1));
            uint8_t *dst = ring + st * T::kStageBytes + (lane < np ? 0 : T::kBytes) + part * part_bytes;
            tma_load_2d(dst, lane < np ? static_cast<const void *>(&k_map) : static_cast<const void *>(&v_map), 0,
                        static_cast<int32_t>(row * lines_per_tok), &my_full[st], kWindow ? make_policy() : policy);
        }
    };

    const int pro = my_chunks < T::kStages ? my_chunks : T::kStages;
    for (int it = 0; it < pro; ++it)
        issue(it);

    if (step_check) {
        // kvq_decode_step: this split's share of the tag check, its own pages
        // (whose ids are in range here).  The live and expected tags come in
        // by asynchronous copies behind the first bulk copies and are compared
        // once the split has attended: a failure only changes what it
        // publishes.  Thread t copies (and later compares) entries t, t + 128, ...
        const uint32_t *want = a.expected_tags + static_cast<int64_t>(b) * a.max_pages_per_seq + first_page;
#pragma unroll
        for (int k = 0; k < kIdsPerThread; ++k) {
            const int i = threadIdx.x + k * kThreads;
            if (i < n_pages) {
                cp_async_4(tag_live + i, a.page_tags + page_list[i]);
                cp_async_4(tag_want + i, want + i);
            }
        }
        cp_async_commit();
    }

    // Behind the first copies, in one trip: the exponents of the split's
    // blocks, one byte each (through L2: the append that wrote them may have
    // run on this SM beside this CTA), and in the multi-token windowed builds
    // the query rows.
    constexpr int kExpsPerThread = (8192 / kBlockTokens + kThreads - 1) / kThreads;
    [[maybe_unused]] int exps[kExpsPerThread][2];
    if constexpr (kBlocks) {
        const int n_blocks = static_cast<int>((t1 - t0 + kBlockTokens - 1) / kBlockTokens);
        const int bpp_shift = ps_shift - 4;                // blocks per page: ps / 16
#pragma unroll
        for (int k = 0; k < kExpsPerThread; ++k) {
            const int i = threadIdx.x + k * kThreads;
            exps[k][0] = exps[k][1] = 0;                   // the last chunk's second m-tile may hold no token
            if (i < n_blocks) {
                const int64_t at =
                    ((static_cast<int64_t>(page_list[i >> bpp_shift]) * a.num_kv_heads + kvh) << bpp_shift) +
                    (i & ((1 << bpp_shift) - 1));
                exps[k][0] = __ldcg(a.k_exp + at);
                exps[k][1] = __ldcg(a.v_exp + at);
            }
        }
    }
    constexpr bool kMidQ = kWindow && kMulti;
    if constexpr (kMidQ)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
            load_q(nt);
    if constexpr (kBlocks) {
#pragma unroll
        for (int k = 0; k < kExpsPerThread; ++k) {
            const int i = threadIdx.x + k * kThreads;
            if (i < 2 * n_chunks)
                blk_exp[i] = static_cast<uint16_t>(
                    (max(exps[k][0], kReadKeyExpMin) & 0xFF) |
                    (min(max(exps[k][1], kReadValueExpMin), kReadValueExpMax) << 8));
        }
    }

    // Query fragments (mma B operand): lane (gq, tq) holds query row gq of
    // this CTA (with one query token: head gq of the group) at dims 32*tq ..
    // 32*tq+31; k-slot pairs of k-step c map to dims 32*tq + 4*c + {0,1} and
    // {2,3}.
    //
    // FP8 cache: the product runs in f16, whose range is narrower than
    // bf16's.  Each q row is first multiplied by 2^e_h, the power of two that
    // puts its largest magnitude in [2^14, 2^15) (exact: only the exponent
    // changes), so no element overflows and every element within 2^28 of the
    // row's largest keeps all its bits; the score multiplier of head h then
    // carries 2^-e_h.
    uint32_t qf[kNT][8][2];
    int q_exp[kNT];                                        // e of row nt * 8 + gq
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
        q_exp[nt] = 0;
        uint32_t (&w)[16] = q_raw[nt];
        if constexpr (!kEarlyQ && !kMidQ)
            load_q(nt);
        float q_mul = 1.f;
        if constexpr (!kBf16Cache) {
            uint32_t mx = 0;                               // largest |q| of the row, as bf16 bits
#pragma unroll
            for (int i = 0; i < 16; ++i)
                mx = max(mx, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            q_exp[nt] = row_pow2_exponent(mx);
            q_mul = __int_as_float((127 + q_exp[nt]) << 23);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if constexpr (kBf16Cache) {
                    qf[nt][c][j] = w[2 * c + j];
                } else {
                    const float2 f = bf16x2_to_f32x2(w[2 * c + j]);
                    qf[nt][c][j] = f32x2_to_f16x2(f.x * q_mul, f.y * q_mul);
                }
            }
        }
    }

    const float kscale = kBf16Cache || kBlocks ? 1.f : read_plain(a.k_scale + kvh);
    const float vscale = kBf16Cache || kBlocks ? 1.f : read_plain(a.v_scale + kvh);
    // score multiplier (log2 domain) of the two query heads 2tq, 2tq + 1
    // whose scores this lane holds: the softmax scale, the K scale and the
    // undoing of their q rows' power-of-two scaling
    float qk_col[kNT][2];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int e = __shfl_sync(0xFFFFFFFFu, q_exp[nt], 4 * (2 * tq + j));
            qk_col[nt][j] = a.qk_scale_log2 * kscale * __int_as_float((127 - e) << 23);
        }
    // Causal limit of those two rows: query token i sees the positions below
    // len - n_query + 1 + i (with one query token: all of them), kept as a
    // count from the split's start, at most one chunk past its end.  Below
    // full_end every row of the CTA sees every token.
    [[maybe_unused]] int vis_col[kNT][2] = {};
    [[maybe_unused]] int64_t full_end = t1;
    if constexpr (kMulti && !kWindow) {
        const int64_t vis0 = len - a.n_query + 1;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int64_t v = vis0 + (R.row0 + nt * kMaxGroup + 2 * tq + j) / g - t0;
                vis_col[nt][j] = static_cast<int>(
                    v < -1 ? -1 : (v > a.split_tokens + kChunkTokens ? a.split_tokens + kChunkTokens : v));
            }
        full_end = min(t1, vis0 + R.row0 / g);
    }
    // Windowed builds keep less in registers, counts from the split's start
    // (t0) all: query token i of the call sees the positions below vis0 + i
    // but for those from sink_end to win + i; the tokens i of this lane's score
    // columns lie in a nibble each of tok_col.  V rows that no row of the CTA
    // sees (sink_end up to win_first) are zeroed, so what they hold cannot
    // reach the product.  Below full_to and outside [sink_end, mask_hi) no
    // token is masked.
    [[maybe_unused]] uint32_t tok_col = 0;
    [[maybe_unused]] int vis0 = 0, sink_end = 0, full_to = 0;
    [[maybe_unused]] int win = -2 * kChunkTokens, win_first = win, mask_hi = win;      // window 0: before everything
    if constexpr (kWindow) {
        auto rel = [&](int64_t v) {                        // query tokens are at most 15 further on
            v -= t0;
            const int64_t most = split_tokens + 2 * kChunkTokens;
            return static_cast<int>(v < -2 * kChunkTokens ? -2 * kChunkTokens : (v > most ? most : v));
        };
        const int first = kMulti ? R.row0 / g : 0, last = kMulti ? (R.row0 + R.nrows - 1) / g : 0;
        vis0 = rel(len - a.n_query + 1);
        full_to = rel(min(t1, len - a.n_query + 1 + first));
        if constexpr (kMulti)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    tok_col |= static_cast<uint32_t>(min((R.row0 + nt * kMaxGroup + 2 * tq + j) / g, 15))
                               << (4 * (2 * nt + j));
        if (a.window > 0) {
            win = rel(win0);
            sink_end = rel(a.num_sinks);
            win_first = rel(win0 + first);
            mask_hi = rel(win0 + last);
        }
    }
    if constexpr (kSmemQ) {                                // each warp stores a quarter of the fragments
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            if (kk / 2 == warp)
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
                    q_frag[(kk * kNT + nt) * 32 + lane] = make_uint2(qf[nt][kk][0], qf[nt][kk][1]);
    }
    if constexpr (kBlocks || kSmemQ)
        __syncthreads();                                   // the exponents and fragments are in place

    // The windowed and block-scaled builds over FP8 keep weights, sums and
    // accumulators 2^15 times larger (the quotient is the same, and f16 ends at
    // 65504): an f16 weight, and with it the second term of the precise form,
    // is then cut at 2^-39 of the largest weight instead of 2^-24.  A bf16
    // cache's weights are bf16 terms, whose range needs no lift, and its values
    // (up to 2^128) leave no room for one.
    constexpr float kLift = kWindow && !kBf16Cache ? 15.f : 0.f;
    // 16-bit terms of a weight in the PV product: one for bf16 output (f16
    // 2^-12, for a bf16 cache bf16 2^-9: an output of many tokens averages
    // them below its own 2^-9; a second bf16 term cost 2 to 10 %), for fp32
    // output two f16 terms (2^-24) or two bf16 ones (2^-18), in the windowed
    // builds three (2^-27).
    constexpr int kTerms = !kPreciseP ? 1 : kWindow && kBf16Cache ? 3 : 2;
    // For fp32 output a tile's products are summed from zero and added to O
    // by fp32 additions that round: the tensor core cuts what it adds to a
    // large accumulator, always towards zero (error against fp64, 64 requests
    // of up to 5,000 tokens: bf16 cache 1.6e-6, 3.9e-7 so; FP8 9.9e-7, 3.7e-7).
    constexpr bool kSumApart = kWindow && kPreciseP;
    float m_run[kNT][2], l_run[kNT][2];
    float o[kNT][8][4];
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
        m_run[nt][0] = m_run[nt][1] = -INFINITY;
        l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }

    bool failed = false;
    int it = 0;
    for (; it < my_chunks; ++it) {
        const int st = it % T::kStages;
        // every lane polls; the warp gives up as one if any lane did
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&my_full[st], (it / T::kStages) & 1, a.copy_wait_ns))) {
            failed = true;
            break;
        }
        if (it == 0 && warp == 0)
            KVQ_STAMP(2);
        const uint8_t *ks = ring + st * T::kStageBytes;
        const uint8_t *vs = ks + T::kBytes;
        const int c = warp + it * kWarps;
        const int64_t tok = t0 + static_cast<int64_t>(c) * kChunkTokens;
        if (it == it_new) {                  // fused append: the new token's row
            const int r = static_cast<int>(len - 1 - tok);
            uint8_t *kt = ring + st * T::kStageBytes;
            uint8_t *vt = kt + T::kBytes;
            if constexpr (kBf16Cache) {
                const uint32_t off = swz(2 * r + (lane >> 4), (lane & 15) >> 1) + 8 * (lane & 1);
                *reinterpret_cast<uint2 *>(kt + off) = new_k;
                *reinterpret_cast<uint2 *>(vt + off) = new_v;
            } else {
                const uint32_t off = swz(r, lane >> 2) + 4 * (lane & 3);
                *reinterpret_cast<uint32_t *>(kt + off) = new_k;
                *reinterpret_cast<uint32_t *>(vt + off) = new_v;
            }
            __syncwarp();
        }
        const int64_t left = t1 - tok;
        const int n_valid = left < kChunkTokens ? static_cast<int>(left) : kChunkTokens;   // V rows
        [[maybe_unused]] int s_valid[kNT][2];            // tokens of the chunk each score column sees
        if constexpr (!kWindow)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    s_valid[nt][j] = kMulti ? min(n_valid, vis_col[nt][j] - c * kChunkTokens) : n_valid;
        [[maybe_unused]] float blk_mul[2], blk_add[2];     // 2^ek and ev of the two 16-token m-tiles
        if constexpr (kBlocks) {
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                const int e = static_cast<int16_t>(blk_exp[2 * c + mt]);
                blk_mul[mt] = __int_as_float((127 + static_cast<int8_t>(e & 0xFF)) << 23);
                blk_add[mt] = static_cast<float>(e >> 8);
            }
        }

        // The chunk's arithmetic; a full chunk (every token valid, the
        // common case) is compiled without the masking of tail tokens.
        auto chunk = [&](auto full) {
            constexpr bool kFull = decltype(full)::value;
            // ---- S^T = K Q^T for the two 16-token m-tiles; each K fragment,
            // converted once, feeds every n-tile of query rows
            float sc[kNT][2][4];
            if constexpr (kSmemQ && !kBf16Cache) {
                // both m-tiles together: a fragment of Q is read once for four products
                uint32_t kw[2][2][8];
    #pragma unroll
                for (int mt = 0; mt < 2; ++mt)
    #pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int r = mt * 16 + half * 8 + gq;
                        const uint4 xa = lds128(ks, swz(r, 2 * tq)), xb = lds128(ks, swz(r, 2 * tq + 1));
                        uint32_t(&w)[8] = kw[mt][half];
                        w[0] = xa.x; w[1] = xa.y; w[2] = xa.z; w[3] = xa.w;
                        w[4] = xb.x; w[5] = xb.y; w[6] = xb.z; w[7] = xb.w;
                    }
    #pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
    #pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
                        sc[nt][mt][0] = sc[nt][mt][1] = sc[nt][mt][2] = sc[nt][mt][3] = 0.f;
    #pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    uint2 qv[kNT];
    #pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
                        qv[nt] = q_frag[(kk * kNT + nt) * 32 + lane];
    #pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const uint32_t k0 = lo16_e4m3x2_to_f16x2(kw[mt][0][kk]), k1 = lo16_e4m3x2_to_f16x2(kw[mt][1][kk]);
                        const uint32_t k2 = hi16_e4m3x2_to_f16x2(kw[mt][0][kk]), k3 = hi16_e4m3x2_to_f16x2(kw[mt][1][kk]);
    #pragma unroll
                        for (int nt = 0; nt < kNT; ++nt)
                            mma_f16(sc[nt][mt], k0, k1, k2, k3, qv[nt].x, qv[nt].y);
                    }
                }
            } else {
    #pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
    #pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
                    sc[nt][mt][0] = sc[nt][mt][1] = sc[nt][mt][2] = sc[nt][mt][3] = 0.f;
                const int r0 = mt * 16 + gq, r1 = r0 + 8;
                if constexpr (kBf16Cache) {
                    uint32_t w0[16], w1[16];
    #pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int line0 = 2 * r0 + (tq >> 1), line1 = 2 * r1 + (tq >> 1);
                        const uint4 x0 = lds128(ks, swz(line0, (tq & 1) * 4 + j));
                        const uint4 x1 = lds128(ks, swz(line1, (tq & 1) * 4 + j));
                        w0[4 * j] = x0.x; w0[4 * j + 1] = x0.y; w0[4 * j + 2] = x0.z; w0[4 * j + 3] = x0.w;
                        w1[4 * j] = x1.x; w1[4 * j + 1] = x1.y; w1[4 * j + 2] = x1.z; w1[4 * j + 3] = x1.w;
                    }
    #pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
    #pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) {
                            uint2 qv;
                            if constexpr (kSmemQ)
                                qv = q_frag[(kk * kNT + nt) * 32 + lane];
                            else
                                qv = make_uint2(qf[nt][kk][0], qf[nt][kk][1]);
                            mma_bf16(sc[nt][mt], w0[2 * kk], w1[2 * kk], w0[2 * kk + 1], w1[2 * kk + 1], qv.x, qv.y);
                        }
                } else {
                    const uint4 x0a = lds128(ks, swz(r0, 2 * tq)), x0b = lds128(ks, swz(r0, 2 * tq + 1));
                    const uint4 x1a = lds128(ks, swz(r1, 2 * tq)), x1b = lds128(ks, swz(r1, 2 * tq + 1));
                    const uint32_t w0[8] = {x0a.x, x0a.y, x0a.z, x0a.w, x0b.x, x0b.y, x0b.z, x0b.w};
                    const uint32_t w1[8] = {x1a.x, x1a.y, x1a.z, x1a.w, x1b.x, x1b.y, x1b.z, x1b.w};
    #pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t k0 = lo16_e4m3x2_to_f16x2(w0[kk]), k1 = lo16_e4m3x2_to_f16x2(w1[kk]);
                        const uint32_t k2 = hi16_e4m3x2_to_f16x2(w0[kk]), k3 = hi16_e4m3x2_to_f16x2(w1[kk]);
    #pragma unroll
                        for (int nt = 0; nt < kNT; ++nt)
                            mma_f16(sc[nt][mt], k0, k1, k2, k3, qf[nt][kk][0], qf[nt][kk][1]);
                    }
                }
            }
            }

            // ---- online softmax (log2 domain); lane holds rows nt*8 + 2tq, +1
            float alpha[kNT][2];
    #pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                float mx[2] = {-INFINITY, -INFINITY};
    #pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    [[maybe_unused]] float mul[2];
                    if constexpr (kBlocks) {
                        mul[0] = qk_col[nt][0] * blk_mul[mt];
                        mul[1] = qk_col[nt][1] * blk_mul[mt];
                    }
    #pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = mt * 16 + gq + ((i & 2) ? 8 : 0);
                        float x;
                        if constexpr (kBlocks)
                            x = fmaf(sc[nt][mt][i], mul[i & 1], blk_add[mt]);
                        else
                            x = sc[nt][mt][i] * qk_col[nt][i & 1];
                        bool keep = true;
                        if constexpr (kWindow && !kFull) {
                            const int at = c * kChunkTokens + row, ti = (tok_col >> (4 * (2 * nt + (i & 1)))) & 15;
                            keep = row < n_valid && at < vis0 + ti && !(at >= sink_end && at < win + ti);
                        } else if constexpr (!kFull) {
                            keep = row < s_valid[nt][i & 1];
                        }
                        x = keep ? x : -INFINITY;
                        sc[nt][mt][i] = x;
                        mx[i & 1] = fmaxf(mx[i & 1], x);
                    }
                }
                float base[2];
    #pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float mnew = fmaxf(m_run[nt][j], warp_max_over_rows(mx[j]));
                    base[j] = mnew == -INFINITY ? 0.f : mnew;
                    alpha[nt][j] = fast_exp2(m_run[nt][j] - base[j]);
                    m_run[nt][j] = mnew;
                }
                const float lift[2] = {base[0] - kLift, base[1] - kLift};
                float psum[2] = {0.f, 0.f};
    #pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    [[maybe_unused]] float tsum[2] = {0.f, 0.f};
    #pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = fast_exp2(sc[nt][mt][i] - lift[i & 1]);
                        sc[nt][mt][i] = p;
                        if constexpr (kBlocks)
                            tsum[i & 1] += p;
                        else
                            psum[i & 1] += p;
                    }
                    if constexpr (kBlocks) {               // back to the softmax's own weights: times 2^-ev
                        const float undo = __int_as_float((127 - static_cast<int>(blk_add[mt])) << 23);
                        psum[0] = fmaf(tsum[0], undo, psum[0]);
                        psum[1] = fmaf(tsum[1], undo, psum[1]);
                    }
                }
    #pragma unroll
                for (int j = 0; j < 2; ++j)
                    l_run[nt][j] = l_run[nt][j] * alpha[nt][j] + psum[j];
    #pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[nt][i][0] *= alpha[nt][0];
                    o[nt][i][1] *= alpha[nt][1];
                    o[nt][i][2] *= alpha[nt][0];
                    o[nt][i][3] *= alpha[nt][1];
                }
            }

            // ---- O^T += V^T P^T; each V fragment, converted once, feeds
            // every n-tile
    #pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                // a weight as the sum of kTerms 16-bit terms, each carrying
                // what the rounding of those before it dropped
                uint32_t pb0[kNT], pb1[kNT];
                [[maybe_unused]] uint32_t pl0[kNT], pl1[kNT], pm0[kNT], pm1[kNT];
    #pragma unroll
                for (int nt = 0; nt < kNT; ++nt) {
                    uint32_t x0, x1;
                    if constexpr (kBf16Cache) {
                        x0 = f32x2_to_bf16x2(sc[nt][mt][0], sc[nt][mt][1]);
                        x1 = f32x2_to_bf16x2(sc[nt][mt][2], sc[nt][mt][3]);
                    } else {
                        x0 = f32x2_to_f16x2(sc[nt][mt][0], sc[nt][mt][1]);
                        x1 = f32x2_to_f16x2(sc[nt][mt][2], sc[nt][mt][3]);
                    }
                    pb0[nt] = movmatrix_trans(x0);
                    pb1[nt] = movmatrix_trans(x1);
                    if constexpr (kTerms > 1) {
                        const float2 h0 = kBf16Cache ? bf16x2_to_f32x2(x0) : f16x2_to_f32x2(x0);
                        const float2 h1 = kBf16Cache ? bf16x2_to_f32x2(x1) : f16x2_to_f32x2(x1);
                        const float *p = sc[nt][mt];
                        const uint32_t y0 = kBf16Cache ? f32x2_to_bf16x2(p[0] - h0.x, p[1] - h0.y)
                                                       : f32x2_to_f16x2(p[0] - h0.x, p[1] - h0.y);
                        const uint32_t y1 = kBf16Cache ? f32x2_to_bf16x2(p[2] - h1.x, p[3] - h1.y)
                                                       : f32x2_to_f16x2(p[2] - h1.x, p[3] - h1.y);
                        pl0[nt] = movmatrix_trans(y0);
                        pl1[nt] = movmatrix_trans(y1);
                        if constexpr (kTerms > 2) {
                            const float2 l0 = bf16x2_to_f32x2(y0), l1 = bf16x2_to_f32x2(y1);
                            pm0[nt] = movmatrix_trans(f32x2_to_bf16x2(p[0] - h0.x - l0.x, p[1] - h0.y - l0.y));
                            pm1[nt] = movmatrix_trans(f32x2_to_bf16x2(p[2] - h1.x - l1.x, p[3] - h1.y - l1.y));
                        }
                    }
                }
                // V rows of token slots 2tq, 2tq+1, 2tq+8, 2tq+9 of this m-tile
                const int rv = mt * 16 + 2 * tq;
                const int rows[4] = {rv, rv + 1, rv + 8, rv + 9};
                if constexpr (kBf16Cache) {
                    uint32_t R[4][8];
    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int line = 2 * rows[q] + (gq >> 2);
                        const uint4 lo = lds128(vs, swz(line, (gq & 3) * 2));
                        const uint4 hi = lds128(vs, swz(line, (gq & 3) * 2 + 1));
                        bool keep = kFull || rows[q] < n_valid;
                        if constexpr (kWindow && !kFull)
                            keep = keep && !(c * kChunkTokens + rows[q] >= sink_end && c * kChunkTokens + rows[q] < win_first);
                        R[q][0] = keep ? lo.x : 0u; R[q][1] = keep ? lo.y : 0u;
                        R[q][2] = keep ? lo.z : 0u; R[q][3] = keep ? lo.w : 0u;
                        R[q][4] = keep ? hi.x : 0u; R[q][5] = keep ? hi.y : 0u;
                        R[q][6] = keep ? hi.z : 0u; R[q][7] = keep ? hi.w : 0u;
                    }
    #pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t a0 = prmt(R[0][i], R[1][i], 0x5410);
                        const uint32_t a1 = prmt(R[0][i], R[1][i], 0x7632);
                        const uint32_t a2 = prmt(R[2][i], R[3][i], 0x5410);
                        const uint32_t a3 = prmt(R[2][i], R[3][i], 0x7632);
    #pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) {
                            if constexpr (kSumApart) {
                                float t[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_bf16(t, a0, a1, a2, a3, pm0[nt], pm1[nt]);
                                mma_bf16(t, a0, a1, a2, a3, pl0[nt], pl1[nt]);
                                mma_bf16(t, a0, a1, a2, a3, pb0[nt], pb1[nt]);
    #pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    o[nt][i][q] += t[q];
                            } else {
                                mma_bf16(o[nt][i], a0, a1, a2, a3, pb0[nt], pb1[nt]);
                                if constexpr (kTerms > 1)
                                    mma_bf16(o[nt][i], a0, a1, a2, a3, pl0[nt], pl1[nt]);
                            }
                        }
                    }
                } else {
                    uint32_t R[4][4];
    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 v = lds128(vs, swz(rows[q], gq));
                        bool keep = kFull || rows[q] < n_valid;
                        if constexpr (kWindow && !kFull)
                            keep = keep && !(c * kChunkTokens + rows[q] >= sink_end && c * kChunkTokens + rows[q] < win_first);
                        R[q][0] = keep ? v.x : 0u; R[q][1] = keep ? v.y : 0u;
                        R[q][2] = keep ? v.z : 0u; R[q][3] = keep ? v.w : 0u;
                    }
    #pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
                        const uint32_t p01 = prmt(R[0][i >> 1], R[1][i >> 1], sel);
                        const uint32_t p23 = prmt(R[2][i >> 1], R[3][i >> 1], sel);
                        const uint32_t a0 = lo16_e4m3x2_to_f16x2(p01), a1 = hi16_e4m3x2_to_f16x2(p01);
                        const uint32_t a2 = lo16_e4m3x2_to_f16x2(p23), a3 = hi16_e4m3x2_to_f16x2(p23);
    #pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) {
                            if constexpr (kSumApart) {
                                float t[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_f16(t, a0, a1, a2, a3, pl0[nt], pl1[nt]);
                                mma_f16(t, a0, a1, a2, a3, pb0[nt], pb1[nt]);
    #pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    o[nt][i][q] += t[q];
                            } else {
                                mma_f16(o[nt][i], a0, a1, a2, a3, pb0[nt], pb1[nt]);
                                if constexpr (kTerms > 1)
                                    mma_f16(o[nt][i], a0, a1, a2, a3, pl0[nt], pl1[nt]);
                            }
                        }
                    }
                }
            }
        };
        const int chunk_end = (c + 1) * kChunkTokens;
        if (kWindow ? chunk_end <= full_to && (chunk_end <= sink_end || chunk_end - kChunkTokens >= mask_hi)
                    : tok + kChunkTokens <= full_end)
            chunk(std::true_type{});
        else
            chunk(std::false_type{});

        // ---- refill this stage with the chunk kStages ahead
        __syncwarp();
        if (it + T::kStages < my_chunks) {
            fence_proxy_async_smem();
            issue(it + T::kStages);
        }
    }

    if (failed) {
        // Drain the copies this warp still has in flight -- the one it gave
        // up on and those issued after it -- with the full limit, so none
        // lands in shared memory after the CTA has moved on.  A drain that
        // gives up too is reported as bit 1.
        if (lane == 0) {
            atomicOr(&g_device_error, 1u);
            s_failed = 1;
        }
        const int issued = my_chunks < it + T::kStages ? my_chunks : it + T::kStages;
        bool drained = true;
        for (int j = it; j < issued; ++j)
            drained &= mbar_wait_bounded(&my_full[j % T::kStages], (j / T::kStages) & 1, kCopyWaitLimitNs);
        if (!drained && lane == 0)
            atomicOr(&g_device_error, 2u);
    }
    if (step_check) {                                      // this thread's tag entries
        cp_async_wait_all();
        bool stale = false;
#pragma unroll
        for (int k = 0; k < kIdsPerThread; ++k) {
            const int i = threadIdx.x + k * kThreads;
            if (i < n_pages)
                stale |= tag_live[i] != tag_want[i];
        }
        if (stale)
            s_stale = 1;
    }
    __syncthreads();
    KVQ_STAMP(3);
    if (s_stale || s_failed) {                             // a failed check outranks a timeout
        if constexpr (kCluster) {
            const bool stale = cluster_finish<kMulti, kWindow>(a, R, s_stale ? kPartialStale : kPartialInvalid, part, finisher);
            if (split == finisher)
                finish_here(stale);
        } else
            drop_split<kMulti, kWindow>(a, R, split, nsplit, reinterpret_cast<float *>(smem),
                       s_stale ? kLseStale : kLseInvalid);
        return;
    }

    // ---- merge the four warps' states in shared memory (ring is free now)
    float *sm_o = reinterpret_cast<float *>(smem);                     // [kWarps][kRowsT][128]
    float *sm_m = sm_o + kWarps * kRowsT * kMergeStride;              // [kWarps][kRowsT]
    float *sm_l = sm_m + kWarps * kRowsT;                             // [kWarps][kRowsT]
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            l_run[nt][j] = warp_sum_over_rows(l_run[nt][j]);
    {
        float *ow = sm_o + warp * kRowsT * kMergeStride;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            const int r = nt * kMaxGroup + 2 * tq;                  // rows r, r + 1 of this lane
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = merge_col(16 * gq + 2 * i);
                *reinterpret_cast<float2 *>(ow + r * kMergeStride + c) = make_float2(o[nt][i][0], o[nt][i][2]);
                *reinterpret_cast<float2 *>(ow + (r + 1) * kMergeStride + c) =
                    make_float2(o[nt][i][1], o[nt][i][3]);
            }
            if (gq == 0) {
                sm_m[warp * kRowsT + r] = m_run[nt][0];
                sm_m[warp * kRowsT + r + 1] = m_run[nt][1];
                sm_l[warp * kRowsT + r] = l_run[nt][0];
                sm_l[warp * kRowsT + r + 1] = l_run[nt][1];
            }
        }
    }
    __syncthreads();

    // per-row merge factors of the four warps, computed once (thread h)
    float *sm_f = sm_l + kWarps * kRowsT;                             // [kRowsT][kWarps] weights
    float *sm_t = sm_f + kRowsT * kWarps;                             // [kRowsT] 1 / sum, [kRowsT] lse
    if (threadIdx.x < R.nrows) {
        const int h = threadIdx.x;
        float mmax = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            mmax = fmaxf(mmax, sm_m[w * kRowsT + h]);
        float lsum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = sm_m[w * kRowsT + h];
            const float f = mw == -INFINITY ? 0.f : fast_exp2(mw - mmax);
            sm_f[h * kWarps + w] = f;
            lsum += sm_l[w * kRowsT + h] * f;
        }
        // a row that saw no token of this split (causal limit): weight 0
        if constexpr (kWindow) {
            sm_t[h] = lsum == 0.f ? 0.f : vscale / lsum;
            sm_t[kRowsT + h] = lsum == 0.f ? -INFINITY : lsum == lsum ? mmax + __log2f(lsum) - kLift : INFINITY;
        } else {
            sm_t[h] = lsum > 0.f ? vscale / lsum : 0.f;
            sm_t[kRowsT + h] = lsum > 0.f ? mmax + __log2f(lsum) : -INFINITY;
        }
    }
    __syncthreads();
    if constexpr (kWindow) {
        // warp w takes rows w, w + 4, ..; a lane four dims of each
        const int d = 4 * lane, c = merge_col(d);
#pragma unroll
        for (int q = 0; q < kRowsT / kWarps; ++q) {
            const int h = warp + q * kWarps;
            if (h >= R.nrows)
                break;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float *row = sm_o + (w * kRowsT + h) * kMergeStride + c;
                const float2 lo = *reinterpret_cast<const float2 *>(row), hi = *reinterpret_cast<const float2 *>(row + 2);
                const float f = sm_f[h * kWarps + w];
                acc.x += lo.x * f;
                acc.y += lo.y * f;
                acc.z += hi.x * f;
                acc.w += hi.y * f;
            }
            const float t = sm_t[h];
            acc = make_float4(acc.x * t, acc.y * t, acc.z * t, acc.w * t);
            if constexpr (kCluster) {
                *reinterpret_cast<float4 *>(part + kRowsT + h * kHeadDim + d) = acc;
                if (lane == 0)
                    part[h] = sm_t[kRowsT + h];
            } else if (!kSharing && nsplit == 1) {
                store_out4(a.out, R.ids[h] * kHeadDim + d, acc, a.out_fp32);
            } else {
                const int64_t at = R.part(a, h, split);
                *reinterpret_cast<float4 *>(a.ws_o + at * kHeadDim + d) = acc;
                if (lane == 0)
                    a.ws_lse[at] = sm_t[kRowsT + h];
            }
        }
    } else
    for (int d = threadIdx.x; d < kHeadDim; d += kThreads)
#pragma unroll
    for (int h = 0; h < kRowsT; ++h) {
        if (h >= R.nrows)
            break;
        float acc = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            acc += sm_o[(w * kRowsT + h) * kMergeStride + merge_col(d)] * sm_f[h * kWarps + w];
        const float val = acc * sm_t[h];
        const int64_t bh = R.id(a, h);
        if constexpr (kCluster) {
            part[kRowsT + h * kHeadDim + d] = val;
            if (d == 0)
                part[h] = sm_t[kRowsT + h];
        } else if (nsplit == 1) {
            store_out(a.out, bh * kHeadDim + d, val, a.out_fp32);
        } else {
            a.ws_o[(bh * a.max_splits + split) * kHeadDim + d] = val;
            if (d == 0)
                a.ws_lse[bh * a.max_splits + split] = sm_t[kRowsT + h];
        }
    }
    KVQ_STAMP(4);
    if constexpr (kCluster) {
        const bool stale = cluster_finish<kMulti, kWindow>(a, R, kPartialOk, part, finisher);
        if (split == finisher)
            finish_here(stale);
    } else if (nsplit > 1) {
        publish_and_combine<kMulti, kWindow>(a, R, nsplit, reinterpret_cast<float *>(smem) + (kMulti ? 0 : kScratchOffset));
    } else if (step_check) {                               // one split: its own verdict
        finish_here(false);
    }
    KVQ_STAMP(6);
