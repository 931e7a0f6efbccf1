"""Cases of the block-scaled cache and of the windowed reads, with the operators' plain forms.

Operators (``case["op"]``):

  append_blocks  quantise-on-append into an e4m3 cache with one power-of-two
                 exponent per (16-token block, KV head), K and V
  attn_blocks    decode attention over that cache, n new query tokens per
                 request, with or without a window
  attn_window    decode attention with a sliding window and a few first tokens
                 that stay visible, over an e4m3 cache with per-head scales or
                 a bf16 cache
  tag_window     the per-page tag check of windowed requests
  copy_pages     pages of every layer's caches copied inside the pool

Where ``own`` is false ``run`` computes them with elementary torch operations;
where it is true it calls the library.
"""
import math
import random

import torch

own = False

DEV = "cuda"
D = 128
BLOCK = 16
E_MIN, E_MAX = -48, 48
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one chat request, a short context: launch latency
        dict(name="blocks_tiny", op="attn_blocks", batch=1, hkv=8, g=1, ps=16, lo=512, hi=512, n=1,
             window=0, sinks=0, fp32=False),
        # drafts of several tokens verified for a mixed batch
        dict(name="blocks_verify", op="attn_blocks", batch=16, hkv=8, g=4, ps=64, lo=1024, hi=16384, n=4,
             window=0, sinks=0, fp32=False),
        # a few very long documents: the largest case
        dict(name="blocks_long", op="attn_blocks", batch=4, hkv=8, g=2, ps=64, lo=131072, hi=1048576, n=1,
             window=0, sinks=0, fp32=False),
        # the same cache with a window, odd sizes, fp32 output
        dict(name="blocks_windowed", op="attn_blocks", batch=8, hkv=4, g=5, ps=32, lo=700, hi=9001, n=1,
             window=2047, sinks=5, fp32=True),
        # serving a mixed batch with a window of 4,096 and four sinks
        dict(name="window_ragged", op="attn_window", batch=64, hkv=8, g=4, ps=64, lo=1024, hi=32768, n=1,
             window=4096, sinks=4, fp32=False, bf16=False),
        # draft verification over a bf16 cache, lengths below and above the window
        dict(name="window_verify_bf16", op="attn_window", batch=8, hkv=2, g=8, ps=16, lo=40, hi=8193, n=7,
             window=1000, sinks=3, fp32=False, bf16=True),
        # a batch of chats, page ids of 16 tokens
        dict(name="tags_small", op="tag_window", batch=32, ps=16, lo=8193, hi=8193, n=1, window=4096, sinks=4),
        # a full batch of long contexts
        dict(name="tags_large", op="tag_window", batch=256, ps=16, lo=2048, hi=65536, n=1, window=32768, sinks=64),
        # the append of a decode step
        dict(name="append_decode", op="append_blocks", batch=64, hkv=8, ps=16, lo=1, hi=8192, new_lo=1, new_hi=1),
        # chunks of prompts of several requests
        dict(name="append_prompts", op="append_blocks", batch=16, hkv=8, ps=64, lo=1, hi=16384, new_lo=1,
             new_hi=8192),
        # 64 requests forked: the last page of each, 16 layers
        dict(name="copy_fork", op="copy_pages", layers=16, pages=4096, listed=64, hkv=8, ps=16, bf16=False),
        # half of a pool moved, one layer
        dict(name="copy_move", op="copy_pages", layers=1, pages=8192, listed=4001, hkv=8, ps=64, bf16=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_blocks", "attn_blocks", "attn_blocks", "attn_window", "attn_window", "tag_window",
                     "append_blocks", "append_blocks", "copy_pages"])
    ps = rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    if op in ("attn_blocks", "attn_window"):
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, min(65536, max(1, 2000000 // (batch * hkv))))
        case = dict(op=op, batch=batch, hkv=hkv, g=rng.randint(1, 8), ps=ps, lo=rng.randint(1, hi), hi=hi,
                    n=rng.choice([1, 1, 1, 1, 2, 3, 4, 5, 8, 11, 16]), window=_log(rng, 1, 20000),
                    sinks=rng.choice([0, 1, 4, 5, 16, 64, 100]), fp32=rng.random() < 0.25)
        if op == "attn_window":
            case["bf16"] = rng.random() < 0.4
        elif rng.random() < 0.6:
            case["window"] = case["sinks"] = 0
        return case
    if op == "tag_window":
        hi = _log(rng, 1, 65536)
        return dict(op=op, batch=_log(rng, 24, 256), ps=ps, lo=rng.randint(1, hi), hi=hi, n=rng.randint(1, 16),
                    window=_log(rng, 1, 40000), sinks=rng.choice([0, 1, 4, 17, 64, 200]))
    if op == "append_blocks":
        batch = _log(rng, 1, 64)
        new_hi = rng.choice([1, 1, rng.randint(2, 16), _log(rng, 16, 100000 // batch)])
        return dict(op=op, batch=batch, hkv=hkv, ps=ps, lo=1, hi=max(new_hi, _log(rng, 16, 8192)),
                    new_lo=1 if new_hi == 1 else rng.randint(0, new_hi - 1), new_hi=new_hi)
    pages = _log(rng, 8, 16384 * 16 // ps)
    layers = max(1, min(32, int(2 ** 31 // (pages * ps * hkv * D * 2))))
    return dict(op=op, layers=rng.randint(1, layers), pages=pages, listed=rng.randint(1, pages // 2), hkv=hkv,
                ps=ps, bf16=rng.random() < 0.3)


def _lens(case):
    """Context lengths, the same for every seed."""
    r = random.Random(1000003 * case["batch"] + case["hi"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def _new_tokens(case):
    """(context length, new tokens) of each request of an append; the lengths count the new tokens."""
    r = random.Random(7 * case["batch"] + case["hi"])
    out = []
    for _ in range(case["batch"]):
        n = r.randint(case["new_lo"], case["new_hi"])
        out.append((max(n, r.randint(case["lo"], case["hi"])), n))
    return out


def _up(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _table(lens, ps, gen, spare):
    """Pages of each request at distinct random places of the pool; -1 past a request's pages."""
    counts = [max(1, _up(x, ps)) for x in lens]
    maxp, total = max(counts), sum(counts)
    pool = total + spare
    perm = torch.randperm(pool, generator=gen, device=DEV)[:total].to(torch.int32)
    cnt = torch.tensor(counts, device=DEV)
    used = torch.arange(maxp, device=DEV)[None, :] < cnt[:, None]
    bt = torch.full((len(lens), maxp), -1, dtype=torch.int32, device=DEV)
    bt[used] = perm
    return bt, pool


def _normal(shape, gen, outliers=True):
    x = torch.randn(shape, generator=gen, device=DEV)
    if outliers:
        x = torch.where(torch.rand(shape, generator=gen, device=DEV) < 0.01, x * 8, x)
    return x


def _pages(pool, hkv, ps, gen, bf16=False):
    """Random cache contents, made in pieces: bf16 values, or e4m3 codes (as bytes) of values whose largest
    magnitude in a block of 16 tokens is near the format's."""
    out = torch.empty((pool, hkv, ps, D), dtype=torch.bfloat16 if bf16 else torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (hkv * ps * D))
    for at in range(0, pool, step):
        x = torch.randn((min(step, pool - at), hkv, ps, D), generator=gen, device=DEV)
        out[at:at + step] = x.bfloat16() if bf16 else (x * 90).clamp(-448, 448).to(F8).view(torch.uint8)
    return out


def _exponents(pool, hkv, ps, gen):
    """Exponents of blocks whose values are of the order of 1, a few blocks far larger or smaller."""
    shape = (pool, hkv, ps // BLOCK)
    e = torch.randint(-9, -5, shape, generator=gen, device=DEV)
    far = torch.randint(-14, -2, shape, generator=gen, device=DEV)
    return torch.where(torch.rand(shape, generator=gen, device=DEV) < 0.05, far, e).to(torch.int8)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = _generator(seed)
    op, ps = case["op"], case["ps"]
    st = dict(case=case)
    if op in ("attn_blocks", "attn_window"):
        lens, hkv = _lens(case), case["hkv"]
        bf16 = bool(case.get("bf16"))
        st["bt"], pool = _table(lens, ps, gen, 3)
        st["seq"] = _int32(lens)
        st["k"], st["v"] = (_pages(pool, hkv, ps, gen, bf16) for _ in range(2))
        st["q"] = _normal((case["batch"], case["n"], hkv * case["g"], D), gen, False).bfloat16()
        if op == "attn_blocks":
            st["ke"], st["ve"] = (_exponents(pool, hkv, ps, gen) for _ in range(2))
        else:
            st["ks"], st["vs"] = (torch.rand(hkv, generator=gen, device=DEV) * 0.01 + 0.006 for _ in range(2))
    elif op == "tag_window":
        lens = _lens(case)
        st["bt"], pool = _table(lens, ps, gen, 64)
        st["seq"] = _int32(lens)
        st["tags"] = torch.randint(0, 1 << 31, (pool,), generator=gen, device=DEV).to(torch.int32)
        st["expected"] = torch.where(st["bt"] >= 0, st["tags"][st["bt"].clamp(min=0).long()], 0)
        # pages outside the window were given to others; some requests hold one stale page somewhere
        first, last = _entries(case, st["seq"])
        idx = torch.arange(st["bt"].shape[1], device=DEV)[None, :]
        hole = (idx >= first[:, None]) & (idx < last[:, None])
        st["expected"] = torch.where(hole, st["expected"] ^ 5, st["expected"]).to(torch.int32)
        pick = torch.rand((len(lens), 1), generator=gen, device=DEV) * ((st["seq"] + ps - 1) // ps)[:, None]
        stale = (idx == pick.long()) & (torch.rand((len(lens), 1), generator=gen, device=DEV) < 0.5)
        st["expected"] = torch.where(stale, st["expected"] ^ 3, st["expected"]).to(torch.int32)
    elif op == "append_blocks":
        pairs, hkv = _new_tokens(case), case["hkv"]
        st["bt"], pool = _table([p[0] for p in pairs], ps, gen, 3)
        st["seq"] = _int32([p[0] for p in pairs])
        offsets = [0]
        for p in pairs:
            offsets.append(offsets[-1] + p[1])
        st["offsets"] = None if case["new_lo"] == case["new_hi"] == 1 else _int32(offsets)
        st["most"] = case["new_hi"]
        st["k"], st["v"] = (_pages(pool, hkv, ps, gen) for _ in range(2))
        st["ke"], st["ve"] = (_exponents(pool, hkv, ps, gen) for _ in range(2))
        st["k_new"], st["v_new"] = (_normal((offsets[-1], hkv, D), gen).bfloat16() for _ in range(2))
    else:
        layers, pages, hkv = case["layers"], case["pages"], case["hkv"]
        st["caches"] = _pages(layers * 2 * pages, hkv, ps, gen, case["bf16"]).view(
            layers * 2, pages, hkv, ps, D)
        st["exps"] = None if case["bf16"] else _exponents(layers * 2 * pages, hkv, ps, gen).view(
            layers * 2, pages, hkv, ps // BLOCK)
        perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
        st["src"] = perm[:case["listed"]].contiguous()
        st["dst"] = perm[case["listed"]:2 * case["listed"]].contiguous()
    if own:
        _prepare_own(st)
    return st


def _desc(st, pages, bf16):
    import fp8_quantised_paged_kv_gb300 as kvq
    c = st["case"]
    return kvq.CacheDesc(pages, c["ps"], c["hkv"], D, kvq.KVQ_CACHE_BF16 if bf16 else kvq.KVQ_CACHE_FP8_E4M3)


def _prepare_own(st):
    """What a user's program keeps beside the inputs: the descriptor, the workspace and the output."""
    import fp8_quantised_paged_kv_gb300 as kvq
    c = st["case"]
    if c["op"] in ("attn_blocks", "attn_window"):
        st["desc"] = _desc(st, st["k"].shape[0], c.get("bf16"))
        make = kvq.workspace_for_blocks if c["op"] == "attn_blocks" else kvq.workspace_for_window
        st["ws"] = make(st["desc"], c["batch"], c["n"], c["hkv"] * c["g"], st["bt"].shape[1], c["window"],
                        c["sinks"], device=DEV)
        st["out"] = torch.empty(st["q"].shape, dtype=torch.float32 if c["fp32"] else torch.bfloat16, device=DEV)
    elif c["op"] == "tag_window":
        st["abort"] = torch.empty(c["batch"], dtype=torch.uint8, device=DEV)
    elif c["op"] == "append_blocks":
        st["desc"] = _desc(st, st["k"].shape[0], False)
    else:
        st["desc"] = _desc(st, c["pages"], c["bf16"])
        st["cache_list"] = list(st["caches"].unbind(0))
        st["exp_list"] = [] if st["exps"] is None else list(st["exps"].unbind(0))


# -------------------------------------------------------------------- runs

def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _own_blocks(st):
    import fp8_quantised_paged_kv_gb300 as kvq
    c = st["case"]
    return kvq.kvq_decode_attn_blocks(st["desc"], st["q"], st["k"], st["v"], st["ke"], st["ve"], st["bt"],
                                      st["seq"], 1 / math.sqrt(D), c["window"], c["sinks"], None, st["out"],
                                      st["ws"])


def _own_window(st):
    import fp8_quantised_paged_kv_gb300 as kvq
    c = st["case"]
    return kvq.kvq_decode_attn_window(st["desc"], st["q"], st["k"], st["v"], st["ks"], st["vs"], st["bt"],
                                      st["seq"], 1 / math.sqrt(D), c["window"], c["sinks"], None, st["out"],
                                      st["ws"])


def _own_tags(st):
    import fp8_quantised_paged_kv_gb300 as kvq
    c = st["case"]
    kvq.kvq_tag_check_window(st["bt"], st["expected"], st["seq"], c["ps"], st["tags"], c["window"], c["sinks"],
                             c["n"], st["abort"])
    return st["abort"]


def _own_append(st):
    import fp8_quantised_paged_kv_gb300 as kvq
    kvq.kvq_append_blocks(st["desc"], st["k_new"], st["v_new"], st["offsets"], st["bt"], st["seq"], None,
                          st["k"], st["v"], st["ke"], st["ve"])
    return st["k"].view(F8), st["v"].view(F8), st["ke"], st["ve"]


def _own_copy(st):
    import fp8_quantised_paged_kv_gb300 as kvq
    kvq.kvq_copy_pages(st["desc"], st["cache_list"], st["exp_list"], st["src"], st["dst"])
    return _copied(st)


def _copied(st):
    if st["exps"] is None:
        return st["caches"]
    return st["caches"].view(F8), st["exps"]


def _gather(cache, bt):
    """A request's tokens in order: [B][Hkv][pages * ps][...]."""
    x = cache[bt.clamp(min=0).long()]                       # [B][P][Hkv][ps][...]
    x = x.transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], x.shape[2] * x.shape[3], *x.shape[4:])


def _values(st, name):
    """The cache's values as the request sees them, fp32 [B][Hkv][L][D]."""
    codes = _gather(st[name], st["bt"])
    if codes.dtype == torch.bfloat16:
        return codes.float()
    x = codes.view(F8).float()
    if name + "e" in st:
        scale = _pow2(_gather(st[name + "e"], st["bt"]))
        return (x.view(*scale.shape, BLOCK, D) * scale[..., None, None]).view(x.shape)
    return x * st[name + "s"][None, :, None, None]


def _pow2(e):
    """2^e in fp32, exactly (e within [-126, 127])."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_attention(st):
    c = st["case"]
    B, n, hkv, g = c["batch"], c["n"], c["hkv"], c["g"]
    k = _values(st, "k")
    L = k.shape[2]
    q = st["q"].float().view(B, n, hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, n * g, D)
    s = torch.matmul(q, k.transpose(2, 3)) * (1 / math.sqrt(D))
    del k
    pos = st["seq"].long()[:, None] - n + torch.arange(n, device=DEV)[None, :]            # [B][n]
    j = torch.arange(L, device=DEV)
    see = j[None, None, :] <= pos[:, :, None]
    if c["window"]:
        see &= (j < c["sinks"])[None, None, :] | (j[None, None, :] > pos[:, :, None] - c["window"])
    see = see[:, None, :, None, :].expand(B, 1, n, g, L).reshape(B, 1, n * g, L)
    s = torch.where(see, s, -math.inf)
    m = s.amax(dim=3, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(dim=3, keepdim=True)
    o = torch.matmul(p, _values(st, "v")) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(B, hkv, n, g, D).permute(0, 2, 1, 3, 4).reshape(B, n, hkv * g, D)
    return o if c["fp32"] else o.bfloat16()


def _entries(case, seq):
    """Table entries [first, last) of each request that hold no visible token."""
    length = seq.long().clamp(min=0)
    ps = case["ps"]
    first = (length.clamp(max=case["sinks"]) + ps - 1) // ps
    last = (length - case["n"] + 1 - case["window"]).clamp(min=0) // ps
    return first, torch.maximum(first, last)


def _plain_tags(st):
    bt, c = st["bt"], st["case"]
    first, last = _entries(c, st["seq"])
    used = (st["seq"].long().clamp(min=0) + c["ps"] - 1) // c["ps"]
    i = torch.arange(bt.shape[1], device=DEV)[None, :]
    look = (i < used[:, None]) & ((i < first[:, None]) | (i >= last[:, None]))
    fine = (bt >= 0) & (bt < st["tags"].shape[0])
    live = st["tags"][torch.where(fine, bt, 0).long()]
    bad = (look & (~fine | (live != st["expected"]))).any(dim=1) | (used > bt.shape[1])
    return bad.to(torch.uint8)


def _plain_append(st):
    """Every block that holds a new token, laid out densely [request][block][16 tokens]."""
    c = st["case"]
    ps, hkv, B = c["ps"], c["hkv"], c["batch"]
    T = st["k_new"].shape[0]
    if st["offsets"] is None:
        off = torch.arange(B + 1, device=DEV) * (T // B)
    else:
        off = st["offsets"].long()
    count = off[1:] - off[:-1]
    start = st["seq"].long() - count
    M = (st["most"] + 2 * BLOCK - 2) // BLOCK
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(off[1:].contiguous(), t, right=True)
    pos = start[r] + t - off[r]
    dense = (r * M + pos // BLOCK - start[r] // BLOCK) * BLOCK + pos % BLOCK
    written = torch.zeros(B * M * BLOCK, dtype=torch.bool, device=DEV)
    written[dense] = True
    written = written.view(B * M, BLOCK)
    at = torch.nonzero(written.any(dim=1)).flatten()       # the blocks that get a token
    written = written[at]
    block = (start[:, None] // BLOCK + torch.arange(M, device=DEV)[None, :]).view(-1)[at]
    page = st["bt"][at // M, block * BLOCK // ps].long()
    sub = block % (ps // BLOCK)
    older = block * BLOCK < start[at // M]                  # holds earlier tokens
    row = block[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)[None, :]
    earlier = row < start[at // M][:, None]
    results = []
    for name in ("k", "v"):
        x = torch.zeros((B * M * BLOCK, hkv, D), device=DEV)
        x[dense] = st[name + "_new"].float()
        x = x.view(B * M, BLOCK, hkv, D)[at]
        need = _exponent(x.abs().amax(dim=(1, 3)))          # [blocks][Hkv]
        exps = st[name + "e"]
        e_old = exps[page, :, sub].long()
        e = torch.where(older[:, None], torch.maximum(e_old, need), need)
        view = st[name].view(-1, hkv, ps // BLOCK, BLOCK, D)
        codes = view[page, :, sub]                          # [blocks][Hkv][16][D]
        moved = codes.view(F8).float() * _pow2(torch.where(older[:, None], e_old - e, 0))[..., None, None]
        fresh = x.transpose(1, 2) * _pow2(-e)[..., None, None]
        values = torch.where(written[:, None, :, None], fresh, moved).clamp(-448, 448).to(F8).view(torch.uint8)
        keep = (written | earlier)[:, None, :, None]
        view[page, :, sub] = torch.where(keep, values, codes)
        exps[page, :, sub] = e.to(torch.int8)
        results += [st[name].view(F8), exps]
    return results[0], results[2], results[1], results[3]


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, within [-48, 48]."""
    m, x = torch.frexp(amax)                                # amax = m * 2^x, 0.5 <= m < 1
    e = x.long() - 9 + (m > 0.875).long()
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _plain_copy(st):
    src, dst = st["src"].long(), st["dst"].long()
    words = st["caches"].view(torch.int64)
    words[:, dst] = words[:, src]
    if st["exps"] is not None:
        st["exps"][:, dst] = st["exps"][:, src]
    return _copied(st)


_plain = dict(attn_blocks=_plain_attention, attn_window=_plain_attention, tag_window=_plain_tags,
              append_blocks=_plain_append, copy_pages=_plain_copy)
_own = dict(attn_blocks=_own_blocks, attn_window=_own_window, tag_window=_own_tags, append_blocks=_own_append,
            copy_pages=_own_copy)


# -------------------------------------------------------------------- work

def _visible(case):
    """(positions that some query of the request sees, pairs of query and position) over the batch."""
    seen = pairs = 0
    n, w, s = case["n"], case["window"], case["sinks"]
    for length in _lens(case):
        lowest = length
        sink = 0
        for i in range(n):
            p = length - n + i
            if p < 0:
                continue
            low = max(0, p - w + 1) if w else 0
            few = min(s, low) if w else 0
            pairs += p + 1 - low + few
            lowest, sink = min(lowest, low), max(sink, few)
        seen += length - lowest + min(sink, lowest)
    return seen, pairs


def work(case):
    op, ps = case["op"], case["ps"]
    if op in ("attn_blocks", "attn_window"):
        seen, pairs = _visible(case)
        hkv, rows = case["hkv"], case["batch"] * case["n"] * case["hkv"] * case["g"]
        per = 2 * D * (2 if case.get("bf16") else 1) + (2 / BLOCK if op == "attn_blocks" else 0)
        return dict(bytes=seen * hkv * per + seen / ps * 4 + rows * D * (2 + (4 if case["fp32"] else 2)),
                    flops=4.0 * D * case["g"] * hkv * pairs)
    if op == "tag_window":
        entries = _up(_visible(case)[0], ps)
        return dict(bytes=entries * 12 + case["batch"] * 5, flops=2.0 * entries)
    if op == "append_blocks":
        pairs = _new_tokens(case)
        tokens = sum(p[1] for p in pairs)
        blocks = sum(_up(p[0], BLOCK) - (p[0] - p[1]) // BLOCK for p in pairs if p[1])
        row = case["hkv"] * D * 2
        return dict(bytes=tokens * row * 3 + blocks * case["hkv"] * 2 + len(pairs) * 8, flops=4.0 * tokens * row)
    page = case["hkv"] * ps * D * (2 if case["bf16"] else 1) + (0 if case["bf16"] else case["hkv"] * ps // BLOCK)
    return dict(bytes=2.0 * page * case["listed"] * case["layers"] * 2 + case["listed"] * 8, flops=0.0)


# ------------------------------------------------------------------- exact

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("attn_blocks", "attn_window"):
        return _exact_attention(st)
    if op == "append_blocks":
        return _exact_append(st)
    return None                                             # whole numbers and copies


def _e4m3_table():
    """The 256 codes' values in 64 bits, from the format's definition."""
    out = []
    for c in range(256):
        field, mant = (c >> 3) & 15, c & 7
        v = math.nan if field == 15 and mant == 7 else (
            mant * 2.0 ** -9 if field == 0 else (8 + mant) * 2.0 ** (field - 10))
        out.append(-v if c & 128 else v)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _powers():
    """2^(i - 128) at place i, 64 bits."""
    return torch.tensor([2.0 ** i for i in range(-128, 129)], dtype=torch.float64, device=DEV)


def _exact_attention(st):
    """Request by request and head by head, the visible positions picked out before anything is computed."""
    c, table, power = st["case"], _e4m3_table(), _powers()
    n, g, hkv, ps = c["n"], c["g"], c["hkv"], c["ps"]
    bf16 = bool(c.get("bf16"))
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    for b, length in enumerate(_lens(c)):
        for h in range(hkv):
            for i in range(n):
                p = length - n + i
                if p < 0:
                    continue
                j = torch.arange(p + 1, device=DEV)
                if c["window"]:
                    j = j[(j < c["sinks"]) | (p - j < c["window"])]
                page, at = st["bt"][b].long()[j // ps], j % ps
                kv = []
                for name in ("k", "v"):
                    x = st[name][page, h, at]
                    if bf16:
                        kv.append(x.double())
                    elif name + "e" in st:
                        kv.append(table[x.long()] * power[st[name + "e"][page, h, at // BLOCK].long() + 128][:, None])
                    else:
                        kv.append(table[x.long()] * st[name + "s"][h].double())
                s = kv[0] @ st["q"][b, i, h * g:(h + 1) * g].double().T / math.sqrt(D)      # [positions][g]
                s = torch.softmax(s, dim=0)
                out[b, i, h * g:(h + 1) * g] = s.T @ kv[1]
    return out


def _exact_append(st):
    """Block by block: the exponent from the largest magnitude, then the nearest code (ties to even)."""
    c, table, power = st["case"], _e4m3_table(), _powers()
    ps, hkv = c["ps"], c["hkv"]
    pairs = _new_tokens(c)
    if sum(p[1] for p in pairs) > 150000:
        return None
    grid = torch.sort(table[(table >= 0) & ~torch.isnan(table)])[0].unique()
    mid = (grid[1:] + grid[:-1]) / 2

    def nearest(x):
        a = x.abs().clamp(max=448.0)
        lo = torch.searchsorted(mid, a)                     # a on a midpoint: the lower neighbour
        tie = (lo < mid.numel()) & (mid[lo.clamp(max=mid.numel() - 1)] == a) & (lo % 2 == 1)
        return torch.sign(x) * grid[lo + tie.long()]        # even codes are the even places

    caches = {k: table[st[k].long()] for k in ("k", "v")}
    exps = {k: st[k + "e"].clone() for k in ("k", "v")}
    at = 0
    for b, (length, n) in enumerate(pairs):
        pos = length - n
        while pos < length:
            end = min(length, (pos // BLOCK + 1) * BLOCK)
            page, sub, lo = int(st["bt"][b, pos // ps]), pos % ps // BLOCK, pos % ps // BLOCK * BLOCK
            for k in ("k", "v"):
                x = st[k + "_new"][at:at + end - pos].double().transpose(0, 1)       # [Hkv][tokens][D]
                amax = x.abs().amax(dim=(1, 2)).clamp(min=2.0 ** -60)
                need = torch.ceil(torch.log2(amax / 448.0))
                need = torch.where(power[need.long() + 127] * 448.0 >= amax, need - 1, need)
                need = need.clamp(E_MIN, E_MAX)
                e = need
                if pos % BLOCK:
                    old = exps[k][page, :, sub].double()
                    e = torch.maximum(old, need)
                    rows = caches[k][page, :, lo:lo + pos % BLOCK]
                    caches[k][page, :, lo:lo + pos % BLOCK] = nearest(
                        rows * power[(old - e).long() + 128][:, None, None])
                caches[k][page, :, pos % ps:pos % ps + end - pos] = nearest(
                    x * power[128 - e.long()][:, None, None])
                exps[k][page, :, sub] = e.to(torch.int8)
            at += end - pos
            pos = end
    return caches["k"], caches["v"], exps["k"], exps["v"]
