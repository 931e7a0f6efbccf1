"""Cases of the shared-prefix attention and of the page tables kept on the GPU, with the operators' plain forms.

Operators (``case["op"]``):

  prefix   decode attention of requests of which several share their first
           pages, n new query tokens per request: over an e4m3 cache with
           per-head scales or a bf16 cache (kvq_decode_attn_prefix), or over
           the block-scaled cache (kvq_decode_attn_prefix_blocks)
  tables   the rows of a block table on the GPU: forked onto other rows'
           pages (kvq_fork_tables), given pages and slots for new tokens
           (kvq_extend_tables), and trimmed (kvq_trim_tables), one pass after
           which every row holds again what it held before

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
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases

def listed():
    return [
        # four samples of one short prompt: launch latency
        dict(name="prefix_tiny", op="prefix", kind="fp8", batch=4, groups=1, hkv=8, g=1, ps=16, plo=512, phi=512,
             lo=16, hi=16, n=1, fp32=False),
        # 64 chats behind one system prompt
        dict(name="prefix_chat", op="prefix", kind="fp8", batch=64, groups=1, hkv=8, g=4, ps=64, plo=8192, phi=8192,
             lo=100, hi=2000, n=1, fp32=False),
        # two long documents, 64 questions on each: the largest case
        dict(name="prefix_long", op="prefix", kind="fp8", batch=128, groups=2, hkv=8, g=8, ps=64, plo=30000,
             phi=32768, lo=1, hi=2000, n=1, fp32=False),
        # samples of a few prompts, odd sizes, fp32 output
        dict(name="prefix_sampling", op="prefix", kind="fp8", batch=33, groups=5, hkv=4, g=5, ps=32, plo=700,
             phi=9001, lo=1, hi=700, n=1, fp32=True),
        # drafts of five tokens verified behind one document, over a bf16 cache
        dict(name="prefix_verify_bf16", op="prefix", kind="bf16", batch=16, groups=1, hkv=2, g=8, ps=16, plo=16001,
             phi=16001, lo=5, hi=900, n=5, fp32=False),
        # agents that start from three prompts, over a bf16 cache, fp32 output
        dict(name="prefix_bf16", op="prefix", kind="bf16", batch=24, groups=3, hkv=8, g=2, ps=64, plo=1000, phi=6000,
             lo=1, hi=3000, n=1, fp32=True),
        # the block-scaled cache: eight prompts, several answers to each
        dict(name="prefix_blocks", op="prefix", kind="blocks", batch=64, groups=8, hkv=8, g=4, ps=64, plo=4096,
             phi=16384, lo=1, hi=1000, n=1, fp32=False),
        # the same cache, drafts of three tokens, one prompt, fp32 output
        dict(name="prefix_blocks_verify", op="prefix", kind="blocks", batch=13, groups=1, hkv=4, g=3, ps=16, plo=5003,
             phi=5003, lo=3, hi=200, n=3, fp32=True),
        # a decode step of drafts that are all rejected
        dict(name="tables_draft", op="tables", batch=64, ps=16, lo=1, hi=8192, new_lo=4, new_hi=4, parents=0, spare=1.0),
        # a batch of prompts admitted, and finished
        dict(name="tables_admit", op="tables", batch=256, ps=16, lo=0, hi=0, new_lo=1, new_hi=8192, parents=0,
             spare=1.0),
        # 60 samples forked from four long prompts, one token each
        dict(name="tables_fork", op="tables", batch=64, ps=16, lo=2000, hi=32768, new_lo=1, new_hi=1, parents=4,
             spare=1.0),
        # prompts and forks that a nearly full pool cannot all hold
        dict(name="tables_scarce", op="tables", batch=101, ps=64, lo=1, hi=3000, new_lo=0, new_hi=999, parents=7,
             spare=0.6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    ps = rng.choice([16, 32, 64, 128])
    if rng.random() < 0.7:
        hkv, g = rng.choice([1, 2, 4, 8]), rng.randint(1, 8)
        kind = rng.choice(["fp8", "fp8", "bf16", "blocks"])
        batch = _log(rng, 1, 128)
        groups = min(batch, _log(rng, 1, 16))
        tokens = (600000 if kind == "bf16" else 1200000) // hkv        # in the cache
        phi = _log(rng, 32, max(33, min(32768, tokens // (2 * groups), 20000000 // (batch * hkv))))
        hi = _log(rng, 1, max(1, min(4096, tokens // (2 * batch))))
        n = rng.choice([1, 1, 1, 2, 3, 4, 5, 8, 11, 16])
        n = max(1, min(n, 240000000 // (batch * hkv * g * (phi + hi))))
        return dict(op="prefix", kind=kind, batch=batch, groups=groups, hkv=hkv, g=g, ps=ps, plo=rng.randint(1, phi),
                    phi=phi, lo=rng.randint(0, hi), hi=hi, n=n, fp32=rng.random() < 0.3)
    batch = _log(rng, 1, 256)
    parents = rng.choice([0, rng.randint(0, batch // 2)])
    hi = rng.choice([0, _log(rng, 1, 32768)])
    new_hi = rng.choice([1, rng.randint(2, 16), _log(rng, 16, 8192)])
    return dict(op="tables", batch=batch, ps=ps, lo=rng.randint(0, hi), hi=hi, new_lo=rng.randint(0 if batch > 8 else 1, new_hi),
                new_hi=new_hi, parents=parents if hi else 0, spare=rng.choice([1.0, 1.0, rng.uniform(0.1, 0.95)]))


def _up(a, b):
    return -(-a // b)


def _groups(case):
    """(first request, requests, prefix length) of each group, and every request's context length: the same for
    every seed."""
    r = random.Random(1000003 * case["batch"] + 31 * case["phi"] + case["hi"])
    cuts = sorted(r.sample(range(1, case["batch"]), case["groups"] - 1)) if case["groups"] > 1 else []
    edges = [0] + cuts + [case["batch"]]
    groups, lens = [], []
    for a, b in zip(edges, edges[1:]):
        p = r.randint(case["plo"], case["phi"])
        groups.append((a, b - a, p))
        lens += [p + r.randint(case["lo"], case["hi"]) for _ in range(b - a)]
    return groups, lens


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pages(pool, hkv, ps, gen, bf16):
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


def _prepare_prefix(case, gen):
    groups, lens = _groups(case)
    ps, hkv, kind = case["ps"], case["hkv"], case["kind"]
    maxp = max(1, _up(max(lens), ps))
    rows, copies, used = [], [], 0
    leader, shared = [], []
    for first, m, p in groups:
        whole = p // ps if m > 1 else 0                    # pages that the group shares
        prefix = list(range(used, used + whole))
        used += whole
        for r in range(first, first + m):
            mine = _up(lens[r], ps) - whole
            rows.append(prefix + list(range(used, used + mine)))
            if m > 1 and r > first and p % ps:             # a copy of the page in which the prefix ends
                copies.append((rows[first][whole], used))
            used += mine
            leader.append(first if m > 1 else -1)
            shared.append(p if m > 1 else 0)
    pool = used + 3
    perm = torch.randperm(pool, generator=gen, device=DEV)
    bt = torch.tensor([x + [-1] * (maxp - len(x)) for x in rows], device=DEV)
    st = dict(case=case, bt=torch.where(bt >= 0, perm[bt.clamp(min=0)], -1).to(torch.int32), seq=_int32(lens),
              leader=_int32(leader), shared=_int32(shared))
    st["k"], st["v"] = (_pages(pool, hkv, ps, gen, kind == "bf16") for _ in range(2))
    names = ["k", "v"]
    if kind == "blocks":
        st["ke"], st["ve"] = (_exponents(pool, hkv, ps, gen) for _ in range(2))
        names += ["ke", "ve"]
    else:
        st["ks"], st["vs"] = (torch.rand(hkv, generator=gen, device=DEV) * 0.01 + 0.006 for _ in range(2))
    if copies:
        c = perm[torch.tensor(copies, device=DEV)]
        for name in names:
            st[name][c[:, 1]] = st[name][c[:, 0]]
    st["q"] = torch.randn((case["batch"], case["n"], hkv * case["g"], D), generator=gen, device=DEV).bfloat16()
    return st


def _table_plan(case):
    """(length, new tokens, parent, length forked) of each request before the pass, the same for every seed.  A forked
    request is empty before."""
    r = random.Random(7 * case["batch"] + case["hi"] + 13 * case["new_hi"])
    out = []
    for i in range(case["batch"]):
        new = r.randint(case["new_lo"], case["new_hi"])
        if case["parents"] and i >= case["parents"]:
            p = r.randrange(case["parents"])
            out.append((0, new, p, r.randint(max(0, out[p][0] - 100), out[p][0])))
        else:
            out.append((r.randint(case["lo"], case["hi"]), new, -1, 0))
    return out


def _prepare_tables(case, gen):
    plan, ps, B = _table_plan(case), case["ps"], case["batch"]
    held = [_up(p[0], ps) for p in plan]
    final = [_up((p[3] if p[2] >= 0 else p[0]) + p[1], ps) for p in plan]
    fresh = sum(f - (p[3] // ps if p[2] >= 0 else h) for f, h, p in zip(final, held, plan))
    free = max(1, int(fresh * case["spare"]) + (64 if case["spare"] >= 1 else 0))
    pool, maxp, used = sum(held) + free, max(1, max(final)), sum(held)
    perm = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    cnt = torch.tensor(held, device=DEV)
    st = dict(case=case, seq=_int32([p[0] for p in plan]), parents=_int32([p[2] for p in plan]),
              fork=_int32([p[3] for p in plan]), keep=_int32([p[0] for p in plan]))
    bt = torch.full((B, maxp), -1, dtype=torch.int32, device=DEV)
    mask = torch.arange(maxp, device=DEV)[None, :] < cnt[:, None]
    bt[mask] = perm[:used]
    st["bt"] = bt
    st["tags"] = torch.randint(0, 1 << 31, (pool,), generator=gen, device=DEV).to(torch.int32)
    st["expected"] = torch.where(bt >= 0, st["tags"][bt.clamp(min=0).long()], 0).to(torch.int32)
    st["refs"] = torch.zeros(pool, dtype=torch.int32, device=DEV)
    st["refs"][perm[:used].long()] = 1
    st["free"] = torch.zeros(pool, dtype=torch.int32, device=DEV)
    st["free"][:free] = perm[used:]
    st["count"] = _int32([free])
    offsets = [0]
    for p in plan:
        offsets.append(offsets[-1] + p[1])
    even = case["new_lo"] == case["new_hi"]
    st["offsets"], st["tokens"] = None if even else _int32(offsets), offsets[-1]
    return st


def prepare(case, seed):
    gen = _generator(seed)
    st = _prepare_prefix(case, gen) if case["op"] == "prefix" else _prepare_tables(case, gen)
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    """What a user's program keeps beside the inputs: descriptors, workspaces and outputs."""
    import fp8_quantised_paged_kv_gb300 as kvq
    c = st["case"]
    if c["op"] == "prefix":
        kind = kvq.KVQ_CACHE_BF16 if c["kind"] == "bf16" else kvq.KVQ_CACHE_FP8_E4M3
        st["desc"] = kvq.CacheDesc(st["k"].shape[0], c["ps"], c["hkv"], D, kind)
        st["ws"] = kvq.workspace_for_prefix(st["desc"], c["batch"], c["n"], c["hkv"] * c["g"], st["bt"].shape[1],
                                            device=DEV)
        st["out"] = torch.empty(st["q"].shape, dtype=torch.float32 if c["fp32"] else torch.bfloat16, device=DEV)
    else:
        st["pool"] = kvq.PagePool(st["tags"].shape[0], c["ps"], st["free"], st["count"], st["refs"], st["tags"])
        st["slots"] = torch.empty(st["tokens"], dtype=torch.int64, device=DEV)
        st["forked"], st["served"] = (torch.empty(c["batch"], dtype=torch.uint8, device=DEV) for _ in range(2))
        st["src"], st["dst"] = (torch.empty(c["batch"], dtype=torch.int32, device=DEV) for _ in range(2))


# -------------------------------------------------------------------- runs

def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _own_prefix(st):
    import fp8_quantised_paged_kv_gb300 as kvq
    blocks = st["case"]["kind"] == "blocks"
    call = kvq.kvq_decode_attn_prefix_blocks if blocks else kvq.kvq_decode_attn_prefix
    a, b = ("ke", "ve") if blocks else ("ks", "vs")
    return call(st["desc"], st["q"], st["k"], st["v"], st[a], st[b], st["bt"], st["seq"], st["leader"], st["shared"],
                1 / math.sqrt(D), None, st["out"], st["ws"])


def _own_tables(st):
    import fp8_quantised_paged_kv_gb300 as kvq
    if st["case"]["parents"]:
        kvq.kvq_fork_tables(st["pool"], st["parents"], st["fork"], st["seq"], st["bt"], st["expected"], st["src"],
                            st["dst"], st["forked"])
    kvq.kvq_extend_tables(st["pool"], st["offsets"], st["tokens"], st["seq"], st["bt"], st["expected"], st["slots"],
                          st["served"])
    got = _of_tables(st, st["slots"], st["served"])
    if st["case"]["parents"]:
        got += [st["src"], st["dst"], st["forked"]]
    kvq.kvq_trim_tables(st["pool"], st["keep"], st["seq"], st["bt"])
    return got + [st["bt"], st["seq"], st["refs"], st["free"], st["count"]]


def _of_tables(st, slots, served):
    """What a pass leaves behind of the tables' middle state: the tags say which pages the rows were given."""
    return [slots, served, st["expected"], st["tags"]]


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


def _plain_prefix(st):
    """Every request over its own row of the table: shared pages hold the same for all that name them."""
    c = st["case"]
    B, n, hkv, g = c["batch"], c["n"], c["hkv"], c["g"]
    k = _values(st, "k")
    L = k.shape[2]
    q = st["q"].float().view(B, n, hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, n * g, D)
    s = torch.matmul(q, k.transpose(2, 3)) * (1 / math.sqrt(D))
    del k
    pos = st["seq"].long()[:, None] - n + torch.arange(n, device=DEV)[None, :]            # [B][n]
    see = torch.arange(L, device=DEV)[None, None, :] <= pos[:, :, None]
    see = see[:, None, :, None, :].expand(B, 1, n, g, L).reshape(B, 1, n * g, L)
    s = torch.where(see, s, -math.inf)
    m = s.amax(dim=3, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(dim=3, keepdim=True)
    o = torch.matmul(p, _values(st, "v")) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(B, hkv, n, g, D).permute(0, 2, 1, 3, 4).reshape(B, n, hkv * g, D)
    return o if c["fp32"] else o.bfloat16()


def _ceil(x, ps):
    return (x + ps - 1) // ps


def _put(into, at, what, where):
    """into[at] = what where `where` holds, without asking the GPU how many those are."""
    spare = torch.cat([into, into.new_zeros(1)])
    spare[torch.where(where, at, into.shape[0]).reshape(-1)] = what.to(into.dtype).reshape(-1)
    into.copy_(spare[:-1])


def _plain_fork(st):
    ps, bt, seq = st["case"]["ps"], st["bt"], st["seq"].long()
    B, maxp = bt.shape
    parent, L = st["parents"].long(), st["fork"].long()
    of = parent.clamp(0, B - 1)
    fine = (parent >= 0) & (parent < B) & (parent != torch.arange(B, device=DEV)) & (seq == 0) & (L >= 0) & (L <= seq[of])
    whole, part = L // ps, fine & (L % ps > 0)
    upto = torch.cumsum(part.long(), 0)
    ok = fine & (~part | (upto <= st["count"].long()))
    part &= ok
    i = torch.arange(maxp, device=DEV)[None, :]
    theirs = bt[of]
    copied = ok[:, None] & (i < whole[:, None])
    fresh = part[:, None] & (i == whole[:, None])
    page = st["free"][(st["count"].long() - upto).clamp(min=0)].long()                    # [B]
    st["refs"].index_add_(0, theirs.clamp(min=0).reshape(-1).long(), copied.reshape(-1).int())
    _put(st["tags"], page, st["tags"][page] + 1, part)
    _put(st["refs"], page, torch.ones_like(page), part)
    src = torch.where(part, theirs.gather(1, whole.clamp(max=maxp - 1)[:, None])[:, 0], -1)
    dst = torch.where(part, page, -1).to(torch.int32)
    st["expected"].copy_(torch.where(copied, st["expected"][of],
                                     torch.where(fresh, st["tags"][page][:, None], st["expected"])))
    bt.copy_(torch.where(copied, theirs, torch.where(fresh, page[:, None].int(), bt)))
    st["seq"].copy_(torch.where(ok, L, seq))
    st["count"] -= part.sum().int()
    return [src.to(torch.int32), dst, ((parent >= 0) & ~ok).to(torch.uint8)]


def _plain_extend(st):
    ps, bt, old, T = st["case"]["ps"], st["bt"], st["seq"].long(), st["tokens"]
    B, maxp = bt.shape
    off = torch.arange(B + 1, device=DEV) * (T // B) if st["offsets"] is None else st["offsets"].long()
    new = old + off[1:] - off[:-1]
    have = _ceil(old, ps)
    fits = new <= maxp * ps
    need = torch.where(fits, _ceil(new, ps) - have, 0)
    upto = torch.cumsum(need, 0)
    ok = fits & ((need == 0) | (upto <= st["count"].long()))
    i = torch.arange(maxp, device=DEV)[None, :]
    taken = ok[:, None] & (i >= have[:, None]) & (i < (have + need)[:, None])
    at = st["count"].long() - 1 - ((upto - need - have)[:, None] + i)
    page = st["free"][torch.where(taken, at, 0)].long()
    _put(st["tags"], page, st["tags"][page] + 1, taken)
    _put(st["refs"], page, torch.ones_like(page), taken)
    bt.copy_(torch.where(taken, page.int(), bt))
    st["expected"].copy_(torch.where(taken, st["tags"][page], st["expected"]))
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(off[1:].contiguous(), t, right=True)
    pos = old[r] + t - off[r]
    slot = bt[r, (pos // ps).clamp(max=maxp - 1)].long() * ps + pos % ps
    slots = torch.where(ok[r], slot, -1)
    st["seq"].copy_(torch.where(ok, new, old))
    st["count"] -= torch.where(ok, need, 0).sum().int()
    return slots, (~ok).to(torch.uint8)


def _plain_trim(st):
    ps, bt, seq, keep = st["case"]["ps"], st["bt"], st["seq"].long(), st["keep"].long()
    act = (keep >= 0) & (keep < seq)
    i = torch.arange(bt.shape[1], device=DEV)[None, :]
    drop = act[:, None] & (i >= _ceil(keep, ps)[:, None]) & (i < _ceil(seq, ps)[:, None])
    less = torch.zeros_like(st["refs"]).index_add_(0, bt.clamp(min=0).reshape(-1).long(), (drop & (bt >= 0)).reshape(-1).int())
    freed = (st["refs"] > 0) & (less >= st["refs"])
    st["refs"].copy_((st["refs"] - less).clamp(min=0))
    at = st["count"].long() + torch.cumsum(freed.long(), 0) - 1
    _put(st["free"], at, torch.arange(freed.shape[0], device=DEV), freed)
    st["count"] += freed.sum().int()
    bt.copy_(torch.where(drop, -1, bt))
    st["seq"].copy_(torch.where(act, keep, seq))


def _plain_tables(st):
    more = _plain_fork(st) if st["case"]["parents"] else []
    got = _of_tables(st, *_plain_extend(st)) + more
    _plain_trim(st)
    return got + [st["bt"], st["seq"], st["refs"], st["free"], st["count"]]


_plain = dict(prefix=_plain_prefix, tables=_plain_tables)
_own = dict(prefix=_own_prefix, tables=_own_tables)


# -------------------------------------------------------------------- work

def work(case):
    ps = case["ps"]
    if case["op"] == "prefix":
        groups, lens = _groups(case)
        n, hkv, g = case["n"], case["hkv"], case["g"]
        tokens = sum(lens) - sum((m - 1) * (p // ps * ps) for _, m, p in groups)
        pairs = sum(max(0, x - n + 1 + i) for x in lens for i in range(n))
        per = 2 * D * (2 if case["kind"] == "bf16" else 1) + (2 / BLOCK if case["kind"] == "blocks" else 0)
        rows = case["batch"] * n * hkv * g
        return dict(bytes=tokens * hkv * per + tokens / ps * 4 + rows * D * (2 + (4 if case["fp32"] else 2)) +
                    case["batch"] * 12, flops=4.0 * D * g * hkv * pairs)
    plan = _table_plan(case)
    bytes_ = 0
    for length, new, parent, fork in plan:
        start = fork if parent >= 0 else length
        fresh = _up(start + new, ps) - (fork // ps if parent >= 0 else _up(length, ps))
        # forked entries (page, tag and count read and written), fresh pages (from and back to the list, entry,
        # expected and live tag, count), slots, and the request's numbers
        bytes_ += (fork // ps if parent >= 0 else 0) * 36 + fresh * 52 + new * 8 + 40
    return dict(bytes=float(bytes_), flops=0.0)


# ------------------------------------------------------------------- exact

def exact(case, seed):
    if case["op"] != "prefix":
        return None                                         # whole numbers
    st = prepare(case, seed)
    return _exact_attention(st)


def _e4m3_table():
    """The 256 codes' values in 64 bits, from the format's definition."""
    out = []
    for c in range(256):
        field, mant = (c >> 3) & 15, c & 7
        v = math.nan if field == 15 and mant == 7 else (
            mant * 2.0 ** -9 if field == 0 else (8 + mant) * 2.0 ** (field - 10))
        out.append(-v if c & 128 else v)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _exact_attention(st):
    """Request by request and head by head, over the positions up to the query's own."""
    c, table = st["case"], _e4m3_table()
    power = torch.tensor([2.0 ** i for i in range(-128, 129)], dtype=torch.float64, device=DEV)
    n, g, hkv, ps = c["n"], c["g"], c["hkv"], c["ps"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    _, lens = _groups(c)
    for b, length in enumerate(lens):
        if length == 0:
            continue
        j = torch.arange(length, device=DEV)
        page, at = st["bt"][b].long()[j // ps], j % ps
        first = max(0, n - length)                          # the first query with a position to see
        for h in range(hkv):
            kv = []
            for name in ("k", "v"):
                x = st[name][page, h, at]
                if c["kind"] == "bf16":
                    kv.append(x.double())
                elif c["kind"] == "blocks":
                    kv.append(table[x.long()] * power[st[name + "e"][page, h, at // BLOCK].long() + 128][:, None])
                else:
                    kv.append(table[x.long()] * st[name + "s"][h].double())
            q = st["q"][b, first:, h * g:(h + 1) * g].double()                             # [queries][g][D]
            s = torch.einsum("igd,jd->igj", q, kv[0]) / math.sqrt(D)
            last = length - n + torch.arange(first, n, device=DEV)
            s = s.masked_fill(j[None, None, :] > last[:, None, None], -math.inf)
            out[b, first:, h * g:(h + 1) * g] = torch.einsum("igj,jd->igd", torch.softmax(s, dim=2), kv[1])
    return out
