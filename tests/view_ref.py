"""Plain fp64 implementations of the block-scaled cache, the windowed reads and
their error bounds, shared by the tests of those operators (numpy; the e4m3
codec is the oracle's)."""
from __future__ import annotations

import numpy as np

import oracle
import workloads as W

D = 128
BLOCK = 16
E_MIN, E_MAX = -48, 48
NAN_CODE = 0x7F


def view_mask(length, n, window, sinks):
    """see[i][j]: does query token i of a request of ``length`` positions see position j."""
    p = length - n + np.arange(n)[:, None]
    j = np.arange(max(length, 0))[None, :]
    see = j <= p
    if window:
        see = see & ((j < sinks) | (j > p - window))
    return see


def positions(cache, bt_row, ps, h, pos):
    """Rows of a [N][Hkv][ps][D] cache that hold the positions ``pos`` of KV head h."""
    return cache[bt_row[pos // ps], h, pos % ps]


def attention(q_bits, k, v, bt, lens, scale, window, sinks, *, ks=None, vs=None, ke=None, ve=None,
              abort=None, fp32=False, cut=2.0 ** -40):
    """(out, bound) in fp64, [B][n][Hq][D].

    q_bits bf16 bits; k, v caches: uint8 codes (scales ks, vs per head, or
    exponents ke, ve per block) or uint16 bf16 bits.  ``bound`` is how far the
    kernels may be off, from their roundings:
      - a score is a sum of 128 exact products accumulated in fp32:
        ds = 128 * 2^-23 * sum |q k| * scale, and its use as an exponent rounds
        the scaled score and its distance to the maximum to fp32: 2^-22 of
        their size in log2 units; a score error moves its own weight by that
        much relative (the far smaller weights of far smaller scores too), and
        with it the weighted sum and the sum of the weights;
      - a weight becomes 16-bit terms, each rounding what those before it left
        (one f16 term for bf16 output, 2^-11, two for fp32, 2^-22; with a bf16
        cache one bf16 term, 2^-8, and three, 2^-24); f16
        terms, which hold 2^15 times the weight relative to the largest, are
        cut at multiples of 2^-24, so by at most 2^-40 of the largest
        (``cut``; the tensor-memory kernel holds 2^7 times: 2^-32);
      - sums in fp32 of up to L / 32 terms per warp and a merge of at most
        1024 partials: (L / 32 + 64) * 2^-23;
      - the output's own rounding, 2^-8 or 2^-24 of it.
    """
    B, n, Hq, _ = q_bits.shape
    _, Hkv, ps, _ = k.shape
    g = Hq // Hkv
    is_bf16 = k.dtype == np.uint16
    q = W.bf16_bits_to_f32(q_bits).astype(np.float64)
    out = np.zeros((B, n, Hq, D))
    bound = np.zeros_like(out)
    for b in range(B):
        L = int(lens[b])
        if L <= 0 or L > bt.shape[1] * ps or (abort is not None and abort[b]):
            continue
        see = view_mask(L, n, window, sinks)
        pos = np.flatnonzero(see.any(axis=0))
        if pos.size == 0:
            continue
        see = see[:, pos]
        pages = bt[b][pos // ps]
        if (pages < 0).any() or (pages >= k.shape[0]).any():
            continue
        for h in range(Hkv):
            rows = [positions(c, bt[b], ps, h, pos) for c in (k, v)]
            if is_bf16:
                kv = [W.bf16_bits_to_f32(x).astype(np.float64) for x in rows]
                unit = np.ones(pos.size)
            else:
                kv = [oracle.e4m3_decode(x) for x in rows]
                if ke is not None:
                    e = [x[pages, h, pos % ps // BLOCK].astype(np.float64) for x in (ke, ve)]
                    kv = [x * np.exp2(y)[:, None] for x, y in zip(kv, e)]
                    unit = np.exp2(e[1])
                else:
                    kv = [kv[0] * float(ks[h]), kv[1] * float(vs[h])]
                    unit = np.full(pos.size, float(vs[h]))
            qh = q[b, :, h * g:(h + 1) * g].reshape(n * g, D)
            s = (qh @ kv[0].T) * scale
            ds = 128 * 2.0 ** -23 * (np.abs(qh) @ np.abs(kv[0]).T) * abs(scale)
            seen = np.repeat(see, g, axis=0)
            s = np.where(seen, s, -np.inf)
            m = s.max(axis=1, keepdims=True)
            some = np.isfinite(m)
            p = np.exp(s - np.where(some, m, 0.0))
            total = p.sum(axis=1, keepdims=True)
            safe = np.where(total > 0, total, 1.0)
            o = p @ kv[1] / safe
            mean = p @ np.abs(kv[1]) / safe
            # the kernel's weights: w = p * unit relative to its largest
            w = p * unit[None, :]
            top = w.max(axis=1, keepdims=True)
            size = np.where(seen, np.abs(s) / np.log(2) + np.abs(np.log2(unit))[None, :] + 32, 0)
            wrong = p * np.expm1(ds + 2.0 ** -22 * size) / safe         # each weight's own share
            scores = wrong @ np.abs(kv[1]) + wrong.sum(axis=1, keepdims=True) * np.abs(o)
            rel = (2.0 ** -24 if fp32 else 2.0 ** -8) if is_bf16 else (2.0 ** -22 if fp32 else 2.0 ** -11)
            rel = rel + (L / 32 + 64) * 2.0 ** -23
            lost = 0.0
            if not is_bf16:
                lost = cut * top * (seen @ (np.abs(kv[1]) / unit[:, None])) / safe
            bnd = scores + rel * mean + lost
            bnd = bnd + (2.0 ** -24 if fp32 else 2.0 ** -8) * (np.abs(o) + bnd) + 1e-37
            out[b, :, h * g:(h + 1) * g] = np.where(some, o, 0).reshape(n, g, D)
            bound[b, :, h * g:(h + 1) * g] = np.where(some, bnd, 0).reshape(n, g, D)
    return out, bound


def assert_within(got, ref, bound, what=""):
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    err = np.where(nan, 0, np.abs(got - np.where(nan, 0, ref)))
    bad = err > np.where(nan, 0, bound)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; at {at}: {got[at]} for {ref[at]} "
                             f"+- {bound[at]}; worst {np.max(err / np.maximum(bound, 1e-300)):.2f} times")


def exponent(amax):
    """Least e of [-48, 48] with amax <= 448 * 2^e."""
    if not amax > 0:
        return E_MIN
    if np.isinf(amax):
        return E_MAX
    e = int(np.floor(np.log2(float(amax)))) - 10
    while float(amax) > 448.0 * 2.0 ** e:
        e += 1
    return max(E_MIN, min(E_MAX, e))


def append_blocks(k, v, ke, ve, k_new, v_new, offsets, bt, lens, abort=None):
    """In place: k, v uint8 codes, ke, ve int8 exponents; k_new, v_new bf16 bits [T][Hkv][D]."""
    _, Hkv, ps, _ = k.shape
    T = k_new.shape[0]
    for r in range(len(lens)):
        o0, o1, L = int(offsets[r]), int(offsets[r + 1]), int(lens[r])
        start = L - (o1 - o0)
        if (abort is not None and abort[r]) or o1 <= o0 or o0 < 0 or o1 > T or start < 0 or L > bt.shape[1] * ps:
            continue
        for block in range(start // BLOCK, (L - 1) // BLOCK + 1):
            lo, hi = max(start, block * BLOCK), min(L, (block + 1) * BLOCK)
            page = int(bt[r, block * BLOCK // ps])
            if page < 0 or page >= k.shape[0]:
                continue
            at, sub = lo % ps, block * BLOCK % ps // BLOCK
            first = block * BLOCK % ps
            for cache, exps, new in ((k, ke, k_new), (v, ve, v_new)):
                for h in range(Hkv):
                    x = W.bf16_bits_to_f32(new[o0 + lo - start:o0 + hi - start, h]).astype(np.float64)
                    mag = np.abs(x)
                    need = exponent(np.max(np.where(np.isnan(mag), 0, mag)))
                    e = need
                    if lo % BLOCK:
                        old = int(exps[page, h, sub])
                        e = max(old, need)
                        if e > old:
                            c = oracle.e4m3_decode(cache[page, h, first:at]) * 2.0 ** (old - e)
                            cache[page, h, first:at] = encode(c)
                    cache[page, h, at:at + hi - lo] = encode(x * 2.0 ** -e)
                    exps[page, h, sub] = e


def encode(x64):
    """e4m3 codes of fp64 values that an fp32 holds exactly (or too small for any code but 0)."""
    with np.errstate(over="ignore"):
        return oracle.e4m3_encode(np.asarray(x64).astype(np.float32))


def tag_check(bt, expected, lens, ps, tags, window, sinks, n):
    out = np.zeros(len(lens), np.uint8)
    for r, L in enumerate(int(x) for x in lens):
        used = -(-max(L, 0) // ps)
        if used > bt.shape[1]:
            out[r] = 1
            continue
        entries = np.arange(used)
        if window:
            first = -(-min(max(L, 0), sinks) // ps)
            entries = entries[(entries < first) | (entries >= max(0, L - n + 1 - window) // ps)]
        for i in entries:
            page = int(bt[r, i])
            if page < 0 or page >= len(tags) or tags[page] != expected[r, i]:
                out[r] = 1
    return out
