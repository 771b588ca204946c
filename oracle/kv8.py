"""Oracle of the 8-bit paged K/V cache in NumPy, request by request and in 64 bits: page
tables, quantising append, page selection and attention over the cached values."""
import math

import numpy as np

E4M3_MAX = 448.0


def e4m3_round(x):
    """The e4m3 value nearest to x (ties to even mantissa), saturating; NaN stays."""
    x = np.asarray(x, np.float64)
    mag = np.abs(x)
    with np.errstate(divide="ignore", invalid="ignore"):
        exp = np.where(mag >= 2.0 ** -6, np.floor(np.log2(np.where(mag > 0, mag, 1.0))), -6.0)
    step = np.exp2(np.where(np.isfinite(exp), exp, 8.0) - 3)
    with np.errstate(invalid="ignore"):
        r = np.round(x / step) * step
        return np.where(np.isnan(x), np.nan, np.clip(r, -E4M3_MAX, E4M3_MAX))


def scale_exponent(amax, top):
    """Least integer e >= -126 with amax <= top * 2^e."""
    if amax == 0:
        return -126
    e = math.floor(math.log2(amax / top)) - 1
    while amax > top * 2.0 ** e:
        e += 1
    return max(-126, e)


def page_tables(page_table, old, new, ring, state, page, max_tokens):
    """(page_table, ring, next_state, kv_lens, cu_q, slots, positions) after a step."""
    table, ring = page_table.copy(), ring.copy()
    width, n = table.shape[1], len(ring)
    head, count = int(state[0]), int(state[1])
    pages = lambda L: (L + page - 1) // page  # noqa: E731
    goal, bad = [], False
    for o, w in zip(old, new):
        if w < 0 or w > width * page:
            bad = True
            w = o
        goal.append(int(w))
    tokens = sum(max(0, w - o) for o, w in zip(old, goal))
    need = sum(max(0, pages(w) - pages(o)) for o, w in zip(old, goal))
    status = 2 if bad else 3 if tokens > max_tokens else 1 if need > count else 0
    lens, cu, slots, pos, taken, given = [], [0], [], [], 0, 0
    for b, (o, w) in enumerate(zip(old, goal)):
        if w > o and status:
            w = int(o)
        for p in range(pages(o), pages(w)):
            table[b, p] = ring[(head + taken) % n]
            taken += 1
        for p in range(pages(w), pages(o)):
            ring[(head + count + given) % n] = page_table[b, p]
            given += 1
        for t in range(o, w):
            slots.append(int(table[b, t // page]) * page + t % page)
            pos.append(t)
        lens.append(w)
        cu.append(len(slots))
    pad = [-1] * (max_tokens - len(slots))
    nxt = [(head + taken) % n, count - taken + given, status, need - count if status == 1 else 0]
    i32 = lambda v: np.asarray(v, np.int32)  # noqa: E731
    return table, ring, i32(nxt), i32(lens), i32(cu), i32(slots + pad), i32(pos + pad)


def append(codes, scale, bounds, x, slots, page):
    """codes (values of the codes, float64 [pages, hkv, page, d]), scale [pages, hkv] and bounds (int [pages,
    hkv, 2, d] or None) after writing x [T, hkv, d] to slots."""
    codes, scale = codes.copy(), scale.copy()
    bounds = None if bounds is None else bounds.astype(np.int64).copy()
    pages, hkv = scale.shape
    live = [t for t, s in enumerate(slots) if 0 <= s < pages * page]
    while live:
        pg = int(slots[live[0]]) // page
        e = 1
        while e < len(live) and slots[live[e]] // page == pg:
            e += 1
        run, live = live[:e], live[e:]
        at = [int(slots[t]) % page for t in run]
        off = at[0]
        for h in range(hkv):
            v = x[run, h].astype(np.float64)
            fin = np.abs(v[np.isfinite(v)])
            need = 2.0 ** scale_exponent(fin.max() if fin.size else 0.0, E4M3_MAX)
            was = scale[pg, h] if off else 0.0
            nan = np.isnan(v).any() or np.isnan(was)
            now, ratio = (need, 1.0) if nan else (max(need, was), was / max(need, was))
            codes[pg, h, :off] = e4m3_round(codes[pg, h, :off] * ratio)
            new = e4m3_round(np.where(np.isnan(v), 0.0, v) / now)
            codes[pg, h, at] = new
            if bounds is not None:
                q = new / 4
                hi, lo = np.ceil(q).max(0), np.floor(q).min(0)
                if off:
                    before = bounds[pg, h] * ratio
                    if math.frexp(was)[0] not in (0.0, 0.5) and ratio < 1:    # codes may have been rounded away from zero
                        before = e4m3_round(4.0 * before) / 4
                    hi = np.maximum(hi, np.ceil(before[0]))
                    lo = np.minimum(lo, np.floor(before[1]))
                bounds[pg, h] = np.stack([hi, lo])
            scale[pg, h] = np.nan if nan else now
    return codes, scale, bounds


def rows_of(kv_lens, cu_q, total):
    """(request, position, kv_len) of each token, None behind the last request."""
    out = [None] * total
    for b, n in enumerate(kv_lens):
        nq = int(cu_q[b + 1] - cu_q[b])
        for i in range(nq):
            out[int(cu_q[b]) + i] = (b, int(n) - nq + i, int(n))
    return out


def visible(pos, n, mask="causal", window=0):
    """[lo, hi) of the keys that a token at pos of a request of n tokens sees."""
    hi = n if mask == "full" else max(0, min(n, pos + 1))
    lo = max(0, pos - window + 1) if mask == "sliding" else 0
    return lo, max(lo, hi)


def select(q, bounds, k_scale, page_table, rows, page, k, sink, recent, mask="causal"):
    """Selected pages [T, hkv, k] (-1 past the last) and scores {(t, h): array}; rows as rows_of()."""
    T, hq, _ = q.shape
    hkv = bounds.shape[1]
    group = hq // hkv
    sel, scores = np.full((T, hkv, k), -1, np.int32), {}
    for t, row in enumerate(rows):
        if row is None:
            continue
        b, pos, n = row
        have = (visible(pos, n, mask)[1] + page - 1) // page
        for h in range(hkv):
            sc = np.full(have, -np.inf)
            for p in range(have):
                pg = page_table[b, p]
                if not 0 <= pg < len(bounds):
                    continue
                best = -np.inf
                for a in range(h * group, (h + 1) * group):
                    x = q[t, a].astype(np.float64)
                    fin = np.abs(x[np.isfinite(x)])
                    unit = 2.0 ** scale_exponent(fin.max() if fin.size else 0.0, 127.0)
                    qi = np.clip(np.round(np.where(np.isnan(x), 0.0, x) / unit), -127, 127)
                    best = max(best, unit * np.where(qi > 0, qi * bounds[pg, h, 0], qi * bounds[pg, h, 1]).sum())
                sc[p] = 3.4028234663852886e38 if np.isnan(k_scale[pg, h]) else 4 * k_scale[pg, h] * best
            scores[t, h] = sc.copy()
            sc[:sink] = np.inf
            sc[max(0, have - recent):] = np.inf
            pick = sorted(sorted(range(have), key=lambda p: (-sc[p], p))[:k])
            sel[t, h, :len(pick)] = pick
    return sel, scores


def attention(q, k, v, scale, lo, hi, keys=None):
    """One query row over the values k, v [n, d] of its request: (out, lse, sum_j p_j |v_j|, sum_j |v_j|,
    largest sum_c |q_c k_jc|) over keys [lo, hi), or over the listed ones."""
    at = np.arange(lo, hi) if keys is None else np.asarray(keys, np.int64)
    d = v.shape[1]
    if not len(at):
        return np.zeros(d), -np.inf, np.zeros(d), np.zeros(d), 0.0
    kk, vv, q = k[at], v[at], q.astype(np.float64)
    s = kk @ q * scale
    m = s.max()
    p = np.exp(s - m)
    l = p.sum()
    p = p / l
    return p @ vv, m + math.log(l), p @ np.abs(vv), np.abs(vv).sum(0), float((np.abs(kk) @ np.abs(q)).max())
