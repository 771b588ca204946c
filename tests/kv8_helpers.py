"""Shared by the tests of the 8-bit paged K/V cache: random caches and the comparison of
attention with the 64-bit oracle under a bound derived from the arithmetic."""
import numpy as np
import torch

import masked_flash_attention_attn_b200 as M
from oracle import decode_e4m3
from oracle import kv8 as O

E4M3 = torch.float8_e4m3fn


def values(t):
    """float64 values of an e4m3 tensor."""
    return decode_e4m3(t.view(torch.uint8).cpu().numpy())


def make_cache(seed, pages, hkv, page, d, exp_lo=-8, exp_hi=-5, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    code = lambda: (torch.randn(pages, hkv, page, d, generator=g) * 60).clamp(-448, 448).to(E4M3)  # noqa: E731
    sc = lambda: torch.exp2(torch.randint(exp_lo, exp_hi + 1, (pages, hkv), generator=g).float())  # noqa: E731
    k, v = code(), code()
    x = k.float()
    bounds = torch.stack([torch.ceil(x.amax(2) / 4), torch.floor(x.amin(2) / 4)], 2).to(torch.int8)
    return M.Kv8Cache.wrap(k.to(dev), v.to(dev), sc().to(dev), sc().to(dev), bounds.to(dev))


def make_table(seed, lens, page, pages, width=None):
    """Randomly placed pages; unused entries hold a page outside the cache."""
    rng = np.random.default_rng(seed)
    need = [(int(n) + page - 1) // page for n in lens]
    width = width or max(1, max(need, default=1))
    assert sum(need) <= pages
    perm = rng.permutation(pages)
    table = np.full((len(lens), width), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table


def i32(v, dev="cuda"):
    return torch.as_tensor(np.asarray(v, np.int32)).to(dev)


def cu_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


class Keys:
    """float64 values of the cached keys and values of a request and head (pages outside: zeros)."""

    def __init__(self, cache):
        self.c = cache
        self.k, self.v = values(cache.k), values(cache.v)
        self.ks, self.vs = cache.k_scale.double().cpu().numpy(), cache.v_scale.double().cpu().numpy()

    def of(self, table_row, n, h):
        page, d = self.c.page_size, self.c.head_dim
        out = []
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            parts = [x[p, h] * s[p, h] if 0 <= p < len(x) else np.zeros((page, d))
                     for p in table_row[:(n + page - 1) // page]]
            out.append(np.concatenate(parts)[:n] if parts else np.zeros((0, d)))
        return out


def check_rows(cache, q, table, rows, out, lse, *, scale, mask="causal", window=0, selected=None, sample=None, seed=0,
               p_err=2.0 ** -11, exp_err=2.0 ** -21, lse_abs=0.0):
    """out [T, hq, d], lse [T, hq] against the oracle. Bound, with S = sum_j p_j |v_j|: fp16 P (2^-11
    relative; 2^-25 / l absolute below 2^-14, l >= 2^-8 of the unit of P because the running maximum is
    within 2^8 of the true one), P's exponent off by the fp32 score sum (d additions and three
    products: (d + 4) 2^-24 sum |q k| scale) and by ex2 (2^-21), fp32 sums over n keys (2 n 2^-24 of S,
    but at least a few roundings of the joins), and the bf16 result (2^-8 relative). ``p_err``, ``exp_err``,
    ``lse_abs``: the roundings of P and of the exponential and the lse bound of another forward."""
    keys = Keys(cache)
    qn = q.float().cpu().numpy().astype(np.float64)
    out = out.float().cpu().numpy().astype(np.float64)
    lse = lse.cpu().numpy().astype(np.float64)
    T, hq, d = qn.shape
    group = hq // cache.hkv
    todo = [(t, h) for t in range(T) if rows[t] is not None for h in range(hq)]
    if sample and len(todo) > sample:
        rng = np.random.default_rng(seed)
        todo = [todo[i] for i in sorted(rng.choice(len(todo), sample, replace=False))]
    memo = {}
    worst = 0.0
    for t, a in todo:
        b, pos, n = rows[t]
        h = a // group
        if (b, h) not in memo:
            memo = {(b, h): keys.of(table[b], n, h)}
        k, v = memo[b, h]
        lo, hi = O.visible(pos, n, mask, window)
        at = None
        if selected is not None:
            page = cache.page_size
            at = [j for p in selected[t, h] if p >= 0 for j in range(p * page, (p + 1) * page) if lo <= j < hi]
        ref, rl, S, A, qk = O.attention(qn[t, a], k, v, scale, lo, hi, at)
        nk = max(1, hi - lo if at is None else len(at))
        if not np.isfinite(rl) and rl < 0:
            assert lse[t, a] == -np.inf and (out[t, a] == 0).all(), (t, a)
            continue
        dp = (d + 4) * 2.0 ** -24 * qk * scale + exp_err
        tol = (p_err + 2 * dp + (nk + 64) * 2.0 ** -23) * S + 2.0 ** -17 * A / nk + 2.0 ** -8 * np.abs(ref) + 1e-30
        err = np.abs(out[t, a] - ref)
        assert (np.isnan(ref) == np.isnan(out[t, a])).all(), (t, a)
        ok = (err <= tol) | np.isnan(ref)
        assert ok.all(), (t, a, float(np.nanmax(err / tol)))
        worst = max(worst, float(np.nanmax(np.where(np.isnan(ref), 0, err / tol))))
        if np.isfinite(rl):
            assert abs(lse[t, a] - rl) <= lse_abs + dp + (nk + 64) * 2.0 ** -23 + abs(rl) * 2.0 ** -22, (t, a, lse[t, a], rl)
    return worst
