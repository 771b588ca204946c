"""Cases, plain forms and exact values of the 8-bit paged K/V cache operators.

Five paths: "tables" (page tables and slot maps from request lengths), "append" (quantise new
keys / values into the cache), "attend" (attention of a few tokens per request over the
cache), "prefill" (a long chunk of queries over the cache: the pages gathered as bf16, then
the masked forward) and "sparse" (pages selected by a cheap score, then attention over them).

The cache holds K and V as e4m3 codes [num_pages][hkv][page][d] with one fp32 scale per page
and head, and int8 channel-wise bounds of each page's K codes [num_pages][hkv][2][d] (max,
min, in steps of 4 codes). ``own`` selects between the library's calls and the plain forms.
"""
import math
import random

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
PAGES = (16, 32, 64, 128)


# ---- cases ---------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a small server: 16 requests, one token each
        dict(name="tables_decode", op="tables", batch=16, page=16, len_min=100, len_max=4000, prefill=0, finished=0, mix=1),
        # a large mixed step: most requests decode, some are admitted with long prompts, some end
        dict(name="tables_mixed", op="tables", batch=771, page=64, len_min=64, len_max=8192, prefill=9, finished=25, mix=2),
        # the new keys / values of a decode step: a few tokens into pages that hold others
        dict(name="append_decode", op="append", batch=32, hkv=8, d=128, page=16, q_min=1, q_max=1, len_min=512, len_max=4096, mix=3),
        # a prompt chunk of several requests, odd lengths, large pages
        dict(name="append_prefill", op="append", batch=5, hkv=8, d=128, page=64, q_min=1500, q_max=4001, len_min=0, len_max=3000, mix=4),
        # the smallest call: one request, one token
        dict(name="decode_one", op="attend", batch=1, hq=16, hkv=8, d=128, page=16, q_min=1, q_max=1, len_min=1000, len_max=1000, mask="causal", window=0, mix=5),
        # a decode step of a batch, grouped queries
        dict(name="decode_batch", op="attend", batch=32, hq=32, hkv=8, d=128, page=16, q_min=1, q_max=1, len_min=512, len_max=4096, mask="causal", window=0, mix=6),
        # long contexts, ragged
        dict(name="decode_long", op="attend", batch=8, hq=32, hkv=8, d=128, page=64, q_min=1, q_max=1, len_min=40000, len_max=65536, mask="causal", window=0, mix=7),
        # a few draft tokens per request under a sliding window, head_dim 256
        dict(name="verify_sliding_d256", op="attend", batch=16, hq=16, hkv=8, d=256, page=32, q_min=2, q_max=8, len_min=1024, len_max=8192, mask="sliding", window=4096, mix=8),
        # a prompt chunk that follows a cached prefix
        dict(name="prefill_chunk", op="prefill", batch=4, hq=32, hkv=8, d=128, page=64, q_min=700, q_max=1024, len_min=2048, len_max=8192, mix=9),
        # a short prompt chunk, head_dim 64, every head its own keys
        dict(name="prefill_small_d64", op="prefill", batch=3, hq=8, hkv=8, d=64, page=16, q_min=17, q_max=130, len_min=130, len_max=900, mix=10),
        # sparse decode: a small batch at moderate length
        dict(name="sparse_small", op="sparse", batch=4, hq=32, hkv=8, d=128, page=16, q_min=1, q_max=1, len_min=2000, len_max=8000, budget=64, sink=1, recent=2, mix=11),
        # sparse decode: a batch of long contexts
        dict(name="sparse_long", op="sparse", batch=32, hq=32, hkv=8, d=128, page=32, q_min=1, q_max=1, len_min=16000, len_max=32768, budget=64, sink=1, recent=4, mix=12),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tables", "append", "attend", "attend", "prefill", "sparse"))
    page, mix = rng.choice(PAGES), rng.randrange(1 << 30)
    if op == "tables":
        batch = _log(rng, 1, 2000)
        hi = _log(rng, 16, 8192)
        return dict(op=op, batch=batch, page=page, len_min=rng.randint(0, hi), len_max=hi, prefill=min(batch, rng.choice((0, 1, 3, 8))),
                    finished=rng.choice((0, 0, 1, batch // 10)), mix=mix)
    d = rng.choice((64, 128, 128, 256))
    hkv = rng.choice((1, 2, 3, 4, 8, 16))
    if op == "append":
        batch = _log(rng, 1, 64)
        q = _log(rng, 1, max(1, min(4000, 6_000_000 // (batch * hkv * d))))
        return dict(op=op, batch=batch, hkv=hkv, d=d, page=page, q_min=rng.randint(1, q), q_max=q, len_min=0, len_max=_log(rng, 1, 2000), mix=mix)
    hq = hkv * rng.choice((1, 2, 3, 4, 5, 8)) if op != "prefill" else hkv * rng.choice((1, 2, 4))
    if op == "prefill":
        batch = _log(rng, 1, 4)
        q = _log(rng, 4, max(4, min(1024, 100_000 // (batch * hq))))
        hi = _log(rng, q, 8192)
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, page=page, q_min=rng.randint(1, q), q_max=q, len_min=rng.randint(q, hi), len_max=hi, mix=mix)
    batch = _log(rng, 1, 64)
    hi = _log(rng, 1 if op == "attend" else 200, max(200, min(65536, 500_000_000 // (batch * hkv * d * 2))))
    lo = max(1, int(hi * rng.choice((0.1, 0.5, 1.0))))
    if op == "attend":
        q = min(lo, rng.choice((1, 1, 1, 2, 3, 7)))
        mask = rng.choice(("causal", "causal", "full", "sliding"))
        return dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, page=page, q_min=1, q_max=q, len_min=lo, len_max=hi, mask=mask,
                    window=_log(rng, 1, hi) if mask == "sliding" else 0, mix=mix)
    return dict(op=op, batch=batch, hq=hq, hkv=hkv, d=d, page=page, q_min=1, q_max=min(lo, rng.choice((1, 1, 2))), len_min=lo, len_max=hi,
                budget=rng.choice((5, 16, 33, 64)), sink=rng.choice((0, 1, 2)), recent=rng.choice((1, 2)), mix=mix)


def _lengths(c):
    """(kv_lens, q_lens) of the requests, from the case alone; kv_lens count the new tokens."""
    rng = random.Random(c["mix"])
    kv = [rng.randint(c["len_min"], c["len_max"]) for _ in range(c["batch"])]
    q = [rng.randint(c["q_min"], c["q_max"]) for _ in range(c["batch"])]
    if c["op"] == "append":                      # len_min .. len_max are the lengths before
        kv = [a + b for a, b in zip(kv, q)]
    return kv, q


def _table_lengths(c):
    """(lengths before, lengths after) of a scheduling step."""
    rng = random.Random(c["mix"])
    old = [rng.randint(c["len_min"], c["len_max"]) for _ in range(c["batch"])]
    new = [n + 1 for n in old]
    order = list(range(c["batch"]))
    rng.shuffle(order)
    for b in order[:c["finished"]]:
        new[b] = 0
    for b in order[c["finished"]:c["finished"] + c["prefill"]]:
        old[b], new[b] = 0, rng.randint(max(1, c["len_min"]), c["len_max"])
    return old, new


def _pages(n, page):
    return (n + page - 1) // page


# ---- inputs --------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lens):
    return _i32(np.concatenate([[0], np.cumsum(lens)]).tolist())


def _page_table(g, lens, page, spare):
    """A page table whose requests hold randomly placed pages, and the number of pages."""
    need = [_pages(n, page) for n in lens]
    width, total = max(1, max(need)), sum(need) + spare
    perm = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    start = torch.tensor(np.concatenate([[0], np.cumsum(need)[:-1]]).tolist(), device="cuda")
    col = torch.arange(width, device="cuda")
    idx = (start[:, None] + col).clamp(max=total - 1)
    table = torch.where(col < torch.tensor(need, device="cuda")[:, None], perm[idx], torch.full_like(perm[idx], -1))
    return table.contiguous(), total, perm[sum(need):].contiguous()


def _fill(g, pages, hkv, page, d, structured):
    """A filled cache: codes with a few large channels, scales that vary from page to page."""
    gain = 20.0 + 60.0 * torch.rand(hkv, 1, d, device="cuda", generator=g)
    out = []
    for _ in range(2):
        codes = torch.empty(pages, hkv, page, d, dtype=E4M3, device="cuda")
        step = max(1, (1 << 26) // (hkv * page * d))
        for s in range(0, pages, step):
            n = min(step, pages - s)
            x = torch.randn(n, hkv, page, d, device="cuda", generator=g)
            if structured and not out:           # the keys of a page are alike
                x += 1.5 * torch.randn(n, hkv, 1, d, device="cuda", generator=g)
            codes[s:s + n] = (x * gain).clamp(-448, 448).to(E4M3)
        out.append(codes)
        out.append(torch.exp2(torch.randint(-8, -5, (pages, hkv), device="cuda", generator=g).float()))
    k, ks, v, vs = out
    bounds = torch.empty(pages, hkv, 2, d, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 26) // (hkv * page * d))
    for s in range(0, pages, step):
        x = k[s:s + step].float()
        bounds[s:s + step, :, 0] = torch.ceil(x.amax(2) / 4).to(torch.int8)
        bounds[s:s + step, :, 1] = torch.floor(x.amin(2) / 4).to(torch.int8)
    return k, v, ks, vs, bounds


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"case": c}
    if c["op"] == "tables":
        old, new = _table_lengths(c)
        width = _pages(max(max(old), max(new)), c["page"]) + 1
        grow = sum(max(0, _pages(b, c["page"]) - _pages(a, c["page"])) for a, b in zip(old, new))
        table, total, spare = _page_table(g, old, c["page"], grow + 64)
        s["page_table"] = torch.full((c["batch"], width), -1, dtype=torch.int32, device="cuda")
        s["page_table"][:, :min(width, table.shape[1])] = table[:, :width]
        ring = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        head = int(torch.randint(0, total, (1,), device="cuda", generator=g))
        ring[(head + torch.arange(len(spare), device="cuda")) % total] = spare
        tokens = sum(max(0, b - a) for a, b in zip(old, new))
        s.update(old_lens=_i32(old), new_lens=_i32(new), free_pages=ring, free_state=_i32([head, len(spare), 0, 0]),
                 next_state=torch.zeros(4, dtype=torch.int32, device="cuda"), kv_lens=torch.zeros(c["batch"], dtype=torch.int32, device="cuda"),
                 cu_q=torch.zeros(c["batch"] + 1, dtype=torch.int32, device="cuda"),
                 slots=torch.zeros(tokens + 5, dtype=torch.int32, device="cuda"), positions=torch.zeros(tokens + 5, dtype=torch.int32, device="cuda"))
        return s
    kv, q = _lengths(c)
    table, pages, _ = _page_table(g, kv, c["page"], 8)
    k8, v8, ks, vs, bounds = _fill(g, pages, c["hkv"], c["page"], c["d"], c["op"] == "sparse")
    s.update(page_table=table, kv_lens=_i32(kv), cu_q=_cu(q), k8=k8, v8=v8, k_scale=ks, v_scale=vs, k_bounds=bounds)
    total = sum(q)
    if c["op"] == "append":
        seq = torch.repeat_interleave(torch.arange(c["batch"], device="cuda"), torch.tensor(q, device="cuda"))
        pos = torch.arange(total, device="cuda") - s["cu_q"].long()[seq] + (torch.tensor(kv, device="cuda") - torch.tensor(q, device="cuda"))[seq]
        s["slots"] = (table.long()[seq, pos // c["page"]] * c["page"] + pos % c["page"]).to(torch.int32)
        gain = torch.exp(0.5 * torch.randn(total, 1, 1, device="cuda", generator=g)) * (0.3 + torch.rand(1, c["hkv"], c["d"], device="cuda", generator=g))
        s["k"] = (torch.randn(total, c["hkv"], c["d"], device="cuda", generator=g) * gain).to(torch.bfloat16)
        s["v"] = torch.randn(total, c["hkv"], c["d"], device="cuda", generator=g).to(torch.bfloat16)
    else:
        s["q"] = torch.randn(total, c["hq"], c["d"], device="cuda", generator=g).to(torch.bfloat16)
        s["out"] = torch.zeros(total, c["hq"], c["d"], dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(total, c["hq"], dtype=torch.float32, device="cuda")
    if c["op"] == "prefill":
        s["cu_k"] = _cu(kv)
        s["k"] = torch.zeros(sum(kv), c["hkv"], c["d"], dtype=torch.bfloat16, device="cuda")
        s["v"] = torch.zeros_like(s["k"])
    if c["op"] == "sparse":
        s["selected"] = torch.full((total, c["hkv"], c["budget"]), -1, dtype=torch.int32, device="cuda")
        s["scores"] = torch.zeros(total, c["hkv"], table.shape[1], dtype=torch.float32, device="cuda")
    if own:
        import masked_flash_attention_attn_b200 as attn
        from masked_flash_attention_attn_b200 import mask as masks
        s["cache"] = attn.Kv8Cache.wrap(k8, v8, ks, vs, bounds)
        if c["op"] in ("attend", "sparse"):
            m = {"causal": masks.causal, "full": masks.full}.get(c.get("mask", "causal"), lambda: masks.sliding_window(c["window"]))()
            s["plan"] = attn.attn_kv8_plan(hq=c["hq"], hkv=c["hkv"], head_dim=c["d"], page_size=c["page"], mask=m, max_q_len=c["q_max"])
        if c["op"] == "prefill":
            s["plan"] = attn.attn_plan(hq=c["hq"], hkv=c["hkv"], head_dim=c["d"], cu_seqlens_q=np.cumsum([0] + q), cu_seqlens_k=np.cumsum([0] + kv), mask=masks.causal())
    return s


# ---- one pass ------------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state["case"]["op"], state)


def _run_own(op, s):
    import masked_flash_attention_attn_b200 as attn
    if op == "tables":
        attn.attn_page_tables(page_table=s["page_table"], old_lens=s["old_lens"], new_lens=s["new_lens"], free_pages=s["free_pages"],
                              free_state=s["free_state"], page_size=s["case"]["page"], next_state=s["next_state"], kv_lens=s["kv_lens"],
                              cu_seqlens_q=s["cu_q"], slots=s["slots"], positions=s["positions"])
    elif op == "append":
        attn.attn_kv8_append(s["cache"], s["k"], s["v"], s["slots"])
    elif op == "attend":
        attn.attn_kv8_fwd(s["plan"], s["cache"], s["q"], s["page_table"], s["kv_lens"], s["out"], s["lse"], cu_seqlens_q=s["cu_q"])
    elif op == "prefill":
        attn.attn_kv8_gather(s["cache"], s["page_table"], s["cu_k"], s["k"], s["v"])
        attn.attn_masked_fwd(s["plan"], s["q"], s["k"], s["v"], s["out"], s["lse"])
    else:
        attn.attn_kv8_select(s["plan"], s["cache"], s["q"], s["page_table"], s["kv_lens"], s["scores"], s["selected"], cu_seqlens_q=s["cu_q"],
                             sink=s["case"]["sink"], recent=s["case"]["recent"])
        attn.attn_kv8_fwd(s["plan"], s["cache"], s["q"], s["page_table"], s["kv_lens"], s["out"], s["lse"], cu_seqlens_q=s["cu_q"],
                          selected=s["selected"])
    return _outputs(op, s)


def _outputs(op, s):
    if op == "tables":
        return [s[n] for n in ("page_table", "free_pages", "next_state", "kv_lens", "cu_q", "slots", "positions")]
    if op == "append":
        return [s[n] for n in ("k8", "v8", "k_scale", "v_scale", "k_bounds")]
    if op == "sparse":
        return [s["selected"], s["out"], s["lse"]]
    return [s["out"], s["lse"]]


def _run_plain(op, s):
    {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend, "prefill": _plain_attend, "sparse": _plain_sparse}[op](s)
    return _outputs(op, s)


def _plain_tables(s):
    page, table, ring = s["case"]["page"], s["page_table"], s["free_pages"]
    cap, n, width, T = table.shape[1] * page, ring.numel(), table.shape[1], s["slots"].numel()
    old, new = s["old_lens"].long().clamp(0, cap), s["new_lens"].long()
    head, count = s["free_state"].long()[0], s["free_state"].long()[1]
    valid = (new >= 0) & (new <= cap)
    new = torch.where(valid, new, old)
    before, after = (old + page - 1) // page, (new + page - 1) // page
    grow, take, give = (new - old).clamp(min=0), (after - before).clamp(min=0), (before - after).clamp(min=0)
    status = torch.where(take.sum() > count, 1, 0)
    status = torch.where(grow.sum() > T, 3, status)
    status = torch.where(valid.all(), status, 2)
    ok = (status == 0).long()
    short = torch.where(status == 1, take.sum() - count, 0)
    grow, take = grow * ok, take * ok
    p = torch.arange(width, device=table.device)
    got = (head + (take.cumsum(0) - take)[:, None] + p - before[:, None]) % n
    put = (head + count + (give.cumsum(0) - give)[:, None] + p - after[:, None]) % n
    taking = (p >= before[:, None]) & (p < (before + take)[:, None])
    giving = (p >= after[:, None]) & (p < (after + give)[:, None])
    ring[put[giving]] = table[giving]
    table.copy_(torch.where(taking, ring[got], table))
    s["kv_lens"].copy_(torch.where((ok > 0) | (new < old), new, old))
    s["cu_q"][1:] = grow.cumsum(0)
    s["next_state"].copy_(torch.stack([(head + take.sum()) % n, count - take.sum() + give.sum(), status, short]))
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(s["cu_q"][1:].long().contiguous(), t, right=True).clamp(max=len(old) - 1)
    pos = old[b] + t - s["cu_q"].long()[b]
    live = t < s["cu_q"][-1]
    slot = table[b, (pos // page).clamp(0, width - 1)].long() * page + pos % page
    s["slots"].copy_(torch.where(live, slot, -1))
    s["positions"].copy_(torch.where(live, pos, -1))


def _at(codes, index):
    """codes[index] of an e4m3 tensor."""
    return codes.view(torch.uint8)[index].view(E4M3)


def _plain_append(s):
    hkv, page = s["case"]["hkv"], s["case"]["page"]
    slot = s["slots"].long()
    pg, off = slot // page, slot % page
    first = torch.ones_like(pg, dtype=torch.bool)
    first[1:] = pg[1:] != pg[:-1]
    run = first.long().cumsum(0) - 1                             # the page run of each token
    rp, ro = pg[first], off[first]                                # its page, and its first offset there
    for x, codes, scale in ((s["k"], s["k8"], s["k_scale"]), (s["v"], s["v8"], s["v_scale"])):
        x = x.float()
        amax = torch.zeros(len(rp), hkv, device=x.device).index_reduce_(0, run, x.abs().amax(2), "amax")
        m, e = torch.frexp(amax)                                  # amax = m 2^e, 448 = 0.875 * 2^9
        e = torch.where(amax > 0, e - 9 + (m > 0.875).int(), -126).clamp(min=-126)
        old = torch.where(ro[:, None] > 0, scale[rp], 0.0)
        now = torch.maximum(old, torch.ldexp(torch.ones_like(amax), e))
        scale[rp] = now
        ratio = old / now
        was = _at(codes, rp)
        keep = torch.arange(page, device=x.device)[None, None, :, None] < ro[:, None, None, None]
        was = torch.where(keep, (was.float() * ratio[:, :, None, None]).to(E4M3).view(torch.uint8), was.view(torch.uint8))
        codes.view(torch.uint8)[rp] = was
        new = (x / now[run][:, :, None]).clamp(-448, 448).to(E4M3)
        codes.view(torch.uint8)[pg, :, off] = new.view(torch.uint8)
        if codes is s["k8"]:
            q = new.float() / 4
            hi = torch.full((len(rp), hkv, q.shape[2]), -128.0, device=x.device).index_reduce_(0, run, torch.ceil(q), "amax")
            lo = torch.full_like(hi, 127.0).index_reduce_(0, run, torch.floor(q), "amin")
            had = (ro > 0)[:, None, None]
            b = s["k_bounds"][rp].float()
            hi = torch.where(had, torch.maximum(hi, torch.ceil(b[:, :, 0] * ratio[:, :, None])), hi)
            lo = torch.where(had, torch.minimum(lo, torch.floor(b[:, :, 1] * ratio[:, :, None])), lo)
            s["k_bounds"][rp] = torch.stack([hi, lo], 2).to(torch.int8)


def _padded(s):
    """Queries as [batch, hkv, tokens * group, d] in 32 bits, and each token's request and place."""
    c, cu = s["case"], s["cu_q"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    i = t - cu[b]
    q = torch.zeros(c["batch"], c["q_max"], c["hq"], c["d"], device="cuda")
    q[b, i] = s["q"].float()
    group = c["hq"] // c["hkv"]
    return q.view(c["batch"], c["q_max"], c["hkv"], group, c["d"]).permute(0, 2, 1, 3, 4).flatten(2, 3), b, i


def _values(codes, scale, table):
    """Cache pages as [batch, hkv, keys, d] in 32 bits."""
    idx = table.long().clamp(min=0)
    x = _at(codes, idx).float() * scale[idx][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _softmax(c, q, k, v, seen):
    """out [batch, hkv, rows, d] and lse [batch, hkv, rows]; seen [batch, 1 or hkv, rows, keys]."""
    x = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(c["d"]))
    x = torch.where(seen, x, float("-inf"))
    top = x.amax(3, keepdim=True)
    p = torch.exp(x - torch.where(top > float("-inf"), top, 0.0))
    total = p.sum(3, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, 1.0)
    return out, (top + torch.log(total)).squeeze(3)


def _rows(s, j, mask):
    """[batch, 1, rows, keys] visibility of key positions j [.., keys] to the padded rows."""
    c = s["case"]
    lens, qn = s["kv_lens"].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    pos = (lens - qn)[:, None] + torch.arange(c["q_max"], device="cuda")
    pos = pos.repeat_interleave(c["hq"] // c["hkv"], 1)[:, None, :, None]
    seen = j < lens[:, None, None, None]
    if mask != "full":
        seen = seen & (j <= pos)
    if mask == "sliding":
        seen = seen & (pos - j < c["window"])
    return seen


def _write(s, out, lse, b, i):
    c = s["case"]
    group = c["hq"] // c["hkv"]
    out = out.view(c["batch"], c["hkv"], c["q_max"], group, c["d"]).permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = lse.view(c["batch"], c["hkv"], c["q_max"], group).permute(0, 2, 1, 3).flatten(2, 3)
    s["out"].copy_(out[b, i])
    s["lse"].copy_(lse[b, i])


def _plain_attend(s):
    q, b, i = _padded(s)
    k, v = _values(s["k8"], s["k_scale"], s["page_table"]), _values(s["v8"], s["v_scale"], s["page_table"])
    j = torch.arange(k.shape[2], device="cuda")
    out, lse = _softmax(s["case"], q, k, v, _rows(s, j, s["case"].get("mask", "causal")))
    _write(s, out, lse, b, i)


def _plain_sparse(s):
    c, table = s["case"], s["page_table"]
    page, group, width, k = c["page"], c["hq"] // c["hkv"], table.shape[1], c["budget"]
    qp, b, i = _padded(s)
    pos = (s["kv_lens"].long() - (s["cu_q"][1:] - s["cu_q"][:-1]).long())[b] + i
    n = pos // page + 1                                           # pages that a token sees
    # queries in 8 bits, one power of two per token and head; scores are exact integers
    q = s["q"].float().view(-1, c["hkv"], group, c["d"])
    amax = q.abs().amax(3)
    m, e = torch.frexp(amax)                                      # 127 = 0.9921875 * 2^7
    e = torch.where(amax > 0, e - 7 + (m > 0.9921875).int(), -126).clamp(min=-126)
    unit = torch.ldexp(torch.ones_like(amax), e)
    qi = torch.round(q / unit[..., None])
    # one table row per token; integers below 2^24 are exact in 32 bits, in any order of the sum
    idx = table.long().clamp(min=0)[b]                            # [T, width]
    bounds = s["k_bounds"][idx].permute(0, 2, 3, 4, 1).float()    # [T, hkv, 2, d, width]
    dots = qi.clamp(min=0) @ bounds[:, :, 0] + qi.clamp(max=0) @ bounds[:, :, 1]
    score = (dots * unit[..., None]).amax(2) * (4.0 * s["k_scale"][idx].transpose(1, 2))
    p = torch.arange(width, device="cuda")
    inside = (p < n[:, None])[:, None]
    s["scores"].copy_(torch.where(inside, score, s["scores"]))
    forced = ((p < c["sink"]) | (p >= (n - c["recent"])[:, None]))[:, None]
    score = torch.where(inside, torch.where(forced, float("inf"), score), float("-inf"))
    order = torch.sort(score, dim=2, descending=True, stable=True).indices[:, :, :k]
    held = torch.arange(order.shape[2], device="cuda") < n.clamp(max=k)[:, None, None]
    order = torch.sort(torch.where(held, order, width), dim=2).values
    s["selected"].fill_(-1)
    s["selected"][:, :, :order.shape[2]] = torch.where(order < width, order, -1).to(torch.int32)
    # attention of each token over its own list, per KV head
    sel = s["selected"].long()
    phys = table.long()[b[:, None, None], sel.clamp(min=0)].clamp(min=0)
    h = torch.arange(c["hkv"], device="cuda")[None, :, None]
    kk = (_at(s["k8"], (phys, h)).float() * s["k_scale"][phys, h][..., None, None]).flatten(2, 3)
    vv = (_at(s["v8"], (phys, h)).float() * s["v_scale"][phys, h][..., None, None]).flatten(2, 3)
    j = (sel[..., None] * page + torch.arange(page, device="cuda")).flatten(2, 3)
    seen = ((sel >= 0)[..., None].expand(-1, -1, -1, page).flatten(2, 3) & (j <= pos[:, None, None]))[:, :, None]
    out, lse = _softmax(c, q, kk, vv, seen)
    s["out"].copy_(out.flatten(1, 2))
    s["lse"].copy_(lse.flatten(1, 2))


# ---- what a pass cannot do without ----------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "tables":
        old, new = _table_lengths(c)
        moved = sum(abs(_pages(b, c["page"]) - _pages(a, c["page"])) for a, b in zip(old, new))
        tokens = sum(max(0, b - a) for a, b in zip(old, new))
        return {"bytes": 16 * len(old) + 8 * tokens + 8 * moved, "flops": 0}
    kv, q = _lengths(c)
    per = c["hkv"] * c["d"]
    if c["op"] == "append":
        runs = sum(_pages(n, c["page"]) - (n - m) // c["page"] for n, m in zip(kv, q))
        return {"bytes": sum(q) * (per * 2 * 3 + 4) + runs * c["hkv"] * (2 * c["d"] + 8), "flops": 0}
    io = sum(q) * c["hq"] * (4 * c["d"] + 4)
    pairs, keys, pages = 0, 0, 0
    for n, m in zip(kv, q):
        if c["op"] == "sparse":
            for i in range(m):
                have = (n - m + i) // c["page"] + 1
                used = min(have, c["budget"])
                seen = (used - 1) * c["page"] + (n - m + i) % c["page"] + 1
                pairs, keys = pairs + seen, keys + seen
            pages += have
            continue
        w = c["window"] if c.get("mask") == "sliding" else n + m
        if c.get("mask") == "full":
            pairs += n * m
        else:
            pairs += sum(min(w, n - m + i + 1) for i in range(m))
        keys += n - max(0, n - m + 1 - w)
    scan = pages * (2 * per + 4 * c["hkv"]) if c["op"] == "sparse" else 0
    return {"bytes": keys * 2 * per + keys // c["page"] * (8 * c["hkv"] + 4) + io + scan, "flops": 4 * c["d"] * c["hq"] * pairs}


# ---- 64-bit values from the definitions, request by request ---------------------------------
def exact(case, seed):
    if case["op"] == "tables":
        return None                       # whole numbers only
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


def _e4m3_nearest(x):
    """The e4m3 value nearest to each x (ties to even), |x| <= 464, in 64 bits."""
    x = np.asarray(x, dtype=np.float64)
    exp = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    step = np.exp2(exp - 3)
    return np.clip(np.round(x / step) * step, -448, 448)


def _exact_append(s):
    c = s["case"]
    page = c["page"]
    slots = s["slots"].cpu().numpy().astype(np.int64)
    out = []
    for name, codes, scale in (("k", "k8", "k_scale"), ("v", "v8", "v_scale")):
        x = s[name].double().cpu().numpy()
        code, sc = s[codes].cpu().float().numpy().astype(np.float64), s[scale].double().cpu().numpy()
        t = 0
        while t < len(slots):
            pg, o, e = slots[t] // page, slots[t] % page, t
            while e < len(slots) and slots[e] // page == pg:
                e += 1
            block = x[t:e].transpose(1, 0, 2)                     # [hkv, tokens, d]
            peak = np.abs(block).max((1, 2))
            need = np.exp2(np.array([max(-126, math.ceil(math.log2(a / 448))) if a > 0 else -126 for a in peak], dtype=np.float64))
            was = sc[pg] if o > 0 else np.zeros(c["hkv"])
            now = np.maximum(need, was)
            code[pg, :, :o] = _e4m3_nearest(code[pg, :, :o] * (was / now)[:, None, None])
            code[pg, :, o:o + e - t] = _e4m3_nearest(block / now[:, None, None])
            sc[pg] = now
            t = e
        out.append((code, sc))
    (k, ks), (v, vs) = out
    return [torch.from_numpy(k), torch.from_numpy(v), torch.from_numpy(ks), torch.from_numpy(vs), None]


def _exact_attention(s):
    c = s["case"]
    page, group = c["page"], c["hq"] // c["hkv"]
    kv, qn = _lengths(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
    picked = _exact_selection(s) if c["op"] == "sparse" else None
    t0 = 0
    for r, (n, m) in enumerate(zip(kv, qn)):
        pages = s["page_table"][r, :_pages(n, page)].long()
        first = n - m
        for h in range(c["hkv"]):
            keys = (_at(s["k8"], (pages, h)).double() * s["k_scale"][pages, h].double()[:, None, None]).reshape(-1, c["d"])[:n]
            vals = (_at(s["v8"], (pages, h)).double() * s["v_scale"][pages, h].double()[:, None, None]).reshape(-1, c["d"])[:n]
            at = torch.arange(n, device="cuda")
            own_pos = first + torch.arange(m, device="cuda")
            vis = torch.ones(m, n, dtype=torch.bool, device="cuda")
            if c.get("mask") != "full":
                vis &= at[None] <= own_pos[:, None]
            if c.get("mask") == "sliding":
                vis &= at[None] > own_pos[:, None] - c["window"]
            if picked is not None:
                for i in range(m):
                    vis[i] &= torch.isin(at // page, picked[t0 + i][h])
            for e in range(h * group, (h + 1) * group):
                logits = s["q"][t0:t0 + m, e].double() @ keys.T / math.sqrt(c["d"])
                logits = logits.masked_fill(~vis, float("-inf"))
                lse[t0:t0 + m, e] = torch.logsumexp(logits, 1)
                weight = torch.exp(logits - lse[t0:t0 + m, e, None]).nan_to_num(0.0)
                out[t0:t0 + m, e] = weight @ vals
        t0 += m
    return [None, out, lse] if picked is not None else [out, lse]


def _exact_selection(s):
    """The pages of every token and KV head, by the score in 64 bits."""
    c = s["case"]
    page, group = c["page"], c["hq"] // c["hkv"]
    kv, qn = _lengths(c)
    picked, t = [], 0
    for r, (n, m) in enumerate(zip(kv, qn)):
        for i in range(m):
            have = (n - m + i) // page + 1
            pages = s["page_table"][r, :have].long()
            per_head = []
            for h in range(c["hkv"]):
                best = torch.full((have,), float("-inf"), dtype=torch.float64, device="cuda")
                hi, lo = s["k_bounds"][pages, h, 0].double(), s["k_bounds"][pages, h, 1].double()
                for e in range(h * group, (h + 1) * group):
                    q = s["q"][t, e].double()
                    peak = float(q.abs().max())
                    unit = 2.0 ** (max(-126, math.ceil(math.log2(peak / 127))) if peak > 0 else -126)
                    qi = torch.round(q / unit)
                    best = torch.maximum(best, torch.where(qi > 0, qi * hi, qi * lo).sum(1) * unit)
                best = best * 4 * s["k_scale"][pages, h].double()
                best[:min(have, c["sink"])] = float("inf")
                best[max(0, have - c["recent"]):] = float("inf")
                order = np.lexsort((np.arange(have), -best.cpu().numpy()))[:c["budget"]]
                per_head.append(torch.from_numpy(np.sort(order).copy()).cuda())
            picked.append(per_head)
            t += 1
    return picked
