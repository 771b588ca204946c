"""The 8-bit paged K/V cache on the GPU against its 64-bit oracle (oracle/kv8.py): page
tables, append and page selection exactly, attention within the bound of
kv8_helpers.check_rows, and a run of them together."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import masked_flash_attention_attn_b200 as M
from masked_flash_attention_attn_b200 import mask as masks
from oracle import kv8 as O
from tests import kv8_helpers as H

pytestmark = pytest.mark.gpu
bf16 = torch.bfloat16


# ---- page tables ----------------------------------------------------------------------------
def run_tables(table, old, new, ring, state, page, tokens, positions=True, repeat=1):
    t = dict(page_table=H.i32(table), old_lens=H.i32(old), new_lens=H.i32(new), free_pages=H.i32(ring), free_state=H.i32(state),
             next_state=H.i32([-7] * 4), kv_lens=H.i32([-7] * len(old)), cu_seqlens_q=H.i32([-7] * (len(old) + 1)),
             slots=H.i32([-7] * tokens), positions=H.i32([-7] * tokens) if positions else None)
    for _ in range(repeat):
        M.attn_page_tables(page_size=page, **t)
    n = lambda x: None if x is None else x.cpu().numpy()  # noqa: E731
    return [n(t[k]) for k in ("page_table", "free_pages", "next_state", "kv_lens", "cu_seqlens_q", "slots", "positions")]


def tables_problem(seed, batch, page, width, head=None, spare=None, hi=None):
    rng = np.random.default_rng(seed)
    hi = hi or width * page
    old = rng.integers(0, hi + 1, batch)
    new = np.where(rng.random(batch) < 0.5, np.minimum(hi, old + rng.integers(0, 3 * page, batch)), rng.integers(0, hi + 1, batch))
    new[rng.random(batch) < 0.2] = 0
    pages = lambda x: (x + page - 1) // page  # noqa: E731
    grow = int(np.maximum(0, pages(new) - pages(old)).sum())
    used = int(pages(old).sum())
    spare = grow if spare is None else spare
    total = used + max(spare, grow, 1)
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((batch, width), -1, np.int32)
    at = 0
    for b in range(batch):
        table[b, :pages(old[b])] = perm[at:at + pages(old[b])]
        at += pages(old[b])
    head = int(rng.integers(0, total)) if head is None else head
    ring = np.full(total, -1, np.int32)
    ring[(head + np.arange(spare)) % total] = perm[used:used + spare]
    tokens = int(np.maximum(0, new - old).sum())
    return table, old, new, ring, [head, spare, 0, 0], tokens


def check_tables(table, old, new, ring, state, page, tokens, **kw):
    got = run_tables(table, old, new, ring, state, page, tokens, **kw)
    ref = O.page_tables(table, old, new, ring, state, page, tokens)
    for name, a, b in zip(("page_table", "free_pages", "next_state", "kv_lens", "cu", "slots", "positions"), got, ref):
        if a is not None:
            assert np.array_equal(a, b), name
    return ref


@pytest.mark.parametrize("batch,page,width", [(1, 16, 1), (1, 128, 9), (3, 16, 5), (40, 32, 17), (257, 64, 6), (1500, 16, 12), (16384, 16, 3)])
def test_tables_match_the_oracle(batch, page, width):
    table, old, new, ring, state, tokens = tables_problem(batch + page, batch, page, width)
    ref = check_tables(table, old, new, ring, state, page, tokens + 3)
    assert ref[2][2] == 0
    check_tables(table, old, new, ring, state, page, tokens, positions=False)
    check_tables(table, old, new, ring, state, page, tokens + 3, repeat=3)     # a repeated call gives the same


def test_tables_batches_around_48_kib_of_prefixes_in_a_new_process():
    # 12 bytes a request and the kernel's static shared memory; in a process in which no larger batch ran before
    code = ("from tests.test_gpu_kv8 import check_tables, tables_problem\n"
            "for batch in (2729, 2730, 4051, 4052, 4095, 4096, 16384, 4052):\n"
            "    t, old, new, ring, state, tokens = tables_problem(batch, batch, 16, 3)\n"
            "    check_tables(t, old, new, ring, state, 16, tokens)\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_tables_refuse_on_the_device_and_still_shrink():
    table, old, new, ring, state, tokens = tables_problem(5, 30, 16, 8)
    assert (new < old).any() and (new > old).any()
    short = [state[0], state[1] - 1, 0, 0]
    ref = check_tables(table, old, new, ring, short, 16, tokens)
    assert ref[2][2] == 1 and ref[2][3] == 1
    assert check_tables(table, old, new, ring, state, 16, tokens - 1)[2][2] == 3
    for wrong in (-1, 8 * 16 + 1, -2 ** 31, 2 ** 31 - 1):
        bad = new.copy()
        bad[7] = wrong
        assert check_tables(table, old, bad, ring, state, 16, tokens)[2][2] == 2


def test_tables_empty_batch_and_no_change():
    got = run_tables(np.zeros((0, 4), np.int32), [], [], [3, 1, 2], [2, 3, 0, 0], 16, 2)
    assert list(got[2]) == [2, 3, 0, 0] and list(got[4]) == [0] and list(got[5]) == [-1, -1]
    table = np.array([[4, 2]], np.int32)
    check_tables(table, np.array([20]), np.array([20]), np.array([0, 1, 3], np.int32), [1, 2, 0, 0], 16, 0)


def test_tables_every_page_of_a_full_ring_changes_hands():
    # all of the ring is free and taken; then all of it comes back
    ring = np.random.default_rng(1).permutation(64).astype(np.int32)
    table = np.full((4, 16), -1, np.int32)
    full = np.full(4, 16 * 16)
    ref = check_tables(table, np.zeros(4, int), full, ring, [63, 64, 0, 0], 16, 4 * 256)
    back = check_tables(ref[0], full, np.zeros(4, int), ref[1], ref[2], 16, 0)
    assert back[2][1] == 64 and sorted(back[1]) == list(range(64))


# ---- append -----------------------------------------------------------------------------------
def check_append(cache, k, v, slots, page):
    ref = [O.append(H.values(c), s.double().cpu().numpy(), b if b is None else b.cpu().numpy(), x.float().cpu().numpy(), slots, page)
           for c, s, b, x in ((cache.k, cache.k_scale, cache.k_bounds, k), (cache.v, cache.v_scale, None, v))]
    M.attn_kv8_append(cache, k, v, H.i32(slots))
    for (codes, scale, bounds), c, s, b in ((ref[0], cache.k, cache.k_scale, cache.k_bounds), (ref[1], cache.v, cache.v_scale, None)):
        np.testing.assert_array_equal(s.double().cpu().numpy(), scale)   # NaN equals NaN
        assert np.array_equal(H.values(c), codes)
        if bounds is not None and b is not None:
            assert np.array_equal(b.cpu().numpy().astype(int), bounds)


def slots_for(table, before, count, page):
    out = []
    for b, (o, n) in enumerate(zip(before, count)):
        out += [int(table[b, t // page]) * page + t % page for t in range(o, o + n)]
    return np.asarray(out, np.int32)


def draw_kv(seed, T, hkv, d, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    gain = torch.exp(spread * torch.randn(T, hkv, 1, generator=g))
    return [(torch.randn(T, hkv, d, generator=g) * gain).to(bf16).cuda() for _ in range(2)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,hkv", [(64, 3), (128, 1), (256, 2)])
def test_append_matches_the_oracle(page, d, hkv):
    before, count = [0, 1, page - 1, page, 2 * page + 5, 7], [2 * page + 3, 1, 2, 1, page, 0]
    lens = [a + b for a, b in zip(before, count)]
    cache = H.make_cache(page + d, 24, hkv, page, d, -14, -9)
    table = H.make_table(page, lens, page, 24)
    slots = slots_for(table, before, count, page)
    k, v = draw_kv(d + hkv, len(slots), hkv, d)
    check_append(cache, k, v, slots, page)
    check_append(cache, k, v, slots, page)       # the same call again: nothing grows, the same codes


def test_append_many_tokens_use_wider_ctas():
    page, hkv, d = 16, 8, 64
    before, count = [3, 0, 9], [700, 801, 1]
    table = H.make_table(2, [a + b for a, b in zip(before, count)], page, 110)
    cache = H.make_cache(3, 110, hkv, page, d, -14, -9)
    slots = slots_for(table, before, count, page)
    k, v = draw_kv(9, len(slots), hkv, d)
    check_append(cache, k, v, slots, page)


def test_append_strided_views_and_skipped_slots():
    page, hkv, d = 32, 4, 128
    g = torch.Generator().manual_seed(4)
    fused = torch.randn(50, 3 * hkv * d + 8, generator=g).to(bf16).cuda()
    k = fused[:, :hkv * d].view(50, hkv, d)
    v = fused[:, 2 * hkv * d:3 * hkv * d].view(50, hkv, d)
    assert not k.is_contiguous()
    cache = H.make_cache(5, 8, hkv, page, d, -14, -9)
    slots = slots_for(H.make_table(6, [64], page, 8), [7], [50], page)
    slots[10:13] = [-1, -2, -3]
    slots[30] = 8 * page                         # past the cache
    slots[31] = -2 ** 31
    slots[40] = -2
    check_append(cache, k, v, slots, page)


@pytest.mark.parametrize("page,d", [(16, 64), (64, 64), (128, 64), (64, 256), (128, 256)])
@pytest.mark.parametrize("gap", [1, 31, 128, 2047, 2048, 2049, 5000])
def test_append_between_stretches_of_skipped_slots(page, d, gap):
    # skipped in front, inside a page's tokens, between pages and behind the last token, as a padded step has them
    table = H.make_table(gap, [page + 7, 2 * page + 3, 40], page, 12)
    first, second, third = (slots_for(table[b:b + 1], [o], [n], page) for b, (o, n) in enumerate([(3, page + 4), (0, 2 * page + 3), (33, 7)]))
    skip = [-1] * gap
    for slots in ([skip, first, skip, second, third, skip], [first[:5], skip, first[5:9], skip, first[9:], second[:-1], skip, second[-1:], skip],
                  [first, second, third[:1], skip, third[1:2], skip, third[2:], [12 * page, -2], skip], [skip, [-2 ** 31, 2 ** 31 - 1]]):
        slots = np.concatenate([np.asarray(x, np.int32) for x in slots])
        cache = H.make_cache(page + d, 12, 1, page, d, -14, -9)
        k, v = draw_kv(gap, len(slots), 1, d)
        check_append(cache, k, v, slots, page)


def test_append_passes_long_stretches_of_skipped_slots_quickly():
    # 65536 slots of a captured step with 32 tokens in use. A thread that walks over the skipped slots before a token
    # one by one takes about 3 ms, a CTA that lists those behind a page's last token 130 slots at a time 0.17 ms
    cache = M.Kv8Cache(128, page_size=16, hkv=8, head_dim=128)
    k = torch.zeros(65536, 8, 128, dtype=bf16, device="cuda")

    def shortest(slots):
        s, times = H.i32(slots), []
        for _ in range(9):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            M.attn_kv8_append(cache, k, k, s)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    part, full = np.arange(32) * 16 + 48, np.arange(32) * 16 + 63
    skip = np.full(65536 - 32, -1)
    assert shortest(np.concatenate([skip, part])) < 1.0
    assert shortest(np.concatenate([part, skip])) - shortest(np.concatenate([full, skip])) < 0.08


def test_append_special_values():
    page, hkv, d = 16, 1, 64
    cache = H.make_cache(7, 12, hkv, page, d)
    k, v = draw_kv(8, 12 * 3, hkv, d)
    for x in (k, v):
        x[0] = 0                                 # a page of zeros
        x[1] = 0
        x[2] = 0
        x[3, 0, 5] = float("inf")
        x[4, 0, 6] = float("-inf")
        x[6, 0, 7] = float("nan")
        x[9] = float("nan")                      # no finite value
        x[10] = float("nan")
        x[11] = float("inf")
        x[12] = 3.3e38
        x[15] = 1e-40                            # below the least scale
        x[16] = -1e-40
        x[17] = 2.0 ** -133
        x[18] = 448.0                            # the border of an exponent
        x[21] = 452.0
        x[24] = 2.0 ** -126
    slots = np.concatenate([np.arange(3) + 16 * p for p in range(12)]).astype(np.int32)
    check_append(cache, k, v, slots, page)
    # a page that holds a NaN and an infinity grows
    big = [torch.full((1, hkv, d), 1e6, dtype=bf16).cuda() for _ in range(2)]
    check_append(cache, *big, np.asarray([16 + 3], np.int32), page)
    check_append(cache, *big, np.asarray([0 + 3], np.int32), page)


def test_append_token_by_token_equals_one_call():
    # ascending magnitudes: every token makes the scale grow or stay; values stay normal codes
    page, hkv, d = 16, 2, 128
    g = torch.Generator().manual_seed(11)
    x = torch.rand(40, hkv, d, generator=g) + 1.0
    x = (x * torch.exp2(torch.arange(40).div(8).floor())[:, None, None]).to(bf16).cuda()
    one, many = (M.Kv8Cache(3, page_size=page, hkv=hkv, head_dim=d) for _ in range(2))
    slots = H.i32(np.arange(40))
    M.attn_kv8_append(one, x, -x, slots)
    for t in range(40):
        M.attn_kv8_append(many, x[t:t + 1], -x[t:t + 1], slots[t:t + 1])
    for a, b in ((one.k_scale, many.k_scale), (one.v_scale, many.v_scale), (one.k_bounds, many.k_bounds)):
        assert torch.equal(a, b)
    # code by code: the second rounding of a value that was rounded before is exact
    assert torch.equal(one.k.view(torch.uint8), many.k.view(torch.uint8))
    assert torch.equal(one.v.view(torch.uint8), many.v.view(torch.uint8))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_append_bounds_hold_the_codes_when_any_scale_grows(d):
    # a caller's scales, growing by any factor: the bounds against the codes themselves
    page, hkv, pages = 16, 3, 60
    cache = H.make_cache(d, pages, hkv, page, d, 0, 0)
    g = torch.Generator().manual_seed(d)
    ratio = torch.rand(pages, hkv, generator=g) * 0.97 + 0.02
    ratio[0], ratio[1], ratio[2] = 0.95, 0.6093, 0.5          # codes 288 and 224 are rounded up by the first two
    cache.k_scale.copy_(ratio.cuda())
    k = torch.randn(pages * hkv * page * d, generator=g).mul(120).clamp(-448, 448).view(pages, hkv, page, d)
    k[:, :, :, 2], k[:, :, :, 3], k[:, :, :, 4], k[:, :, :, 5] = 288, 224, -288, -224
    cache.k.copy_(k.to(H.E4M3).cuda())
    x = cache.k.float()
    cache.k_bounds.copy_(torch.stack([torch.ceil(x.amax(2) / 4), torch.floor(x.amin(2) / 4)], 2).to(torch.int8))
    new = torch.zeros(pages, hkv, d, dtype=bf16, device="cuda")
    new[:, :, 7] = 448                                        # needs a scale of 1
    before = H.values(cache.k)                                # the bounds are of all its places
    M.attn_kv8_append(cache, new, new, H.i32(np.arange(pages) * page + page - 1))
    assert (cache.k_scale == 1).all()
    codes, b = H.values(cache.k), cache.k_bounds.cpu().numpy().astype(int)
    assert (4 * b[:, :, 0] >= codes.max(2)).all() and (4 * b[:, :, 1] <= codes.min(2)).all()
    # and no wider: 3 codes from the outward rounding of the old bound, half a step (2^-4) of the format, 4 codes of the new
    r = ratio.numpy()[:, :, None]
    top, low = np.maximum(before.max(2) * r, 0), np.minimum(before.min(2) * r, 0)
    assert (4 * b[:, :, 0] <= np.maximum((top + 3) * (1 + 2.0 ** -4) + 4.01, codes.max(2))).all()
    assert (4 * b[:, :, 1] >= np.minimum((low - 3) * (1 + 2.0 ** -4) - 4.01, codes.min(2))).all()


def test_append_without_bounds_and_empty():
    cache = M.Kv8Cache(4, page_size=16, hkv=2, head_dim=64, bounds=False)
    k, v = draw_kv(1, 5, 2, 64)
    check_append(cache, k, v, np.arange(20, 25).astype(np.int32), 16)
    M.attn_kv8_append(cache, k[:0], v[:0], H.i32([]))


# ---- attention ----------------------------------------------------------------------------------
def attend(seed, lens, qlens, *, hq, hkv, d, page, mask="causal", window=0, cache=None, table=None, q=None, scale=0.0, extra=0,
           max_q=None, plan=None, sample=400, width=None):
    pages = sum((n + page - 1) // page for n in lens) + 3
    cache = cache or H.make_cache(seed, pages, hkv, page, d)
    table = H.make_table(seed, lens, page, cache.num_pages, width) if table is None else table
    cu = H.cu_of(qlens)
    T = int(cu[-1])
    if q is None:
        q = torch.randn(T + extra, hq, d, generator=torch.Generator().manual_seed(seed)).to(bf16).cuda()
    m = {"causal": masks.causal, "full": masks.full, "sliding": lambda: masks.sliding_window(window)}[mask]()
    plan = plan or M.attn_kv8_plan(hq=hq, hkv=hkv, head_dim=d, page_size=page, mask=m, scale=scale, max_q_len=max_q or max(1, max(qlens)))
    out = torch.full((T + extra, hq, d), 7.0, dtype=bf16, device="cuda")
    lse = torch.full((T + extra, hq), 7.0, device="cuda")
    one = all(n == 1 for n in qlens) and not extra and seed % 2 == 0
    for _ in range(2):                           # the second run finds the counters as the first left them
        M.attn_kv8_fwd(plan, cache, q, H.i32(table), H.i32(lens), out, lse, cu_seqlens_q=None if one else H.i32(cu))
    rows = O.rows_of(lens, cu, T)
    H.check_rows(cache, q[:T], table, rows, out[:T], lse[:T], scale=scale or d ** -0.5, mask=mask, window=window, sample=sample)
    if extra:
        assert (out[T:] == 7).all() and (lse[T:] == 7).all()
    return cache, table, q, out, lse, plan


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_ragged(d, page):
    attend(d + page, [1, 15, 16, 17, 100, 0, 333, 1000], [1] * 8, hq=8, hkv=2, d=d, page=page)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (8, 1), (10, 2), (16, 1), (40, 1), (64, 2)])
def test_decode_groups(hq, hkv, d):
    attend(hq + d, [70, 513, 31], [1, 1, 1], hq=hq, hkv=hkv, d=d, page=16)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("mask,window", [("causal", 0), ("full", 0), ("sliding", 1), ("sliding", 37), ("sliding", 5000)])
def test_several_tokens(d, mask, window):
    # 0 tokens, more tokens than keys, one key, tokens over a page border
    attend(7 * d + window, [40, 3, 1, 600, 129, 257], [5, 7, 1, 0, 33, 2], hq=6, hkv=2, d=d, page=16, mask=mask, window=window, extra=3)


def test_more_tokens_than_the_plan_expects():
    attend(3, [300, 200], [70, 9], hq=8, hkv=2, d=128, page=32, max_q=1)
    attend(4, [300, 200], [1, 1], hq=8, hkv=2, d=128, page=32, max_q=64)


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (64, 16, 2), (256, 2, 1)])
def test_long_contexts_are_split_over_ctas(d, hq, hkv):
    attend(21, [30011, 1], [1, 1], hq=hq, hkv=hkv, d=d, page=64, sample=12)
    attend(22, [9000], [3], hq=hq, hkv=hkv, d=d, page=16, sample=12)


@pytest.mark.parametrize("d,hq,hkv,q", [(64, 8, 4, 1), (128, 8, 4, 1), (256, 4, 4, 1), (64, 8, 4, 6), (128, 32, 4, 2), (128, 32, 4, 4),
                                        (256, 16, 4, 3)])
def test_many_short_requests(d, hq, hkv, q):
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(q, 90, 350)]
    lens[7], lens[200] = 2000, 1500
    attend(30, lens, [q] * 350, hq=hq, hkv=hkv, d=d, page=16, sample=300)


@pytest.mark.parametrize("d,hq,hkv,page", [(128, 8, 2, 64), (64, 2, 2, 16), (256, 4, 2, 32)])
@pytest.mark.parametrize("batch,lo,hi", [(3, 9000, 20000), (16, 2000, 3000), (40, 300, 4000), (150, 200, 900), (333, 1, 700)])
def test_work_is_shared_out_whole(batch, lo, hi, d, hq, hkv, page):
    # few long items on many CTAs, about one piece per CTA, several items per CTA
    rng = np.random.default_rng(batch + d)
    lens = [int(x) for x in rng.integers(lo, hi + 1, batch)]
    lens[batch // 2] = 0
    attend(batch + d, lens, [1] * batch, hq=hq, hkv=hkv, d=d, page=page, sample=24)


@pytest.mark.parametrize("chunks", [295, 296, 297, 300, 591, 592, 593, 1200])
def test_work_near_the_number_of_ctas(chunks):
    # one KV head: the chunks (of 128 keys) of all requests about as many as CTAs
    lens = [128 * (chunks // 3)] * 2 + [128 * (chunks - 2 * (chunks // 3)) - 60]
    attend(chunks, lens, [1] * 3, hq=2, hkv=1, d=64, page=128, sample=6)


def test_any_scale():
    # scales that a caller wrote: any positive number
    cache = H.make_cache(3, 30, 2, 16, 128)
    g = torch.Generator().manual_seed(2)
    for s in (cache.k_scale, cache.v_scale):
        s.mul_(torch.rand(s.shape, generator=g).cuda() + 0.3)
    attend(6, [400, 37], [2, 1], hq=8, hkv=2, d=128, page=16, cache=cache)
    before, count = [3, 30], [20, 5]
    table = H.make_table(2, [a + b for a, b in zip(before, count)], 16, 30)
    slots = slots_for(table, before, count, 16)
    k, v = draw_kv(9, len(slots), 2, 128)
    ref = [O.append(H.values(c), s.double().cpu().numpy(), None, x.float().cpu().numpy(), slots, 16)
           for c, s, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v))]
    M.attn_kv8_append(cache, k, v, H.i32(slots))
    for (codes, scale, _), c, s in ((ref[0], cache.k, cache.k_scale), (ref[1], cache.v, cache.v_scale)):
        assert np.array_equal(s.double().cpu().numpy(), scale)
        # a quotient is rounded to fp32 before it is rounded to a code: a code next to a tie may be the neighbour
        got = H.values(c)
        assert np.mean(got != codes) < 1e-3 and np.all(np.abs(got - codes) <= np.maximum(2.0 ** -9, 2.0 ** -3 * np.abs(codes)))


def test_calls_that_are_refused():
    cache = H.make_cache(1, 8, 2, 16, 64)
    plan = M.attn_kv8_plan(hq=4, hkv=2, head_dim=64, page_size=16, mask=masks.causal())
    q = torch.zeros(1, 4, 64, dtype=bf16, device="cuda")
    table, lens = H.i32([[0, 1]]), H.i32([20])
    with pytest.raises(M.AttnError, match="INVALID"):
        M.attn_kv8_fwd(plan, cache, q, table, lens, q)                        # out is q
    sel, sc = H.i32(np.zeros((1, 2, 3))), torch.zeros(1, 2, 2, device="cuda")
    for kw in (dict(sink=-1), dict(recent=0), dict(sink=2, recent=2)):
        with pytest.raises(M.AttnError, match="INVALID"):
            M.attn_kv8_select(plan, cache, q, table, lens, sc, sel, **kw)
    window = M.attn_kv8_plan(hq=4, hkv=2, head_dim=64, page_size=16, mask=masks.sliding_window(5))
    with pytest.raises(M.AttnError, match="UNSUPPORTED"):
        M.attn_kv8_select(window, cache, q, table, lens, sc, sel)
    wide = M.attn_kv8_plan(hq=130, hkv=2, head_dim=64, page_size=16, mask=masks.causal())
    with pytest.raises(M.AttnError, match="UNSUPPORTED"):
        M.attn_kv8_select(wide, cache, torch.zeros(1, 130, 64, dtype=bf16, device="cuda"), table, lens, sc, sel)
    with pytest.raises(ValueError, match="cpu"):
        M.attn_kv8_fwd(plan, cache, q, table.cpu(), lens, torch.empty_like(q))
    ring = H.i32([0, 1])
    z = lambda n: H.i32(np.zeros(n))  # noqa: E731
    good = dict(page_table=table.clone(), old_lens=z(1), new_lens=z(1), free_pages=ring, free_state=z(4), page_size=16, next_state=z(4),
                kv_lens=z(1), cu_seqlens_q=z(2), slots=z(3))
    M.attn_page_tables(**good)
    for name, same in (("next_state", "free_state"), ("kv_lens", "new_lens"), ("kv_lens", "old_lens")):
        with pytest.raises(M.AttnError, match="INVALID"):
            M.attn_page_tables(**dict(good, **{name: good[same]}))
    M.attn_kv8_plan_destroy(plan)
    M.attn_kv8_plan_destroy(plan)
    with pytest.raises(ValueError, match="destroyed"):
        M.attn_kv8_fwd(plan, cache, q, table, lens, torch.empty_like(q))


def test_outputs_that_overlap_are_refused():
    cache = H.make_cache(1, 8, 2, 16, 64)
    plan = M.attn_kv8_plan(hq=4, hkv=2, head_dim=64, page_size=16, mask=masks.causal())
    q = torch.zeros(2, 4, 64, dtype=bf16, device="cuda")
    table, lens = H.i32([[0, 1], [2, 3]]), H.i32([20, 9])
    out = torch.zeros_like(q)
    for at in (0, 256 - 8):                      # out is 256 words
        with pytest.raises(M.AttnError, match="INVALID"):
            M.attn_kv8_fwd(plan, cache, q, table, lens, out, out.view(-1).view(torch.float32)[at:at + 8].view(2, 4))
    both = torch.zeros(2, 2, 2, device="cuda")
    with pytest.raises(M.AttnError, match="INVALID"):
        M.attn_kv8_select(plan, cache, q, table, lens, both, both.view(torch.int32))
    k = torch.zeros(29, 2, 64, dtype=bf16, device="cuda")
    with pytest.raises(M.AttnError, match="INVALID"):
        M.attn_kv8_gather(cache, table, H.i32([0, 20, 29]), k, k)
    shared = M.Kv8Cache.wrap(cache.k, cache.k, cache.k_scale, cache.v_scale)
    with pytest.raises(M.AttnError, match="INVALID"):
        M.attn_kv8_append(shared, k, k, H.i32(np.arange(29)))
    M.attn_kv8_fwd(plan, shared, q, table, lens, out)      # only read: keys that are the values too are fine


def test_scores_that_rise_along_the_keys_and_wide_scales():
    # every step raises the running maximum; the scales of the pages differ by 2^40
    page, d = 16, 128
    cache = H.make_cache(1, 20, 1, page, d)
    k = torch.ones(20, 1, page, d) * torch.linspace(0.1, 200, 20 * page).view(20, 1, page, 1)
    cache.k.copy_(k.to(H.E4M3).cuda())
    cache.k_scale.fill_(2.0 ** -4)
    cache.v_scale.copy_(torch.exp2(torch.arange(20).float() * 2 - 30)[:, None].cuda())
    table = np.arange(20, dtype=np.int32)[None]
    attend(2, [317], [1], hq=4, hkv=1, d=d, page=page, cache=cache, table=table, q=torch.full((1, 4, d), 1.0, dtype=bf16, device="cuda"))
    attend(2, [317], [1], hq=4, hkv=1, d=d, page=page, cache=cache, table=table, q=torch.full((1, 4, d), -1.0, dtype=bf16, device="cuda"))


@pytest.mark.parametrize("at", ["first", "middle", "last", "many"])
@pytest.mark.parametrize("d,hq,tokens,many", [(64, 8, 1, False), (128, 8, 1, False), (256, 8, 1, False), (128, 16, 1, False), (64, 8, 4, False),
                                              (128, 8, 4, False), (256, 8, 2, False), (128, 8, 1, True), (64, 16, 1, True), (256, 8, 2, True)])
def test_keys_far_below_one_that_dominates(d, hq, tokens, many, at):
    # one key 0 .. 60 nats above the others (each head another gap), its value 0: all of the output is the others'.
    # Requests share their pages, so that there are enough of them for a warp to have a large part of a request's keys.
    # Bound: a P is off by 2^-11 of the largest p of its 16 keys or by itself, exponents by the fp32 score sum and ex2, sums
    # over n keys, the result to bf16 (as in kv8_helpers.check_rows, but without its absolute term)
    page, n = 16, 3000
    batch = 1300 if many else 600
    cache = H.make_cache(d, n // page + 5, 1, page, d)
    table = H.make_table(d, [n], page, cache.num_pages)
    stars = {"first": [0], "middle": [1501], "last": [n - tokens], "many": list(range(7, n - tokens, 128 * 3))}[at]
    k, v = cache.k.view(torch.uint8), cache.v.view(torch.uint8)
    k[:, :, :, 0] = 0
    for star in stars:
        k[table[0, star // page], 0, star % page] = 0
        k[table[0, star // page], 0, star % page, 0] = 0x7E                    # 448
        v[table[0, star // page], 0, star % page] = 0
    cache.k_scale.fill_(2.0 ** -8)
    q = torch.randn(tokens, hq, d, generator=torch.Generator().manual_seed(d))
    gap = torch.tensor([0, 8, 12, 14, 17, 21, 30, 60.0])[torch.arange(hq) % 8]
    q[:, :, 0] = gap / (d ** -0.5 * 448 * 2.0 ** -8)
    q = q.to(bf16).cuda()
    plan = M.attn_kv8_plan(hq=hq, hkv=1, head_dim=d, page_size=page, mask=masks.causal(), max_q_len=tokens)
    out, lse = M.forward_kv8(plan, cache, q.repeat(batch, 1, 1), H.i32(np.repeat(table, batch, 0)), H.i32([n] * batch),
                             H.i32(H.cu_of([tokens] * batch)))
    out, lse = out.view(batch, tokens, hq, d), lse.view(batch, tokens, hq)
    kk, vv = H.Keys(cache).of(table[0], n, 0)
    for t in range(tokens):
        hi = n - tokens + t + 1
        step = np.arange(0, hi, 16)
        va = np.abs(vv[:hi])
        for a in range(hq):
            qa = q[t, a].double().cpu().numpy()
            s = kk[:hi] @ qa * d ** -0.5
            p = np.exp(s - s.max())
            z, ref = p.sum(), p @ vv[:hi]
            top = np.repeat(np.maximum.reduceat(p, step), 16)[:hi]
            dp = (d + 4) * 2.0 ** -24 * (np.abs(kk[:hi]) @ np.abs(qa)).max() * d ** -0.5 + 2.0 ** -21
            tol = np.minimum(p, 2.0 ** -11 * top) @ va + (2 * dp + (hi + 64) * 2.0 ** -23) * (p @ va)
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)         # bf16 rounds the value that is off by tol
            for b in (0, batch // 2, batch - 1):
                err = np.abs(out[b, t, a].double().cpu().numpy() - ref / z)
                assert (err <= tol / z).all(), (b, t, a, float(gap[a]), float((err * z / tol).max()), float(err.max() * z / np.abs(ref).max()))
                assert abs(float(lse[b, t, a]) - (s.max() + np.log(z))) <= dp + (hi + 64) * 2.0 ** -23 + abs(s.max()) * 2.0 ** -22


@pytest.mark.parametrize("mag", [1e-30, 2.0 ** -20, 300.0, 1e30])
def test_query_magnitudes(mag):
    cache = H.make_cache(4, 20, 2, 16, 64)
    cache.k_scale.mul_(min(1.0, 1.0 / mag) if mag > 1 else 1.0)
    q = (torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)) * mag).to(bf16).cuda()
    q[1, 2] = 0
    attend(6, [100, 37], [1, 1], hq=4, hkv=2, d=64, page=16, cache=cache, q=q)


def test_softmax_scale_and_strided_queries():
    attend(8, [100, 37], [2, 1], hq=4, hkv=2, d=64, page=16, scale=0.37)
    fused = torch.randn(3, 4 * 64 + 256, generator=torch.Generator().manual_seed(1)).to(bf16).cuda()
    attend(9, [100, 37], [2, 1], hq=4, hkv=2, d=64, page=16, q=fused[:, :256].view(3, 4, 64))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_unused_slots_and_hidden_keys_may_hold_nan(d):
    page, lens, qlens = 32, [75, 40], [4, 1]
    cache = H.make_cache(d, 10, 2, page, d)
    table = H.make_table(1, lens, page, 10)
    kw = dict(hq=4, hkv=2, d=d, page=page, cache=cache, table=table)
    _, _, q, clean, lse, _ = attend(12, lens, qlens, **kw)
    k, v = cache.k.view(torch.uint8), cache.v.view(torch.uint8)
    used = np.zeros((10, page), bool)
    for b, n in enumerate(lens):
        for j in range(n):
            used[table[b, j // page], j % page] = True
    poison = torch.from_numpy(~used).cuda()[:, None, :, None].expand(10, 2, page, d)
    k[poison] = 0x7F
    v[poison] = 0xFF
    _, _, _, out, lse2, _ = attend(12, lens, qlens, **kw)
    assert torch.equal(out, clean) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_nan_shows_in_the_rows_that_see_its_page(d):
    # four draft tokens over a page border: a NaN in the last page's key or value reaches the rows that see
    # the page, in the heads it was written to, and no other row
    page, lens, qlens = 32, [66, 40], [4, 1]
    cache = H.make_cache(d, 10, 2, page, d)
    table = H.make_table(1, lens, page, 10)
    plan = M.attn_kv8_plan(hq=4, hkv=2, head_dim=d, page_size=page, mask=masks.causal(), max_q_len=4)
    q = torch.randn(5, 4, d, generator=torch.Generator().manual_seed(1)).to(bf16).cuda()
    args = (plan, cache, q, H.i32(table), H.i32(lens), H.i32(H.cu_of(qlens)))
    k, v = draw_kv(5, 2, 2, d)
    slots = H.i32([table[0, 2] * page, table[0, 2] * page + 1])
    M.attn_kv8_append(cache, k, v, slots)
    clean, lse = M.forward_kv8(*args)
    for x in (k, v):
        bad = x.clone()
        bad[1, 1, 7] = float("nan")              # position 65, head 1
        M.attn_kv8_append(cache, bad if x is k else k, bad if x is v else v, slots)
        out, l2 = M.forward_kv8(*args)
        assert torch.equal(out[[0, 1, 4]], clean[[0, 1, 4]]) and torch.equal(l2[[0, 1, 4]], lse[[0, 1, 4]])
        assert torch.equal(out[2:4, :2], clean[2:4, :2]) and torch.equal(l2[2:4, :2], lse[2:4, :2])
        assert out[2:4, 2:].isnan().all()
        assert l2[2:4, 2:].isnan().all() if x is k else torch.equal(l2, lse)
        ko, vo = (torch.zeros(66, 2, d, dtype=bf16, device="cuda") for _ in range(2))
        M.attn_kv8_gather(cache, H.i32(table), H.i32([0, 66]), ko, vo)
        assert (ko if x is k else vo)[64:, 1].isnan().all() and ko[:, 0].isfinite().all() and vo[:64].isfinite().all()
        M.attn_kv8_append(cache, k, v, slots)    # place 0 again: the page is new
        out, l2 = M.forward_kv8(*args)
        assert torch.equal(out, clean) and torch.equal(l2, lse)
    # a token behind the NaN keeps it; selection puts the page first
    bad = k.clone()
    bad[0, 0, 0] = float("nan")
    middle = H.i32([table[0, 1] * page, table[0, 1] * page + 1])
    M.attn_kv8_append(cache, bad, v, middle)
    M.attn_kv8_append(cache, k[1:], v[1:], middle[1:])
    assert cache.k_scale[table[0, 1], 0].isnan() and cache.k_scale[table[0, 1], 1].isfinite()
    sel = check_select(cache, q[:1], table[:1], [66], [1], 2, 0, 1, 4, fwd=False)
    assert sel[0, 0].tolist() == [1, 2]


def test_pages_outside_the_cache_read_as_zeros_and_bad_lengths_are_clamped():
    page, d = 16, 64
    cache = H.make_cache(3, 10, 1, page, d)
    table = H.make_table(2, [100], page, 10)
    table[0, 2], table[0, 4] = -1, 10
    attend(5, [100], [1], hq=4, hkv=1, d=d, page=page, cache=cache, table=table)
    # lengths past the table, negative ones, offsets past the tokens: memory-safe, clamped
    plan = M.attn_kv8_plan(hq=4, hkv=1, head_dim=d, page_size=page, mask=masks.causal())
    q = torch.randn(3, 4, d, device="cuda").to(bf16)
    t3 = H.i32(np.repeat(H.make_table(2, [100], page, 10), 3, 0))
    out, lse = M.forward_kv8(plan, cache, q, t3, H.i32([2 ** 31 - 1, -5, 100]))
    assert out[0].isfinite().all() and (out[1] == 0).all() and (lse[1] == float("-inf")).all()
    M.forward_kv8(plan, cache, q, t3, H.i32([100, 100, 100]), H.i32([0, 1, 2 ** 31 - 1, -4]))
    torch.cuda.synchronize()


def test_cache_larger_than_2_31_bytes():
    page, hkv, d = 128, 8, 256
    pages = 8300                                  # 2.18e9 bytes in each of K and V
    cache = M.Kv8Cache(pages, page_size=page, hkv=hkv, head_dim=d, bounds=False)
    small = H.make_cache(5, 4, hkv, page, d)
    for a, b in ((cache.k, small.k), (cache.v, small.v)):
        a.view(torch.uint8)[-4:] = b.view(torch.uint8)
    cache.k_scale[-4:], cache.v_scale[-4:] = small.k_scale, small.v_scale
    q = torch.randn(2, 8, d, generator=torch.Generator().manual_seed(1)).to(bf16).cuda()
    plan = M.attn_kv8_plan(hq=8, hkv=hkv, head_dim=d, page_size=page, mask=masks.causal())
    lens = [300, 90]
    low = np.array([[1, 3, 0], [2, 0, 0]], np.int32)
    a, la = M.forward_kv8(plan, small, q, H.i32(low), H.i32(lens))
    b, lb = M.forward_kv8(plan, cache, q, H.i32(low + pages - 4), H.i32(lens))
    assert torch.equal(a, b) and torch.equal(la, lb)
    k, v = draw_kv(1, 3, hkv, d)
    slots = np.arange(3) + (pages - 1) * page + 90 - 90
    M.attn_kv8_append(cache, k, v, H.i32(slots))
    M.attn_kv8_append(small, k, v, H.i32(np.arange(3) + 3 * page))
    assert torch.equal(cache.k.view(torch.uint8)[-4:], small.k.view(torch.uint8)) and torch.equal(cache.k_scale[-4:], small.k_scale)
    ks, vs = (torch.empty(390, hkv, d, dtype=bf16, device="cuda") for _ in range(2))
    kb, vb = torch.empty_like(ks), torch.empty_like(vs)
    cu = H.i32([0, 300, 390])
    M.attn_kv8_gather(small, H.i32(low), cu, ks, vs)
    M.attn_kv8_gather(cache, H.i32(low + pages - 4), cu, kb, vb)
    assert torch.equal(ks, kb) and torch.equal(vs, vb)


# ---- gather and long queries ----------------------------------------------------------------------
@pytest.mark.parametrize("d,hkv,page", [(64, 3, 16), (128, 8, 64), (256, 1, 128)])
def test_gather(d, hkv, page):
    lens = [5, 0, 200, page, 1]
    cache = H.make_cache(d, 40, hkv, page, d)
    table = H.make_table(3, lens, page, 40)
    table[2, 1] = 40
    cu = H.cu_of(lens)
    k, v = (torch.full((int(cu[-1]) + 9, hkv, d), 7.0, dtype=bf16, device="cuda") for _ in range(2))
    M.attn_kv8_gather(cache, H.i32(table), H.i32(cu), k, v)
    keys = H.Keys(cache)
    for b, n in enumerate(lens):
        for h in range(hkv):
            rk, rv = keys.of(table[b], n, h)
            for x, r in ((k, rk), (v, rv)):
                got = x[int(cu[b]):int(cu[b + 1]), h].float().cpu().numpy()
                assert np.array_equal(got, r.astype(np.float32))          # power-of-two scales: exact
    assert (k[int(cu[-1]):] == 7).all() and (v[int(cu[-1]):] == 7).all()


def check_gathered(cache, table, lens):
    """The requests' cached tokens, gathered, against the oracle's values (power-of-two scales: exact)."""
    cu = H.cu_of(lens)
    k, v = (torch.empty(int(cu[-1]), cache.hkv, cache.head_dim, dtype=bf16, device="cuda") for _ in range(2))
    M.attn_kv8_gather(cache, H.i32(table), H.i32(cu), k, v)
    keys = H.Keys(cache)
    for b, n in enumerate(lens):
        for h in range(cache.hkv):
            for x, r in zip((k, v), keys.of(table[b], int(n), h)):
                assert np.array_equal(x[int(cu[b]):int(cu[b + 1]), h].float().cpu().numpy(), r.astype(np.float32))


@pytest.mark.parametrize("page,d", [(16, 64), (64, 128)])
def test_gather_writes_zeros_past_the_tables_capacity(page, d):
    cache = H.make_cache(d, 6, 2, page, d)
    table = np.array([[0, 1], [2, 3], [4, 5]], np.int32)
    lens = [2 * page + 9, 5, 3 * page]                                    # a row of the table holds 2 pages
    cu = H.cu_of(lens)
    k, v = (torch.full((int(cu[-1]) + 3, 2, d), 7.0, dtype=bf16, device="cuda") for _ in range(2))
    M.attn_kv8_gather(cache, H.i32(table), H.i32(cu), k, v)
    keys = H.Keys(cache)
    for b, n in enumerate(lens):
        held = min(n, 2 * page)
        for h in range(2):
            for x, r in zip((k, v), keys.of(table[b], held, h)):
                got = x[int(cu[b]):int(cu[b + 1]), h].float().cpu().numpy()
                assert np.array_equal(got[:held], r.astype(np.float32)) and (got[held:] == 0).all()
    assert (k[int(cu[-1]):] == 7).all() and (v[int(cu[-1]):] == 7).all()


def test_gather_rounds_other_scales_to_nearest():
    cache = H.make_cache(1, 4, 2, 16, 64)
    cache.k_scale.mul_(1.37)
    k, v = (torch.empty(64, 2, 64, dtype=bf16, device="cuda") for _ in range(2))
    M.attn_kv8_gather(cache, H.i32([[0, 1, 2, 3]]), H.i32([0, 64]), k, v)
    ref = (cache.k.float() * cache.k_scale[:, :, None, None]).transpose(1, 2).reshape(64, 2, 64).to(bf16)
    assert torch.equal(k, ref)


def test_long_chunk_through_the_masked_forward():
    # the gathered form and the streaming form, each against the oracle on the cached values. The
    # masked forward rounds P to bf16 (half a step: 2^-8) and takes a share of its exponentials from
    # a polynomial (relative error below 2^-13); its lse is held to 1e-3 everywhere in this suite
    page, lens, qlens = 32, [500, 300], [200, 33]
    cache, table, q, out, lse, _ = attend(14, lens, qlens, hq=8, hkv=2, d=128, page=page, sample=200)
    k, v = (torch.empty(sum(lens), 2, 128, dtype=bf16, device="cuda") for _ in range(2))
    M.attn_kv8_gather(cache, H.i32(table), H.i32(H.cu_of(lens)), k, v)
    plan = M.attn_plan(hq=8, hkv=2, head_dim=128, cu_seqlens_q=H.cu_of(qlens), cu_seqlens_k=H.cu_of(lens), mask=masks.causal())
    o2, l2 = M.forward(plan, q, k, v)
    H.check_rows(cache, q, table, O.rows_of(lens, H.cu_of(qlens), sum(qlens)), o2, l2, scale=128 ** -0.5, sample=200,
                 p_err=2.0 ** -8, exp_err=2.0 ** -13, lse_abs=1e-3)


# ---- selection ----------------------------------------------------------------------------------
def check_select(cache, q, table, lens, qlens, k, sink, recent, hq, mask="causal", fwd=True):
    cu = H.cu_of(qlens)
    T = int(cu[-1])
    m = masks.causal() if mask == "causal" else masks.full()
    plan = M.attn_kv8_plan(hq=hq, hkv=cache.hkv, head_dim=cache.head_dim, page_size=cache.page_size, mask=m, max_q_len=max(qlens))
    scores = torch.full((T, cache.hkv, table.shape[1]), 7.0, device="cuda")
    sel = torch.full((T, cache.hkv, k), -9, dtype=torch.int32, device="cuda")
    args = (plan, cache, q, H.i32(table), H.i32(lens))
    M.attn_kv8_select(*args, scores, sel, cu_seqlens_q=H.i32(cu), sink=sink, recent=recent)
    rows = O.rows_of(lens, cu, T)
    ref, sc = O.select(q.float().cpu().numpy(), cache.k_bounds.cpu().numpy().astype(float), cache.k_scale.double().cpu().numpy(),
                       table, rows, cache.page_size, k, sink, recent, mask)
    assert np.array_equal(sel.cpu().numpy(), ref)
    got = scores.cpu().numpy()
    for (t, h), x in sc.items():
        assert np.array_equal(got[t, h, :len(x)], x.astype(np.float32)) and (got[t, h, len(x):] == 7).all()
    if fwd:
        out, lse = M.forward_kv8(*args, H.i32(cu), selected=sel)
        H.check_rows(cache, q, table, rows, out, lse, scale=cache.head_dim ** -0.5, mask=mask, selected=ref, sample=200)
    return sel


@pytest.mark.parametrize("d,hq,hkv,page", [(64, 3, 3, 16), (128, 8, 2, 32), (256, 10, 2, 16), (128, 64, 1, 64), (64, 16, 8, 128)])
@pytest.mark.parametrize("k,sink,recent", [(1, 0, 1), (7, 1, 2), (40, 0, 3)])
def test_select_and_attend(d, hq, hkv, page, k, sink, recent):
    lens, qlens = [1, 20 * page - 3, 9 * page, 0, 500], [1, 3, 1, 1, 2]
    cache = H.make_cache(d + page, 80 + 500 // page, hkv, page, d)
    table = H.make_table(k, lens, page, cache.num_pages)
    q = torch.randn(sum(qlens), hq, d, generator=torch.Generator().manual_seed(k)).to(bf16).cuda()
    check_select(cache, q, table, lens, qlens, k, sink, recent, hq)


def test_select_ties_long_rows_and_special_queries():
    page, d = 16, 64
    cache = H.make_cache(4, 1700, 1, page, d)
    lens = [1650 * page - 5]
    table = H.make_table(9, lens, page, 1700)
    q = torch.randn(1, 2, d, generator=torch.Generator().manual_seed(2)).to(bf16).cuda()
    check_select(cache, q, table, lens, [1], 64, 1, 2, 2, fwd=False)
    check_select(cache, q * 0, table, lens, [1], 64, 1, 2, 2, fwd=False)          # every score 0: the lowest pages
    q[0, 0, 3], q[0, 1, 7], q[0, 1, 9] = float("inf"), float("nan"), float("-inf")
    check_select(cache, q, table, lens, [1], 64, 0, 1, 2, fwd=False)
    table[0, ::3] = -1                                                            # pages outside the cache come last
    check_select(cache, q, table, lens, [1], 1200, 0, 1, 2, fwd=False)


@pytest.mark.parametrize("pages", [1024, 1025, 4096, 4097, 9001])
def test_select_row_lengths(pages):
    # around the numbers of keys that the select kernel's threads keep
    page, d = 16, 64
    cache = H.make_cache(pages, pages, 1, page, d)
    table = np.random.default_rng(pages).permutation(pages).astype(np.int32)[None]
    q = torch.randn(1, 2, d, generator=torch.Generator().manual_seed(2)).to(bf16).cuda()
    for k in (1, 500):
        check_select(cache, q, table, [pages * page - 3], [1], k, 0, 1, 2, fwd=False)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens,cap", [(1, 512), (1, 513), (13, 512), (12, 1024), (11, 1024), (12, 1025)])
def test_select_rows_of_every_length_and_ties(d, tokens, cap):
    # 8 heads: 96 rows and 512 pages are where one launch turns into two
    page, rng = 16, np.random.default_rng(cap + tokens)
    cache = H.make_cache(d, cap, 8, page, d)
    table = np.stack([rng.permutation(cap) for _ in range(tokens)]).astype(np.int32)
    pages = [cap, 1, 2, 15, 16, 17, 127, 128, 129, 255, 257, 300, 40][:tokens]
    table[-1, 3::5] = -1
    lens = [n * page - int(rng.integers(0, page)) for n in pages]
    q = torch.randn(tokens, 24, d, generator=torch.Generator().manual_seed(cap)).to(bf16).cuda()
    q[-1, :3] = 0                                                    # every score of one row 0: ties
    for k in (3, 33):
        check_select(cache, q, table, lens, [1] * tokens, k, 1, 1, 24, fwd=False)
    # few different bounds, so scores agree in their leading digits or altogether
    cache.k_bounds[:, :, :, 1:] = 0
    cache.k_bounds[:, :, :, 0] = (cache.k_bounds[:, :, :, 0] // 16) * 16
    cache.k_scale.fill_(0.25)
    check_select(cache, q, table, lens, [1] * tokens, 33, 0, 2, 24, fwd=False)


def test_select_full_mask_sees_every_token():
    cache = H.make_cache(4, 40, 2, 16, 64)
    table = H.make_table(9, [300, 200], 16, 40)
    q = torch.randn(5, 4, 64, generator=torch.Generator().manual_seed(2)).to(bf16).cuda()
    check_select(cache, q, table, [300, 200], [3, 2], 6, 1, 1, 4, mask="full")


def test_selected_lists_of_the_caller():
    # unsorted lists, entries that see nothing, every head its own
    page, d = 16, 64
    cache = H.make_cache(6, 20, 2, page, d)
    table = H.make_table(3, [200], page, 20)
    sel = np.array([[[5, -1, 2, 999], [12, 0, 1, -1]]], np.int32)
    plan = M.attn_kv8_plan(hq=4, hkv=2, head_dim=d, page_size=page, mask=masks.causal())
    q = torch.randn(1, 4, d, generator=torch.Generator().manual_seed(2)).to(bf16).cuda()
    out, lse = M.forward_kv8(plan, cache, q, H.i32(table), H.i32([200]), selected=H.i32(sel))
    H.check_rows(cache, q, table, [(0, 199, 200)], out, lse, scale=d ** -0.5, selected=np.where(sel > 12, -1, sel))
    none = H.i32(np.full((1, 2, 3), -1))
    out, lse = M.forward_kv8(plan, cache, q, H.i32(table), H.i32([200]), selected=none)
    assert (out == 0).all() and (lse == float("-inf")).all()


# ---- together -----------------------------------------------------------------------------------
class Server:
    """A small serving loop over the operators; the oracle keeps every request's tokens."""

    def __init__(self, seed, batch=5, hq=8, hkv=2, d=64, page=16, pages=90, width=20, tokens=64, budget=None):
        self.hq, self.hkv, self.d, self.page, self.width, self.tokens = hq, hkv, d, page, width, tokens
        self.rng = np.random.default_rng(seed)
        self.g = torch.Generator().manual_seed(seed)
        self.cache = M.Kv8Cache(pages, page_size=page, hkv=hkv, head_dim=d)
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.lens, self.want, self.kv = z(batch, width) - 1, z(batch), z(batch), z(batch)
        self.ring = H.i32(self.rng.permutation(pages))
        self.state, self.next = H.i32([pages // 2, pages, 0, 0]), z(4)
        self.cu, self.slots, self.pos = z(batch + 1), z(tokens), z(tokens)
        self.k, self.v, self.q = (torch.zeros(tokens, n, d, dtype=bf16, device="cuda") for n in (hkv, hkv, hq))
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros(tokens, hq, device="cuda")
        self.plan = M.attn_kv8_plan(hq=hq, hkv=hkv, head_dim=d, page_size=page, mask=masks.causal(), max_q_len=4)
        self.budget = budget
        if budget:
            self.scores = torch.zeros(tokens, hkv, width, device="cuda")
            self.sel = z(tokens, hkv, budget)

    def launch(self):
        M.attn_page_tables(page_table=self.table, old_lens=self.lens, new_lens=self.want, free_pages=self.ring, free_state=self.state,
                           page_size=self.page, next_state=self.next, kv_lens=self.kv, cu_seqlens_q=self.cu, slots=self.slots,
                           positions=self.pos)
        M.attn_kv8_append(self.cache, self.k, self.v, self.slots)
        if self.budget:
            M.attn_kv8_select(self.plan, self.cache, self.q, self.table, self.kv, self.scores, self.sel, cu_seqlens_q=self.cu, recent=2)
        M.attn_kv8_fwd(self.plan, self.cache, self.q, self.table, self.kv, self.out, self.lse, cu_seqlens_q=self.cu,
                       selected=self.sel if self.budget else None)
        self.lens.copy_(self.kv)
        self.state.copy_(self.next)

    def step(self, want, launch=None):
        old = self.lens.cpu().numpy()
        self.want.copy_(H.i32(want))
        for x in (self.k, self.v, self.q):
            x.copy_(torch.randn(x.shape, generator=self.g).to(bf16))
        # the oracle's step on the state before it
        tab = O.page_tables(self.table.cpu().numpy(), old, want, self.ring.cpu().numpy(), self.state.cpu().numpy(), self.page, self.tokens)
        ref = [O.append(H.values(c), s.double().cpu().numpy(), b, x.float().cpu().numpy(), tab[5], self.page)
               for c, s, b, x in ((self.cache.k, self.cache.k_scale, self.cache.k_bounds.cpu().numpy(), self.k),
                                  (self.cache.v, self.cache.v_scale, None, self.v))]
        (launch or self.launch)()
        got = [x.cpu().numpy() for x in (self.table, self.ring, self.state, self.lens, self.cu, self.slots, self.pos)]
        for a, b in zip(got, tab):
            assert np.array_equal(a, b)
        for (codes, scale, bounds), c, s in ((ref[0], self.cache.k, self.cache.k_scale), (ref[1], self.cache.v, self.cache.v_scale)):
            assert np.array_equal(H.values(c), codes) and np.array_equal(s.double().cpu().numpy(), scale)
            if bounds is not None:
                assert np.array_equal(self.cache.k_bounds.cpu().numpy(), bounds)
        rows = O.rows_of(got[3], got[4], self.tokens)
        sel = None
        if self.budget:
            sel, _ = O.select(self.q.float().cpu().numpy(), self.cache.k_bounds.cpu().numpy().astype(float),
                              self.cache.k_scale.double().cpu().numpy(), got[0], rows, self.page, self.budget, 1, 2)
            live = [t for t, r in enumerate(rows) if r is not None]
            assert np.array_equal(self.sel.cpu().numpy()[live], sel[live])
        H.check_rows(self.cache, self.q, got[0], rows, self.out, self.lse, scale=self.d ** -0.5, selected=sel, sample=60)
        return got

    def wants(self, n):
        """Prompts, decode steps, draft tokens that are rejected, ends and a fresh prompt."""
        lens = [30, 1, 17, 0, 9]
        yield list(lens)
        for i in range(n):
            lens = [x + (1 if i % 3 else 3) if x else 0 for x in lens]
            yield list(lens)
            if i % 3 == 0:
                lens = [max(0, x - 2) for x in lens]        # two of three draft tokens rejected
                yield list(lens)
            if i == 3:
                lens[2] = 0
                lens[3] = 40
                yield list(lens)


@pytest.mark.parametrize("budget", [None, 4])
def test_serving_steps(budget):
    s = Server(1, budget=budget)
    for want in s.wants(6):
        assert s.step(want)[2][2] == 0


@pytest.mark.parametrize("budget", [None, 4])
def test_serving_steps_from_a_captured_graph(budget):
    s = Server(2, budget=budget)
    it = s.wants(7)
    s.step(next(it))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.launch()                               # want == lens: nothing grows
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.launch()
    for want in it:
        assert s.step(want, launch=graph.replay)[2][2] == 0


def test_calls_without_tokens_change_nothing():
    cache = H.make_cache(1, 8, 2, 16, 64)
    plan = M.attn_kv8_plan(hq=4, hkv=2, head_dim=64, page_size=16, mask=masks.causal())
    out, lse = M.forward_kv8(plan, cache, torch.zeros(0, 4, 64, dtype=bf16, device="cuda"), H.i32(np.zeros((0, 3))), H.i32([]))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # requests, but no query tokens; query rows, but no requests
    q = torch.ones(3, 4, 64, dtype=bf16, device="cuda")
    out, lse = torch.full_like(q, 7), torch.full((3, 4), 7.0, device="cuda")
    M.attn_kv8_fwd(plan, cache, q, H.i32([[0], [1]]), H.i32([5, 9]), out, lse, cu_seqlens_q=H.i32([0, 0, 0]))
    M.attn_kv8_fwd(plan, cache, q, H.i32(np.zeros((0, 1))), H.i32([]), out, lse, cu_seqlens_q=H.i32([0]))
    sel, sc = H.i32(np.full((3, 2, 2), 5)), torch.zeros(3, 2, 1, device="cuda")
    M.attn_kv8_select(plan, cache, q, H.i32([[0], [1]]), H.i32([5, 9]), sc, sel, cu_seqlens_q=H.i32([0, 0, 0]))
    M.attn_kv8_fwd(plan, cache, q, H.i32([[0], [1]]), H.i32([5, 9]), out, lse, cu_seqlens_q=H.i32([0, 0, 0]), selected=sel)
    assert (out == 7).all() and (lse == 7).all() and (sel == 5).all()


def test_two_captured_graphs_of_two_plans_and_eager_calls_between():
    # replays of both graphs and eager calls share a cache, each plan has its own workspace
    lens = [5000, 3000]
    cache, table, q, out, lse, _ = attend(41, lens, [1, 1], hq=8, hkv=2, d=128, page=16, sample=10)
    t, n = H.i32(table), H.i32(lens)
    plans = [M.attn_kv8_plan(hq=8, hkv=2, head_dim=128, page_size=16, mask=masks.causal()) for _ in range(3)]
    outs, graphs = [torch.empty_like(out) for _ in range(3)], []
    torch.cuda.synchronize()
    for p, o in zip(plans[:2], outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            M.attn_kv8_fwd(p, cache, q, t, n, o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        M.attn_kv8_fwd(plans[2], cache, q, t, n, outs[2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)


@pytest.mark.parametrize("raw", [False, True])
def test_results_of_a_call_on_another_stream_are_of_its_pool(raw):
    lens = [900] * 40
    cache, table, q, out, lse, plan = attend(42, lens, [1] * 40, hq=32, hkv=8, d=128, page=16, sample=10)
    t, n = H.i32(table), H.i32(lens)
    s = torch.cuda.Stream()
    for _ in range(2):
        torch.cuda.synchronize()
        x, y = torch.empty_like(out), torch.empty_like(lse)
        at = {x.data_ptr(), y.data_ptr()}
        torch.cuda._sleep(10_000_000)
        x.fill_(3)                               # still to come on the current stream when its block is free again
        y.fill_(3)
        del x, y
        a, b = M.forward_kv8(plan, cache, q, t, n, stream=s.cuda_stream if raw else s)
        assert not at & {a.data_ptr(), b.data_ptr()}
        torch.cuda.synchronize()
        assert torch.equal(a, out) and torch.equal(b, lse)
        del a, b


def test_two_plans_on_two_streams():
    lens = [9000, 20]
    cache, table, q, out, lse, _ = attend(40, lens, [1, 1], hq=8, hkv=2, d=128, page=16, sample=10)
    t, n = H.i32(table), H.i32(lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    plans = [M.attn_kv8_plan(hq=8, hkv=2, head_dim=128, page_size=16, mask=masks.causal()) for _ in range(2)]
    outs = [torch.empty_like(out) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, p, o in zip(streams, plans, outs):
            M.attn_kv8_fwd(p, cache, q, t, n, o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)       # and the same as before: no run-to-run difference
