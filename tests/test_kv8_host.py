"""CPU tests of the 8-bit paged cache: the binding's refusals (before any library call), the C
ABI's, and pins of the oracle."""
import ctypes

import numpy as np
import pytest
import torch

import masked_flash_attention_attn_b200 as M
from masked_flash_attention_attn_b200 import kv8
from masked_flash_attention_attn_b200 import mask as masks
from oracle import decode_e4m3
from oracle import kv8 as O

E4M3, bf16, i32 = torch.float8_e4m3fn, torch.bfloat16, torch.int32


# ---- the oracle ---------------------------------------------------------------------------------
def test_e4m3_rounding_is_to_the_nearest_code():
    codes = np.unique(decode_e4m3(np.arange(256)))
    codes = codes[np.isfinite(codes)]
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=2000) * np.exp2(rng.integers(-12, 9, 2000)), codes, (codes[1:] + codes[:-1]) / 2, [0.0, 460.0, -1e9]])
    got = O.e4m3_round(x)
    near = np.abs(np.clip(x, -448, 448)[:, None] - codes).min(1)
    assert np.array_equal(np.abs(got - np.clip(x, -448, 448)), near)
    lib = torch.from_numpy(np.clip(x, -448, 448)).float().to(E4M3).float().numpy()
    assert np.array_equal(got, lib)                       # ties too
    assert np.isnan(O.e4m3_round(np.nan)) and O.e4m3_round(np.inf) == 448


@pytest.mark.parametrize("top", [448.0, 127.0])
def test_scale_exponent_is_the_least(top):
    for a in [top, np.nextafter(top, 1e9), 1.0, 2.0 ** -130, 3e38, 0.4375]:
        e = O.scale_exponent(a, top)
        assert a <= top * 2.0 ** e and (e == -126 or a > top * 2.0 ** (e - 1))
    assert O.scale_exponent(0.0, top) == -126


def test_page_tables_oracle_on_a_worked_example():
    table = np.array([[5, -1, -1], [2, 7, -1]], np.int32)
    ring = np.array([9, -1, -1, 4, 8, 6], np.int32)
    got = O.page_tables(table, [3, 20], [17, 2], ring, [3, 4, 0, 0], 16, 16)
    assert got[0].tolist() == [[5, 4, -1], [2, 7, -1]] and got[2].tolist() == [4, 4, 0, 0]
    assert got[1].tolist() == [9, 7, -1, 4, 8, 6] and got[3].tolist() == [17, 2] and got[4].tolist() == [0, 14, 14]
    assert got[5].tolist() == [5 * 16 + t for t in range(3, 16)] + [4 * 16, -1, -1]
    assert got[6].tolist() == list(range(3, 17)) + [-1, -1]


def test_selection_oracle_bounds_the_logits():
    rng = np.random.default_rng(1)
    page, d, pages = 16, 64, 12
    codes = O.e4m3_round(rng.normal(size=(pages, 1, page, d)) * 60)
    bounds = np.stack([np.ceil(codes.max(2) / 4), np.floor(codes.min(2) / 4)], 2)
    scale = np.exp2(rng.integers(-8, -4, (pages, 1)).astype(float))
    q = np.round(rng.normal(size=(1, 2, d)) * 32) / 32
    sel, sc = O.select(q, bounds, scale, np.arange(pages)[None], [(0, pages * page - 1, pages * page)], page, 4, 1, 1)
    unit = 2.0 ** O.scale_exponent(np.abs(q).max(), 127.0)
    for p in range(pages):
        top = max((codes[p, 0] * scale[p, 0] @ q[0, a]).max() for a in range(2))
        assert sc[0, 0][p] >= top - d * unit / 2 * 448 * scale[p, 0]      # the rounding of q
    assert sel[0, 0, 0] == 0 and sel[0, 0, -1] == pages - 1 and (np.diff(sel[0, 0]) > 0).all()


def test_append_oracle_bounds_hold_the_codes_when_any_scale_grows():
    rng = np.random.default_rng(5)
    page, d = 16, 64
    for ratio in np.concatenate([rng.uniform(0.02, 1, 40), np.exp2(-np.arange(12.0)), [0.95, 0.6093]]):
        codes = O.e4m3_round(rng.normal(size=(1, 1, page, d)) * 120)
        codes[0, 0, 3, 0], codes[0, 0, 4, 1] = 288, -288
        codes[0, 0, :, 2], codes[0, 0, :, 3] = 288, 224
        bounds = np.stack([np.ceil(codes.max(2) / 4), np.floor(codes.min(2) / 4)], 2)
        x = np.zeros((1, 1, d))
        x[0, 0, -1] = 448                                 # the new scale is 1, the one before `ratio`
        got, scale, b = O.append(codes, np.full((1, 1), ratio), bounds, x, [page - 1], page)
        old = got[0, 0, :page - 1]
        assert scale[0, 0] == 1 and np.array_equal(old, O.e4m3_round(codes[0, 0, :page - 1] * ratio))
        assert (4 * b[0, 0, 0] >= got[0, 0].max(0)).all() and (4 * b[0, 0, 1] <= got[0, 0].min(0)).all(), ratio


def test_attention_oracle_against_torch():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=8), rng.normal(size=(20, 8)), rng.normal(size=(20, 8))
    out, lse, *_ = O.attention(q, k, v, 0.3, 4, 15)
    s = torch.from_numpy(k[4:15] @ q * 0.3)
    assert np.allclose(out, torch.softmax(s, 0).numpy() @ v[4:15]) and np.isclose(lse, float(torch.logsumexp(s, 0)))
    assert O.attention(q, k, v, 0.3, 4, 4)[1] == -np.inf
    assert np.allclose(O.attention(q, k, v, 0.3, 0, 0, keys=range(4, 15))[0], out)


# ---- the binding's refusals ----------------------------------------------------------------------
def cpu_cache(n=4, hkv=2, page=16, d=64):
    """A cache object on the CPU, for the checks that come before the device's."""
    c = kv8.Kv8Cache.__new__(kv8.Kv8Cache)
    c._t = (torch.zeros(n, hkv, page, d, dtype=torch.uint8).view(E4M3),) * 2 + (torch.zeros(n, hkv),) * 2 + (torch.zeros(n, hkv, 2, d, dtype=torch.int8),)
    kv8._init()
    c._c = kv8.attn_kv8_cache_t(*[t.data_ptr() for t in c._t], n, page, hkv, d)
    c._ref = ctypes.byref(c._c)
    c.num_pages, c.page_size, c.hkv, c.head_dim, c.device, c.index = n, page, hkv, d, torch.device("cpu"), -1
    return c


def cpu_plan(hq=4, hkv=2, d=64, page=16):
    p = kv8.Kv8Plan(None, hq, hkv, d, page, -1)
    p.handle = ctypes.c_void_p(1)
    p.__class__ = type("P", (kv8.Kv8Plan,), {"__del__": lambda self: None})
    return p


def codes(*shape):
    return torch.zeros(*shape, dtype=torch.uint8).view(E4M3)


def test_cache_checks():
    good = [codes(4, 2, 16, 64), codes(4, 2, 16, 64), torch.zeros(4, 2), torch.zeros(4, 2), torch.zeros(4, 2, 2, 64, dtype=torch.int8)]
    with pytest.raises(ValueError, match="CUDA"):
        M.Kv8Cache.wrap(*good)
    for i, bad, err in [(0, torch.zeros(4, 2, 16, 64), TypeError), (0, codes(4, 2, 17, 64), ValueError), (0, codes(4, 2, 16, 96), ValueError),
                        (0, codes(4, 16, 64), ValueError), (1, codes(4, 2, 16, 128), ValueError), (2, torch.zeros(4, 3), ValueError),
                        (2, torch.zeros(4, 2).double(), TypeError), (3, torch.zeros(2, 4).t(), ValueError),
                        (4, torch.zeros(4, 2, 2, 64), TypeError), (4, torch.zeros(4, 2, 1, 64, dtype=torch.int8), ValueError), (0, None, TypeError)]:
        args = list(good)
        args[i] = bad
        with pytest.raises(err):
            M.Kv8Cache.wrap(*args)


def test_append_checks():
    c = cpu_cache()
    k, s = torch.zeros(5, 2, 64, dtype=bf16), torch.zeros(5, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        M.attn_kv8_append(c, k, k, s)
    wide = torch.zeros(5, 2, 128, dtype=bf16)
    for args, err in [((k.float(), k, s), TypeError), ((k, k[:4], s), ValueError), ((k, k, s[:4]), ValueError), ((k, k, s.long()), TypeError),
                      ((wide, k, s), ValueError), ((wide[:, :, :64], k, s), ValueError), ((k.transpose(0, 1), k, s), ValueError),
                      ((torch.zeros(5, 2 * 64 + 4, dtype=bf16)[:, :128].view(5, 2, 64), k, s), ValueError), ((k, None, s), TypeError)]:
        with pytest.raises(err):
            M.attn_kv8_append(c, *args)


def test_fwd_and_select_checks():
    c, p = cpu_cache(), cpu_plan()
    q, table, lens, out, lse = (torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 5, dtype=i32), torch.zeros(3, dtype=i32),
                                torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 4))
    with pytest.raises(ValueError, match="CUDA"):
        M.attn_kv8_fwd(p, c, q, table, lens, out, lse)
    cu = torch.zeros(4, dtype=i32)
    for kw, err in [(dict(q=q.float()), TypeError), (dict(q=q[:, :3]), ValueError), (dict(q=torch.zeros(2, 4, 64, dtype=bf16)), ValueError),
                    (dict(page_table=table[:2]), ValueError), (dict(page_table=table.t()), ValueError), (dict(kv_lens=lens.long()), TypeError),
                    (dict(out=out[:2]), ValueError), (dict(out=out.float()), TypeError), (dict(lse=lse.double()), TypeError),
                    (dict(lse=lse[:, :2]), ValueError), (dict(cu_seqlens_q=cu[:3]), ValueError),
                    (dict(selected=torch.zeros(3, 4, 2, dtype=i32)), ValueError), (dict(selected=torch.zeros(3, 2, 0, dtype=i32)), ValueError)]:
        a = dict(q=q, page_table=table, kv_lens=lens, out=out, lse=lse)
        a.update(kw)
        with pytest.raises(err):
            M.attn_kv8_fwd(p, c, **a)
    with pytest.raises(ValueError, match="another"):
        M.attn_kv8_fwd(cpu_plan(page=32), c, q, table, lens, out)
    sc, sel = torch.zeros(3, 2, 5), torch.zeros(3, 2, 4, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        M.attn_kv8_select(p, c, q, table, lens, sc, sel)
    for a, b, err in [(sc[:, :, :4], sel, ValueError), (sc.double(), sel, TypeError), (sc, sel[:, :1], ValueError), (sc, sel.long(), TypeError)]:
        with pytest.raises(err):
            M.attn_kv8_select(p, c, q, table, lens, a, b)
    c._t = c._t[:4] + (None,)
    with pytest.raises(ValueError, match="k_bounds"):
        M.attn_kv8_select(p, c, q, table, lens, sc, sel)
    p.handle = None
    with pytest.raises(ValueError, match="destroyed"):
        M.attn_kv8_fwd(p, c, q, table, lens, out)


def test_forward_kv8_allocates_on_its_stream(monkeypatch):
    # the results of a call on another stream come from that stream's pool
    inside, on, sizes = [], [], []

    class Context:
        def __enter__(self):
            inside.append(True)

        def __exit__(self, *_):
            inside.pop()
    empty = torch.empty
    monkeypatch.setattr(kv8, "_allocating_on", lambda stream, like: on.append((stream, like)) or Context())
    monkeypatch.setattr(torch, "empty", lambda *a, **k: sizes.append(bool(inside)) or empty(*a, **k))
    monkeypatch.setattr(kv8, "attn_kv8_fwd", lambda *a, **k: on.append(k["stream"]))
    q = torch.zeros(3, 4, 64, dtype=bf16)
    kv8._init()
    out, lse = M.forward_kv8(cpu_plan(), cpu_cache(), q, None, None, stream=1234)
    assert on == [(1234, q), 1234] and sizes == [True, True] and out.shape == q.shape and lse.shape == (3, 4)


def test_gather_and_tables_checks():
    c = cpu_cache()
    k, table, cu = torch.zeros(9, 2, 64, dtype=bf16), torch.zeros(2, 5, dtype=i32), torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        M.attn_kv8_gather(c, table, cu, k, k.clone())
    for args, err in [((table[:1], cu, k, k), ValueError), ((table, cu.long(), k, k), TypeError), ((table, cu, k.float(), k), TypeError),
                      ((table, cu, k, k[:8]), ValueError), ((table, cu, k[:, :1], k), ValueError), ((table, cu[:0], k, k), ValueError)]:
        with pytest.raises(err):
            M.attn_kv8_gather(c, *args)
    z = lambda *s: torch.zeros(*s, dtype=i32)  # noqa: E731
    good = dict(page_table=z(3, 4), old_lens=z(3), new_lens=z(3), free_pages=z(8), free_state=z(4), page_size=16, next_state=z(4), kv_lens=z(3),
                cu_seqlens_q=z(4), slots=z(6), positions=z(6))
    with pytest.raises(ValueError, match="CUDA"):
        M.attn_page_tables(**good)
    for name, bad, err in [("page_table", z(2, 4), ValueError), ("new_lens", z(4), ValueError), ("free_state", z(2), ValueError),
                           ("next_state", z(5), ValueError), ("kv_lens", z(2), ValueError), ("cu_seqlens_q", z(3), ValueError),
                           ("positions", z(5), ValueError), ("slots", z(2, 3), Exception), ("old_lens", z(3).long(), TypeError),
                           ("free_pages", z(8).float(), TypeError)]:
        with pytest.raises(err):
            M.attn_page_tables(**dict(good, **{name: bad}))


def test_integers_past_32_bits_are_refused():
    # their low 32 bits would be taken: a window of 2^32 + 5 for one of 5
    good = dict(hq=4, hkv=2, head_dim=64, page_size=16, mask=masks.causal(), max_q_len=1)
    for name in ("hq", "hkv", "head_dim", "page_size", "max_q_len"):
        with pytest.raises(ValueError, match=name):
            M.attn_kv8_plan(**dict(good, **{name: (1 << 32) + good[name]}))
    with pytest.raises(ValueError, match="window"):
        M.attn_kv8_plan(**dict(good, mask=masks.sliding_window((1 << 32) + 5)))
    c, p = cpu_cache(), cpu_plan()
    q, table, lens = torch.zeros(3, 4, 64, dtype=bf16), torch.zeros(3, 5, dtype=i32), torch.zeros(3, dtype=i32)
    sc, sel = torch.zeros(3, 2, 5), torch.zeros(3, 2, 4, dtype=i32)
    for kw in (dict(sink=1 << 32), dict(recent=(1 << 32) + 1)):
        with pytest.raises(ValueError, match="32 bits"):
            M.attn_kv8_select(p, c, q, table, lens, sc, sel, **kw)
    z = lambda *s: torch.zeros(*s, dtype=i32)  # noqa: E731
    with pytest.raises(ValueError, match="page_size"):
        M.attn_page_tables(page_table=z(3, 4), old_lens=z(3), new_lens=z(3), free_pages=z(8), free_state=z(4), page_size=(1 << 32) + 16,
                           next_state=z(4), kv_lens=z(3), cu_seqlens_q=z(4), slots=z(6))


# ---- the C ABI's refusals (no GPU: every one comes before a CUDA call) ------------------------------
INVALID, UNSUPPORTED = 1, 2


def c_cache(**kw):
    a = dict(k=4096, v=4096, k_scale=4096, v_scale=4096, k_bounds=4096, num_pages=4, page_size=16, hkv=2, head_dim=64)
    a.update(kw)
    return kv8.attn_kv8_cache_t(**a)


def test_c_append_and_gather_refusals(attn_lib):
    L = attn_lib.lib()
    app = lambda c, k=4096, ks=128, v=4096, vs=128, s=4096, n=3: L.attn_kv8_append(ctypes.byref(c), k, ks, v, vs, s, n, None)  # noqa: E731
    assert L.attn_kv8_append(None, 4096, 128, 4096, 128, 4096, 3, None) == INVALID
    for c, st in [(c_cache(k=None), INVALID), (c_cache(v_scale=None), INVALID), (c_cache(k=4104), INVALID), (c_cache(k_bounds=4097), INVALID),
                  (c_cache(num_pages=0), INVALID), (c_cache(num_pages=1 << 28), INVALID), (c_cache(hkv=0), INVALID),
                  (c_cache(page_size=24), UNSUPPORTED), (c_cache(head_dim=96), UNSUPPORTED)]:
        assert app(c) == st
        assert L.attn_kv8_gather(ctypes.byref(c), 4096, 2, 4096, 1, 5, 4096, 4096, None) == st
    c = c_cache()
    assert app(c, n=0) == 0 and app(c, n=-1) == INVALID
    assert app(c, k=None) == INVALID and app(c, k=4098) == INVALID and app(c, ks=120) == INVALID and app(c, vs=132) == INVALID
    assert app(c, s=None) == INVALID and app(c, s=4097) == INVALID
    g = lambda *a: L.attn_kv8_gather(ctypes.byref(c), *a, None)  # noqa: E731
    assert g(4096, 0, 4096, 1, 5, 4096, 4096) == INVALID and g(None, 2, 4096, 1, 5, 4096, 4096) == INVALID
    assert g(4096, 2, 4096, 1, 1 << 31, 4096, 4096) == INVALID and g(4096, 2, 4096, 1, 5, 4100, 4096) == INVALID
    assert g(None, 2, None, 0, 0, None, None) == 0


def test_c_refuses_outputs_that_overlap(attn_lib):
    # 4 pages x 2 heads x 16 x 64: 8192 bytes of codes, 32 of scales; 5 rows x 2 x 64 bf16: 1280 bytes
    L = attn_lib.lib()
    app = lambda **kw: L.attn_kv8_append(ctypes.byref(c_cache(**kw)), 1 << 20, 128, 1 << 21, 128, 1 << 22, 3, None)  # noqa: E731
    apart = dict(k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000)
    for kw in (dict(v=0x10000), dict(v=0x10000 + 8192 - 16), dict(v=0x10000 - 8192 + 16), dict(v_scale=0x30000), dict(v_scale=0x30000 + 28)):
        assert app(**{**apart, **kw}) == INVALID, kw
    c = c_cache(**apart)
    for k, v in ((0x50000, 0x50000), (0x50000, 0x50000 + 1280 - 16), (0x50000, 0x50000 - 1280 + 16)):
        assert L.attn_kv8_gather(ctypes.byref(c), 0x60000, 2, 0x70000, 1, 5, k, v, None) == INVALID


def test_c_plan_refusals(attn_lib):
    L = attn_lib.lib()
    h = ctypes.c_void_p()

    def plan(**kw):
        a = dict(hq=4, hkv=2, head_dim=64, page_size=16, scale=0.0, mask=1, window=0, max_q_len=1)
        a.update(kw)
        return L.attn_kv8_plan(ctypes.byref(kv8.attn_kv8_problem_t(**a)), ctypes.byref(h))
    for kw, st in [(dict(hq=5), INVALID), (dict(hkv=0), INVALID), (dict(hq=0), INVALID), (dict(hq=1 << 17, hkv=1), INVALID),
                   (dict(max_q_len=0), INVALID), (dict(scale=float("nan")), INVALID), (dict(mask=2), INVALID), (dict(mask=6), UNSUPPORTED),
                   (dict(mask=3), UNSUPPORTED), (dict(head_dim=80), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED)]:
        assert plan(**kw) == st and not h.value, kw
    assert L.attn_kv8_plan(None, ctypes.byref(h)) == INVALID
    assert L.attn_kv8_plan(ctypes.byref(kv8.attn_kv8_problem_t()), None) == INVALID
    assert L.attn_kv8_plan_destroy(None) == 0
    assert L.attn_kv8_fwd(None, None, None, None, 0, None, None, None) == INVALID
    assert L.attn_kv8_select(None, None, None, 0, 1, None, None, 4, None) == INVALID
    with pytest.raises(M.AttnError):
        M.attn_kv8_plan(hq=4, hkv=2, head_dim=64, page_size=16, mask=masks.prefix_lm(3))


def test_c_tables_refusals(attn_lib):
    L = attn_lib.lib()

    def call(**kw):
        a = dict(batch=2, max_pages_per_seq=3, num_pages=8, page_size=16, max_tokens=4, page_table=0x1000, old_lens=0x2000, new_lens=0x3000,
                 free_pages=0x4000, free_state=0x5000, next_state=0x6000, kv_lens=0x7000, cu_seqlens_q=0x8000, slots=0x9000, positions=0xa000)
        a.update(kw)
        return L.attn_page_tables(ctypes.byref(kv8.attn_page_tables_t(**a)), None)
    assert L.attn_page_tables(None, None) == INVALID
    for kw, st in [(dict(page_size=20), UNSUPPORTED), (dict(batch=16385), UNSUPPORTED), (dict(batch=-1), INVALID), (dict(max_pages_per_seq=0), INVALID),
                   (dict(num_pages=0), INVALID), (dict(max_tokens=-1), INVALID), (dict(num_pages=1 << 28), INVALID),
                   (dict(max_pages_per_seq=1 << 30), INVALID), (dict(page_table=None), INVALID), (dict(slots=None), INVALID),
                   (dict(free_state=None), INVALID), (dict(cu_seqlens_q=None), INVALID), (dict(kv_lens=0x7001), INVALID),
                   (dict(next_state=0x5000), INVALID), (dict(kv_lens=0x2000), INVALID), (dict(kv_lens=0x3004), INVALID),
                   (dict(slots=0xa000 - 8), INVALID), (dict(cu_seqlens_q=0x1010), INVALID), (dict(free_pages=0x1000), INVALID)]:
        assert call(**kw) == st, kw
