"""The 8-bit paged K/V cache: binding of ``include/attn_kv8.h``.

A serving step over a cache of e4m3 codes with one scale per page and KV head::

    cache = attn.Kv8Cache(num_pages, page_size=16, hkv=8, head_dim=128)
    plan = attn.attn_kv8_plan(hq=32, hkv=8, head_dim=128, page_size=16, mask=masks.causal())

    attn.attn_page_tables(page_table=table, old_lens=lens, new_lens=wanted, free_pages=ring,
                          free_state=state, page_size=16, next_state=next_state, kv_lens=kv_lens,
                          cu_seqlens_q=cu_q, slots=slots, positions=positions)
    attn.attn_kv8_append(cache, k, v, slots)                      # per layer: k, v [T, hkv, d]
    attn.attn_kv8_fwd(plan, cache, q, table, kv_lens, out, lse, cu_seqlens_q=cu_q)

    # long contexts: 64 pages per token and KV head instead of all of them
    attn.attn_kv8_select(plan, cache, q, table, kv_lens, scores, selected, cu_seqlens_q=cu_q)
    attn.attn_kv8_fwd(plan, cache, q, table, kv_lens, out, lse, cu_seqlens_q=cu_q, selected=selected)

    # long query chunks: the cached tokens as bf16, then any masked forward
    attn.attn_kv8_gather(cache, table, cu_k, k, v)
    attn.attn_masked_fwd(masked_plan, q, k, v, out, lse)

Lengths, offsets and tables are device tensors; no call allocates device memory (but for
attn_kv8_plan and the constructors) or waits for the GPU, so a step can be captured into a CUDA graph.
As everywhere in this package the C side sees bare pointers, so every tensor is checked here
first: type, shape, layout, device (all on one CUDA device, which must be the current one).
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import MASK_KIND, _check, _stream, lib

_I32, _F32, _BF16, _E4M3, _I8 = "int32", "float32", "bfloat16", "float8_e4m3fn", "int8"
PAGE_SIZES = (16, 32, 64, 128)


class attn_kv8_cache_t(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_bounds", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("hkv", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class attn_page_tables_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("page_table", ctypes.c_void_p),
                ("old_lens", ctypes.c_void_p), ("new_lens", ctypes.c_void_p), ("free_pages", ctypes.c_void_p),
                ("free_state", ctypes.c_void_p), ("next_state", ctypes.c_void_p), ("kv_lens", ctypes.c_void_p),
                ("cu_seqlens_q", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p)]


class attn_kv8_problem_t(ctypes.Structure):
    _fields_ = [("hq", ctypes.c_int32), ("hkv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("scale", ctypes.c_float), ("mask", ctypes.c_int32),
                ("window", ctypes.c_int32), ("max_q_len", ctypes.c_int32)]


class attn_kv8_batch_t(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("total_q", ctypes.c_int32), ("cu_seqlens_q", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("max_pages_per_seq", ctypes.c_int32), ("kv_lens", ctypes.c_void_p)]


_dtypes = None


def _dtype(name):
    global _dtypes
    if _dtypes is None:
        import torch
        _dtypes = {n: getattr(torch, n) for n in (_I32, _F32, _BF16, _E4M3, _I8)}
    return _dtypes[name]


def _is_tensor(t, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")


def _tensor(t, name, dtype, shape, device):
    """The pointer of a contiguous tensor of exactly this type and shape (None: any size) on
    ``device``."""
    _is_tensor(t, name)
    if t.dtype != _dtype(dtype):
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name} must be {['any' if w is None else w for w in shape]}, not {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the others on {device}")
    return t.data_ptr()


def _rows(t, name, heads, head_dim, device):
    """(pointer, elements from token to token) of bf16 rows [tokens][heads][head_dim]; the rows may lie
    apart (a view of a fused projection), each row is contiguous."""
    _is_tensor(t, name)
    if t.dtype != _dtype(_BF16):
        raise TypeError(f"{name} must be {_BF16}, not {t.dtype}")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != head_dim:
        raise ValueError(f"{name} must be [tokens, {heads}, {head_dim}], not {list(t.shape)}")
    s0, s1, s2 = t.stride()
    row = heads * head_dim
    if t.shape[0] <= 1:
        s0 = row
    if s2 != 1 or (s1 != head_dim and heads > 1) or s0 < row or s0 % 8:
        raise ValueError(f"{name}: each token's [{heads}, {head_dim}] must be contiguous, tokens a multiple of 8 "
                         f"elements apart (strides {list(t.stride())})")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the others on {device}")
    return t.data_ptr(), s0


def _on_current(device, stream):
    """The raw stream of a call whose tensors are on ``device``."""
    import torch
    if device.type != "cuda":
        raise ValueError("the tensors must be CUDA tensors")
    if torch.cuda.current_device() != device.index:
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}")
    dev = getattr(stream, "device", None)
    if dev is not None and dev != device:
        raise ValueError(f"the stream is on {dev}, the tensors on {device}")
    return _stream(stream)


class Kv8Cache:
    """An 8-bit paged cache: k, v (float8_e4m3fn [num_pages, hkv, page_size, head_dim]), k_scale, v_scale
    (float32 [num_pages, hkv]) and k_bounds (int8 [num_pages, hkv, 2, head_dim], or None when
    pages are never selected). The tensors are fixed for the life of the object."""

    __slots__ = ("_t", "_c", "num_pages", "page_size", "hkv", "head_dim", "device")

    def __init__(self, num_pages: int, *, page_size: int, hkv: int, head_dim: int, device="cuda", bounds: bool = True):
        import torch
        e = torch.float8_e4m3fn
        code = (num_pages, hkv, page_size, head_dim)
        self._set(torch.zeros(code, dtype=torch.uint8, device=device).view(e),
                  torch.zeros(code, dtype=torch.uint8, device=device).view(e),
                  torch.zeros(code[:2], device=device), torch.zeros(code[:2], device=device),
                  torch.zeros(num_pages, hkv, 2, head_dim, dtype=torch.int8, device=device) if bounds else None)

    @classmethod
    def wrap(cls, k, v, k_scale, v_scale, k_bounds=None) -> "Kv8Cache":
        """A cache in tensors that exist already."""
        self = cls.__new__(cls)
        self._set(k, v, k_scale, v_scale, k_bounds)
        return self

    def _set(self, k, v, ks, vs, bounds):
        _is_tensor(k, "k")
        if k.dim() != 4:
            raise ValueError("k must be [num_pages, hkv, page_size, head_dim]")
        n, hkv, page, d = k.shape
        if page not in PAGE_SIZES or d not in (64, 128, 256) or n < 1 or hkv < 1:
            raise ValueError(f"page_size must be one of {PAGE_SIZES}, head_dim 64, 128 or 256, num_pages and hkv >= 1")
        if n * page >= 1 << 31:
            raise ValueError("num_pages * page_size must be below 2^31")
        p = [_tensor(k, "k", _E4M3, (n, hkv, page, d), k.device), _tensor(v, "v", _E4M3, (n, hkv, page, d), k.device),
             _tensor(ks, "k_scale", _F32, (n, hkv), k.device), _tensor(vs, "v_scale", _F32, (n, hkv), k.device),
             None if bounds is None else _tensor(bounds, "k_bounds", _I8, (n, hkv, 2, d), k.device)]
        if k.device.type != "cuda":
            raise ValueError("the cache must be on a CUDA device")
        self._t = (k, v, ks, vs, bounds)
        self._c = attn_kv8_cache_t(*p, n, page, hkv, d)
        self.num_pages, self.page_size, self.hkv, self.head_dim, self.device = n, page, hkv, d, k.device

    k = property(lambda self: self._t[0])
    v = property(lambda self: self._t[1])
    k_scale = property(lambda self: self._t[2])
    v_scale = property(lambda self: self._t[3])
    k_bounds = property(lambda self: self._t[4])


class Kv8Plan:
    """Owns an attn_kv8_plan_t. Calls on one plan must be ordered one after another."""

    def __init__(self, handle, hq, hkv, head_dim, page_size, device):
        self.handle, self.hq, self.hkv, self.head_dim, self.page_size, self.device = handle, hq, hkv, head_dim, page_size, device

    def __del__(self):
        if getattr(self, "handle", None):
            try:
                attn_kv8_plan_destroy(self)
            except Exception:
                pass


def attn_page_tables(*, page_table, old_lens, new_lens, free_pages, free_state, page_size: int, next_state, kv_lens,
                     cu_seqlens_q, slots, positions=None, stream=None) -> None:
    """attn_page_tables(): page tables, slots and positions of a step that takes request b from
    old_lens[b] to new_lens[b] tokens. int32 CUDA tensors: page_table [batch, max_pages] and the
    ring free_pages [num_pages] are updated; free_state [4] (head, count), old_lens, new_lens
    [batch] are read; next_state [4] (head, count, status, missing pages), kv_lens [batch], cu_seqlens_q
    [batch + 1], slots and positions [max_tokens] are written."""
    _is_tensor(old_lens, "old_lens")
    if old_lens.dim() != 1:
        raise ValueError("old_lens must be [batch]")
    dev, batch = old_lens.device, old_lens.shape[0]
    _is_tensor(slots, "slots")
    tokens = slots.shape[0] if slots.dim() == 1 else None
    a = attn_page_tables_t()
    a.page_table = _tensor(page_table, "page_table", _I32, (batch, None), dev)
    a.old_lens = _tensor(old_lens, "old_lens", _I32, (batch,), dev)
    a.new_lens = _tensor(new_lens, "new_lens", _I32, (batch,), dev)
    a.free_pages = _tensor(free_pages, "free_pages", _I32, (None,), dev)
    a.free_state = _tensor(free_state, "free_state", _I32, (4,), dev)
    a.next_state = _tensor(next_state, "next_state", _I32, (4,), dev)
    a.kv_lens = _tensor(kv_lens, "kv_lens", _I32, (batch,), dev)
    a.cu_seqlens_q = _tensor(cu_seqlens_q, "cu_seqlens_q", _I32, (batch + 1,), dev)
    a.slots = _tensor(slots, "slots", _I32, (tokens,), dev)
    if positions is not None:
        a.positions = _tensor(positions, "positions", _I32, (tokens,), dev)
    a.batch, a.max_pages_per_seq, a.num_pages = batch, page_table.shape[1], free_pages.shape[0]
    a.page_size, a.max_tokens = int(page_size), tokens
    s = _on_current(dev, stream)
    _check(lib().attn_page_tables(ctypes.byref(a), s), "attn_page_tables")


def attn_kv8_append(cache: Kv8Cache, k, v, slots, stream=None) -> None:
    """attn_kv8_append(): quantise k, v (bf16 [T, hkv, head_dim]; views whose tokens lie apart
    work) into the slots (int32 [T], negative: skip) that attn_page_tables() gave them."""
    dev = cache.device
    kp, ks = _rows(k, "k", cache.hkv, cache.head_dim, dev)
    vp, vs = _rows(v, "v", cache.hkv, cache.head_dim, dev)
    n = k.shape[0]
    if v.shape[0] != n:
        raise ValueError(f"v has {v.shape[0]} tokens, k {n}")
    sp = _tensor(slots, "slots", _I32, (None,), dev)
    if slots.shape[0] < n:
        raise ValueError(f"slots has {slots.shape[0]} entries for {n} tokens")
    s = _on_current(dev, stream)
    _check(lib().attn_kv8_append(ctypes.byref(cache._c), kp, ks, vp, vs, sp, n, s), "attn_kv8_append")


def attn_kv8_gather(cache: Kv8Cache, page_table, cu_seqlens_k, k_out, v_out, stream=None) -> None:
    """attn_kv8_gather(): rows cu_seqlens_k[b] .. cu_seqlens_k[b + 1] of k_out, v_out (bf16 [total_k, hkv,
    head_dim]) become request b's cached keys and values; cu_seqlens_k int32 [batch + 1], page_table
    int32 [batch, max_pages]."""
    dev = cache.device
    cp = _tensor(cu_seqlens_k, "cu_seqlens_k", _I32, (None,), dev)
    batch = cu_seqlens_k.shape[0] - 1
    if batch < 0:
        raise ValueError("cu_seqlens_k must be [batch + 1]")
    tp = _tensor(page_table, "page_table", _I32, (None, None), dev)
    if page_table.shape[0] < batch:
        raise ValueError(f"page_table has {page_table.shape[0]} rows for {batch} requests")
    kp = _tensor(k_out, "k_out", _BF16, (None, cache.hkv, cache.head_dim), dev)
    vp = _tensor(v_out, "v_out", _BF16, (k_out.shape[0], cache.hkv, cache.head_dim), dev)
    s = _on_current(dev, stream)
    _check(lib().attn_kv8_gather(ctypes.byref(cache._c), tp, page_table.shape[1], cp, batch, k_out.shape[0], kp, vp, s),
           "attn_kv8_gather")


def attn_kv8_plan(*, hq: int, hkv: int, head_dim: int, page_size: int, mask, scale: float = 0.0,
                  max_q_len: int = 1) -> Kv8Plan:
    """attn_kv8_plan(): a plan on the current device for attn_kv8_fwd() and attn_kv8_select(). ``mask``:
    masks.causal(), masks.full() or masks.sliding_window(w); ``max_q_len``: query tokens per request that
    are common."""
    import torch
    p = attn_kv8_problem_t(int(hq), int(hkv), int(head_dim), int(page_size), float(scale), MASK_KIND[mask.kind],
                           int(getattr(mask, "window", 0) or 0), int(max_q_len))
    h = ctypes.c_void_p()
    _check(lib().attn_kv8_plan(ctypes.byref(p), ctypes.byref(h)), "attn_kv8_plan")
    return Kv8Plan(h.value, p.hq, p.hkv, p.head_dim, p.page_size, torch.device("cuda", torch.cuda.current_device()))


def attn_kv8_plan_destroy(plan: Kv8Plan) -> None:
    if plan.handle:
        h, plan.handle = plan.handle, None
        _check(lib().attn_kv8_plan_destroy(h), "attn_kv8_plan_destroy")


def _batch(plan, cache, q, page_table, kv_lens, cu_seqlens_q):
    if not plan.handle:
        raise ValueError("the plan was destroyed")
    dev = cache.device
    if (cache.hkv, cache.head_dim, cache.page_size) != (plan.hkv, plan.head_dim, plan.page_size):
        raise ValueError("the cache has another hkv, head_dim or page_size than the plan")
    if dev != plan.device:
        raise ValueError(f"the cache is on {dev}, the plan on {plan.device}")
    qp, stride = _rows(q, "q", plan.hq, plan.head_dim, dev)
    total = q.shape[0]
    lp = _tensor(kv_lens, "kv_lens", _I32, (None,), dev)
    batch = kv_lens.shape[0]
    cp = None
    if cu_seqlens_q is not None:
        cp = _tensor(cu_seqlens_q, "cu_seqlens_q", _I32, (batch + 1,), dev)
    elif total != batch:
        raise ValueError(f"q has {total} tokens for {batch} requests: cu_seqlens_q is required")
    tp = _tensor(page_table, "page_table", _I32, (None, None), dev)
    if page_table.shape[0] < batch:
        raise ValueError(f"page_table has {page_table.shape[0]} rows for {batch} requests")
    return attn_kv8_batch_t(qp, stride, batch, total, cp, tp, page_table.shape[1], lp), total, dev


def attn_kv8_fwd(plan: Kv8Plan, cache: Kv8Cache, q, page_table, kv_lens, out, lse=None, *, cu_seqlens_q=None,
                 selected=None, stream=None) -> None:
    """attn_kv8_fwd(): attention of q (bf16 [T, hq, head_dim], the last tokens of their requests) over
    the cache into out (bf16, like q) and lse (fp32 [T, hq]). page_table int32 [batch,
    max_pages], kv_lens int32 [batch], cu_seqlens_q int32 [batch + 1] (None: one token each). ``selected``:
    int32 [T, hkv, k] page numbers of attn_kv8_select()."""
    b, total, dev = _batch(plan, cache, q, page_table, kv_lens, cu_seqlens_q)
    op = _tensor(out, "out", _BF16, (total, plan.hq, plan.head_dim), dev)
    lp = None if lse is None else _tensor(lse, "lse", _F32, (total, plan.hq), dev)
    sp, n = None, 0
    if selected is not None:
        sp = _tensor(selected, "selected", _I32, (total, plan.hkv, None), dev)
        n = selected.shape[2]
        if n < 1:
            raise ValueError("selected must list at least one page")
        sp = sp or None                            # no tokens
    s = _on_current(dev, stream)
    _check(lib().attn_kv8_fwd(plan.handle, ctypes.byref(cache._c), ctypes.byref(b), sp, n, op, lp, s), "attn_kv8_fwd")


def attn_kv8_select(plan: Kv8Plan, cache: Kv8Cache, q, page_table, kv_lens, scores, selected, *, cu_seqlens_q=None,
                    sink: int = 1, recent: int = 1, stream=None) -> None:
    """attn_kv8_select(): the pages with the highest score bounds for each token of q and KV head into
    selected (int32 [T, hkv, k], ascending, -1 past the last); the first ``sink`` and last
    ``recent`` pages always. scores: fp32 [T, hkv, max_pages] receives the scores."""
    b, total, dev = _batch(plan, cache, q, page_table, kv_lens, cu_seqlens_q)
    if cache.k_bounds is None:
        raise ValueError("the cache holds no k_bounds")
    cp = _tensor(scores, "scores", _F32, (total, plan.hkv, page_table.shape[1]), dev)
    sp = _tensor(selected, "selected", _I32, (total, plan.hkv, None), dev)
    s = _on_current(dev, stream)
    _check(lib().attn_kv8_select(plan.handle, ctypes.byref(cache._c), ctypes.byref(b), int(sink), int(recent), cp, sp,
                                 selected.shape[2], s), "attn_kv8_select")


def forward_kv8(plan: Kv8Plan, cache: Kv8Cache, q, page_table, kv_lens, cu_seqlens_q=None, selected=None, stream=None):
    """Allocate out / lse with torch and run attn_kv8_fwd (convenience)."""
    import torch
    _is_tensor(q, "q")
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    lse = torch.empty(q.shape[0], plan.hq, dtype=torch.float32, device=q.device)
    attn_kv8_fwd(plan, cache, q, page_table, kv_lens, out, lse, cu_seqlens_q=cu_seqlens_q, selected=selected, stream=stream)
    return out, lse
