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
import struct

from . import MASK_KIND, _allocating_on, _check, lib

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


# attn_page_tables_t and attn_kv8_batch_t as a call fills them (a ctypes structure takes three times as long)
_TABLES = struct.Struct("5i10P").pack
_BATCH = struct.Struct("Pq2i2PiP").pack

torch = None                       # imported with the first cache, plan or call, as elsewhere in this package
_I32 = _F32 = _BF16 = _E4M3 = _I8 = _device = _raw_stream = None


def _init():
    global torch, _I32, _F32, _BF16, _E4M3, _I8, _device, _raw_stream
    import torch as t
    # without the initialisation checks of torch.cuda's: they are asked when there is a tensor on a CUDA device
    _device = getattr(t._C, "_cuda_getDevice", None) or t.cuda.current_device
    _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None) or (lambda dev: t.cuda.current_stream(dev).cuda_stream)
    _I32, _F32, _BF16, _E4M3, _I8 = t.int32, t.float32, t.bfloat16, t.float8_e4m3fn, t.int8
    torch = t


def _wrong(t, name, dtype, shape, dev):
    """Raise what _ptr() and _rows() found wrong (they only compare: a decode step's checks count)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if len(t.shape) != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name} must be {['any' if w is None else w for w in shape]}, not {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the others on {'cpu' if dev < 0 else f'cuda:{dev}'}")
    raise ValueError(f"{name} must be contiguous (strides {list(t.stride())})")


def _ptr(t, name, dtype, shape, dev):
    """The pointer of a contiguous tensor of exactly this type and shape on device ``dev`` (-1: the CPU)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _wrong(t, name, dtype, shape, dev)


def _i32s(tensors, names, shapes, dev):
    """_ptr() of several int32 tensors."""
    at = []
    try:
        for t, shape in zip(tensors, shapes):
            if not (t.dtype is _I32 and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
                break
            at.append(t.data_ptr())
        else:
            return at
    except AttributeError:
        pass
    _wrong(tensors[len(at)], names[len(at)], _I32, shapes[len(at)], dev)


def _shape(t, name, dims):
    """The shape of a tensor of ``dims`` dimensions."""
    if isinstance(t, torch.Tensor) and len(t.shape) == dims:
        return t.shape
    _wrong(t, name, getattr(t, "dtype", None), (None,) * dims, -1)


def _rows(t, name, heads, head_dim, dev):
    """(pointer, elements from token to token, tokens) of bf16 rows [tokens][heads][head_dim]; the rows may lie
    apart (a view of a fused projection), each row is contiguous."""
    try:
        n, th, td = t.shape
        right = t.dtype is _BF16 and th == heads and td == head_dim and t.get_device() == dev
    except (AttributeError, ValueError):          # not a tensor, or not of three dimensions
        right = False
    if not right:
        _wrong(t, name, _BF16, (None, heads, head_dim), dev)
    row = heads * head_dim
    if t.is_contiguous():
        return t.data_ptr(), row, n
    s0, s1, s2 = t.stride()
    if n <= 1:
        s0 = row
    if s2 != 1 or (s1 != head_dim and heads > 1) or s0 < row or s0 % 8:
        raise ValueError(f"{name}: each token's [{heads}, {head_dim}] must be contiguous, tokens a multiple of 8 "
                         f"elements apart (strides {list(t.stride())})")
    return t.data_ptr(), s0, n


def _int32(x, name):
    """``x`` as an int of 32 bits (ctypes would drop the bits above)."""
    n = int(x)
    if not -1 << 31 <= n < 1 << 31:
        raise ValueError(f"{name} = {n} does not fit in 32 bits")
    return n


def _on_current(dev, stream):
    """The raw stream of a call whose tensors are on device ``dev``."""
    if dev < 0:
        raise ValueError("the tensors must be CUDA tensors")
    if _device() != dev:
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{_device()}")
    if stream is None:
        return _raw_stream(dev)
    at = getattr(stream, "device", None)
    if at is not None and at.index != dev:
        raise ValueError(f"the stream is on {at}, the tensors on cuda:{dev}")
    return getattr(stream, "cuda_stream", stream)


class Kv8Cache:
    """An 8-bit paged cache: k, v (float8_e4m3fn [num_pages, hkv, page_size, head_dim]), k_scale, v_scale
    (float32 [num_pages, hkv]) and k_bounds (int8 [num_pages, hkv, 2, head_dim], or None when
    pages are never selected). The tensors are fixed for the life of the object."""

    __slots__ = ("_t", "_c", "_ref", "num_pages", "page_size", "hkv", "head_dim", "device", "index")

    def __init__(self, num_pages: int, *, page_size: int, hkv: int, head_dim: int, device="cuda", bounds: bool = True):
        _init()
        code = (num_pages, hkv, page_size, head_dim)
        self._set(torch.zeros(code, dtype=torch.uint8, device=device).view(_E4M3),
                  torch.zeros(code, dtype=torch.uint8, device=device).view(_E4M3),
                  torch.zeros(code[:2], device=device), torch.zeros(code[:2], device=device),
                  torch.zeros(num_pages, hkv, 2, head_dim, dtype=torch.int8, device=device) if bounds else None)

    @classmethod
    def wrap(cls, k, v, k_scale, v_scale, k_bounds=None) -> "Kv8Cache":
        """A cache in tensors that exist already."""
        _init()
        self = cls.__new__(cls)
        self._set(k, v, k_scale, v_scale, k_bounds)
        return self

    def _set(self, k, v, ks, vs, bounds):
        n, hkv, page, d = _shape(k, "k", 4)
        dev = k.get_device()
        if page not in PAGE_SIZES or d not in (64, 128, 256) or n < 1 or hkv < 1:
            raise ValueError(f"page_size must be one of {PAGE_SIZES}, head_dim 64, 128 or 256, num_pages and hkv >= 1")
        if n * page >= 1 << 31:
            raise ValueError("num_pages * page_size must be below 2^31")
        p = [_ptr(k, "k", _E4M3, (n, hkv, page, d), dev), _ptr(v, "v", _E4M3, (n, hkv, page, d), dev),
             _ptr(ks, "k_scale", _F32, (n, hkv), dev), _ptr(vs, "v_scale", _F32, (n, hkv), dev),
             None if bounds is None else _ptr(bounds, "k_bounds", _I8, (n, hkv, 2, d), dev)]
        if dev < 0:
            raise ValueError("the cache must be on a CUDA device")
        self._t = (k, v, ks, vs, bounds)
        self._c = attn_kv8_cache_t(*p, n, page, hkv, d)
        self._ref = ctypes.byref(self._c)
        self.num_pages, self.page_size, self.hkv, self.head_dim, self.device, self.index = n, page, hkv, d, k.device, dev

    k = property(lambda self: self._t[0])
    v = property(lambda self: self._t[1])
    k_scale = property(lambda self: self._t[2])
    v_scale = property(lambda self: self._t[3])
    k_bounds = property(lambda self: self._t[4])


class Kv8Plan:
    """Owns an attn_kv8_plan_t. Calls on one plan must be ordered one after another, and a plan must live as long as a
    captured graph that holds its calls is replayed (its workspace is freed with it)."""

    def __init__(self, handle, hq, hkv, head_dim, page_size, index):
        self.handle, self.hq, self.hkv, self.head_dim, self.page_size, self.index = handle, hq, hkv, head_dim, page_size, index

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
    if torch is None:
        _init()
    try:
        (batch,), (tokens,), (pages,), (_, width) = old_lens.shape, slots.shape, free_pages.shape, page_table.shape
        dev = old_lens.get_device()
    except (AttributeError, ValueError):
        for t, name, dims in ((old_lens, "old_lens", 1), (slots, "slots", 1), (free_pages, "free_pages", 1), (page_table, "page_table", 2)):
            _shape(t, name, dims)
        raise
    lens, four = (batch,), (4,)
    at = _i32s((page_table, old_lens, new_lens, free_pages, free_state, next_state, kv_lens, cu_seqlens_q, slots,
                slots if positions is None else positions),
               ("page_table", "old_lens", "new_lens", "free_pages", "free_state", "next_state", "kv_lens", "cu_seqlens_q", "slots", "positions"),
               ((batch, width), lens, lens, (pages,), four, four, lens, (batch + 1,), (tokens,), (tokens,)), dev)
    if positions is None:
        at[9] = 0
    if page_size not in PAGE_SIZES:
        page_size = _int32(page_size, "page_size")       # the library's to refuse
    a = _TABLES(batch, width, pages, page_size, tokens, *at)
    st = lib().attn_page_tables(a, _on_current(dev, stream))
    if st:
        _check(st, "attn_page_tables")


def attn_kv8_append(cache: Kv8Cache, k, v, slots, stream=None) -> None:
    """attn_kv8_append(): quantise k, v (bf16 [T, hkv, head_dim]; views whose tokens lie apart
    work) into the slots (int32 [T], negative: skip) that attn_page_tables() gave them."""
    dev = cache.index
    kp, ks, n = _rows(k, "k", cache.hkv, cache.head_dim, dev)
    vp, vs, nv = _rows(v, "v", cache.hkv, cache.head_dim, dev)
    if nv != n:
        raise ValueError(f"v has {nv} tokens, k {n}")
    m, = _shape(slots, "slots", 1)
    sp = _ptr(slots, "slots", _I32, (m,), dev)
    if m < n:
        raise ValueError(f"slots has {m} entries for {n} tokens")
    st = lib().attn_kv8_append(cache._ref, kp, ks, vp, vs, sp, n, _on_current(dev, stream))
    if st:
        _check(st, "attn_kv8_append")


def attn_kv8_gather(cache: Kv8Cache, page_table, cu_seqlens_k, k_out, v_out, stream=None) -> None:
    """attn_kv8_gather(): rows cu_seqlens_k[b] .. cu_seqlens_k[b + 1] of k_out, v_out (bf16 [total_k, hkv,
    head_dim]) become request b's cached keys and values; cu_seqlens_k int32 [batch + 1], page_table
    int32 [batch, max_pages]."""
    dev = cache.index
    n, = _shape(cu_seqlens_k, "cu_seqlens_k", 1)
    cp = _ptr(cu_seqlens_k, "cu_seqlens_k", _I32, (n,), dev)
    if n < 1:
        raise ValueError("cu_seqlens_k must be [batch + 1]")
    rows, width = _shape(page_table, "page_table", 2)
    tp = _ptr(page_table, "page_table", _I32, (rows, width), dev)
    if rows < n - 1:
        raise ValueError(f"page_table has {rows} rows for {n - 1} requests")
    total = _shape(k_out, "k_out", 3)[0]
    kp = _ptr(k_out, "k_out", _BF16, (total, cache.hkv, cache.head_dim), dev)
    vp = _ptr(v_out, "v_out", _BF16, (total, cache.hkv, cache.head_dim), dev)
    st = lib().attn_kv8_gather(cache._ref, tp, width, cp, n - 1, total, kp, vp, _on_current(dev, stream))
    if st:
        _check(st, "attn_kv8_gather")


def attn_kv8_plan(*, hq: int, hkv: int, head_dim: int, page_size: int, mask, scale: float = 0.0,
                  max_q_len: int = 1) -> Kv8Plan:
    """attn_kv8_plan(): a plan on the current device for attn_kv8_fwd() and attn_kv8_select(). ``mask``:
    masks.causal(), masks.full() or masks.sliding_window(w); ``max_q_len``: query tokens per request that
    are common."""
    _init()
    p = attn_kv8_problem_t(_int32(hq, "hq"), _int32(hkv, "hkv"), _int32(head_dim, "head_dim"), _int32(page_size, "page_size"),
                           float(scale), MASK_KIND[mask.kind], _int32(getattr(mask, "window", 0) or 0, "window"),
                           _int32(max_q_len, "max_q_len"))
    h = ctypes.c_void_p()
    _check(lib().attn_kv8_plan(ctypes.byref(p), ctypes.byref(h)), "attn_kv8_plan")
    return Kv8Plan(h.value, p.hq, p.hkv, p.head_dim, p.page_size, torch.cuda.current_device())


def attn_kv8_plan_destroy(plan: Kv8Plan) -> None:
    if plan.handle:
        h, plan.handle = plan.handle, None
        _check(lib().attn_kv8_plan_destroy(h), "attn_kv8_plan_destroy")


def _batch(plan, cache, q, page_table, kv_lens, cu_seqlens_q):
    if not plan.handle:
        raise ValueError("the plan was destroyed")
    dev = cache.index
    if cache.page_size != plan.page_size or cache.head_dim != plan.head_dim or cache.hkv != plan.hkv:
        raise ValueError("the cache has another hkv, head_dim or page_size than the plan")
    if dev != plan.index:
        raise ValueError(f"the cache is on {cache.device}, the plan on cuda:{plan.index}")
    qp, stride, total = _rows(q, "q", plan.hq, plan.head_dim, dev)
    try:
        (batch,), (rows, width) = kv_lens.shape, page_table.shape
    except (AttributeError, ValueError):
        _shape(kv_lens, "kv_lens", 1), _shape(page_table, "page_table", 2)
        raise
    if rows < batch:
        raise ValueError(f"page_table has {rows} rows for {batch} requests")
    if cu_seqlens_q is not None:
        tp, lp, cp = _i32s((page_table, kv_lens, cu_seqlens_q), ("page_table", "kv_lens", "cu_seqlens_q"),
                           ((rows, width), (batch,), (batch + 1,)), dev)
    else:
        if total != batch:
            raise ValueError(f"q has {total} tokens for {batch} requests: cu_seqlens_q is required")
        tp, lp = _i32s((page_table, kv_lens), ("page_table", "kv_lens"), ((rows, width), (batch,)), dev)
        cp = 0
    return _BATCH(qp, stride, batch, total, cp, tp, width, lp), total, width, dev


def attn_kv8_fwd(plan: Kv8Plan, cache: Kv8Cache, q, page_table, kv_lens, out, lse=None, *, cu_seqlens_q=None,
                 selected=None, stream=None) -> None:
    """attn_kv8_fwd(): attention of q (bf16 [T, hq, head_dim], the last tokens of their requests) over
    the cache into out (bf16, like q) and lse (fp32 [T, hq]). page_table int32 [batch,
    max_pages], kv_lens int32 [batch], cu_seqlens_q int32 [batch + 1] (None: one token each). ``selected``:
    int32 [T, hkv, k] page numbers of attn_kv8_select()."""
    b, total, _, dev = _batch(plan, cache, q, page_table, kv_lens, cu_seqlens_q)
    op = _ptr(out, "out", _BF16, (total, plan.hq, plan.head_dim), dev)
    lp = None if lse is None else _ptr(lse, "lse", _F32, (total, plan.hq), dev)
    sp, n = None, 0
    if selected is not None:
        n = _shape(selected, "selected", 3)[2]
        if n < 1:
            raise ValueError("selected must list at least one page")
        sp = _ptr(selected, "selected", _I32, (total, plan.hkv, n), dev) or None   # no tokens
    st = lib().attn_kv8_fwd(plan.handle, cache._ref, b, sp, n, op, lp, _on_current(dev, stream))
    if st:
        _check(st, "attn_kv8_fwd")


def attn_kv8_select(plan: Kv8Plan, cache: Kv8Cache, q, page_table, kv_lens, scores, selected, *, cu_seqlens_q=None,
                    sink: int = 1, recent: int = 1, stream=None) -> None:
    """attn_kv8_select(): the pages with the highest score bounds for each token of q and KV head into
    selected (int32 [T, hkv, k], ascending, -1 past the last); the first ``sink`` and last
    ``recent`` pages always. scores: fp32 [T, hkv, max_pages] receives the scores."""
    b, total, width, dev = _batch(plan, cache, q, page_table, kv_lens, cu_seqlens_q)
    if cache._t[4] is None:
        raise ValueError("the cache holds no k_bounds")
    n = _shape(selected, "selected", 3)[2]
    cp = _ptr(scores, "scores", _F32, (total, plan.hkv, width), dev)
    sp = _ptr(selected, "selected", _I32, (total, plan.hkv, n), dev)
    st = lib().attn_kv8_select(plan.handle, cache._ref, b, _int32(sink, "sink"), _int32(recent, "recent"), cp, sp, n,
                               _on_current(dev, stream))
    if st:
        _check(st, "attn_kv8_select")


def forward_kv8(plan: Kv8Plan, cache: Kv8Cache, q, page_table, kv_lens, cu_seqlens_q=None, selected=None, stream=None):
    """Allocate out / lse with torch and run attn_kv8_fwd (convenience). With ``stream`` (a torch stream or a raw
    handle) they are allocated on it, like the results of an operation under torch.cuda.stream(stream)."""
    _shape(q, "q", 3)
    with _allocating_on(stream, q):
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        lse = torch.empty(q.shape[0], plan.hq, dtype=torch.float32, device=q.device)
    attn_kv8_fwd(plan, cache, q, page_table, kv_lens, out, lse, cu_seqlens_q=cu_seqlens_q, selected=selected, stream=stream)
    return out, lse
