// Shared by the kernels of the 8-bit paged K/V cache (attn_kv8.cu, attn_kv8_fwd.cu): the
// query batch as the kernels see it, e4m3 conversions, and host-side argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_kv8.h"

struct attn_kv8_plan {
  int32_t hq = 0, hkv = 0, d = 0, page_size = 0, page_shift = 0;
  float scale = 0.f;
  int32_t mask = 0, window = 0;
  int32_t ng = 1;                 // row tile of the attention kernel: 8 ng rows
  int32_t grid[2] = {0, 0};       // persistent CTAs: of few and of many items
  int32_t device = 0;
  void* ws = nullptr;             // partial results and counters
  float* part_o = nullptr;        // [2 CTAs][8 ng][d]
  float* part_ml = nullptr;       // [2 CTAs][8 ng][2]
  uint32_t* counters = nullptr;   // [CTAs], zero between launches
};

namespace kv8 {

// The query tokens of a call and how they see the keys.
struct Batch {
  const int32_t* page_table;
  const int32_t* kv_lens;
  const int32_t* cu_q;            // null: one token per request
  int32_t batch, total_q, max_pages, page_shift;
  int32_t mask, window;
  __device__ __forceinline__ int len(int b) const {
    const long long cap = (long long)max_pages << page_shift;
    const int l = kv_lens[b];
    return l < 0 ? 0 : (l > cap ? int(cap) : l);
  }
  __device__ __forceinline__ int cu(int b) const {
    const int c = cu_q[b];
    return c < 0 ? 0 : (c > total_q ? total_q : c);
  }
  // keys [lo, hi) that the token at position pos of a request of `n` tokens sees
  __device__ __forceinline__ int hi(int pos, int n) const {
    if (mask == ATTN_MASK_FULL) return n;
    return pos < 0 ? 0 : (pos + 1 < n ? pos + 1 : n);
  }
  __device__ __forceinline__ int lo(int pos) const {
    return mask == ATTN_MASK_SLIDING_WINDOW && pos >= window ? pos - window + 1 : 0;
  }
  // request of token t: true and its position and length, or false behind the last request
  __device__ __forceinline__ bool token(int t, int& b, int& pos, int& n) const {
    int i = 0, nq = 1;
    if (cu_q == nullptr) {
      b = t;
    } else {
      b = t < batch ? t : batch - 1;        // one token each is common
      int c0 = cu(b), c1 = cu(b + 1);
      if (c0 > t || c1 <= t) {
        int x = 0, y = batch;     // the largest b with cu[b] <= t
        while (y - x > 1) {
          const int m = (x + y) >> 1;
          if (cu(m) <= t) x = m; else y = m;
        }
        b = x;
        c0 = cu(b), c1 = cu(b + 1);
      }
      i = t - c0;
      nq = c1 - c0;
      if (i < 0 || i >= nq) return false;
    }
    n = len(b);
    pos = n - nq + i;
    return true;
  }
  // the same by a whole warp, all lanes with one t: a 32-ary search, one round of loads per factor of 32
  __device__ __forceinline__ bool token_by_warp(int t, int& b, int& pos, int& n) const {
    if (cu_q == nullptr) return token(t, b, pos, n);
    const int lane = threadIdx.x & 31;
    int x = 0, width = batch;       // the request is one of x .. x + width - 1
    while (width > 1) {
      const int step = (width + 31) >> 5, at = x + lane * step;
      const unsigned m = __ballot_sync(~0u, at < x + width && cu(at) <= t);
      const int k = m ? 31 - __clz(m) : 0;
      width = min(step, width - k * step);
      x += k * step;
    }
    b = x;
    const int first = cu(b), nq = cu(b + 1) - first, i = t - first;
    if (i < 0 || i >= nq) return false;
    n = len(b);
    pos = n - nq + i;
    return true;
  }
};

// Kernels of this cache follow one another in a serving step, each a few microseconds long. They are
// launched with programmatic stream serialization: a kernel's CTAs may become resident once the
// CTAs of the kernel before have ended, and this holds them until its writes are visible: select
// and attend of 4 x 2-8 K tokens 29.9 -> 22.7 us. Letting the next kernel in earlier
// (griddepcontrol.launch_dependents) measured 30.2: its CTAs take the room of ones that still run.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// two e4m3 codes (low byte first) -> two halves; exact
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(two)));
  return r;
}

__device__ __forceinline__ float2 float2_of_e4m3(uint32_t two) {
  const uint32_t h = half2_of_e4m3(two);
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(h));
  return f;
}

// Four fp32 -> four e4m3, `a` in the lowest byte: round to nearest even, saturating at +-448.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return uint32_t(lo) | (uint32_t(hi) << 16);
}

// ---- host checks ------------------------------------------------------------------------------
inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return x && y && na > 0 && nb > 0 && x < y + nb && y < x + na;
}
inline int shift_of(int32_t page_size) {
  return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : page_size == 128 ? 7 : -1;
}

inline attn_status_t check_cache(const attn_kv8_cache_t* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return ATTN_ERR_INVALID_ARG;
  if (shift_of(c->page_size) < 0) return ATTN_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return ATTN_ERR_UNSUPPORTED;
  if (c->num_pages < 1 || c->hkv < 1 || c->hkv > 65535) return ATTN_ERR_INVALID_ARG;
  if (int64_t(c->num_pages) * c->page_size >= (int64_t(1) << 31)) return ATTN_ERR_INVALID_ARG;
  if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_scale, 4) || misaligned(c->v_scale, 4) ||
      misaligned(c->k_bounds, 16))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

inline attn_status_t check_batch(const attn_kv8_plan_t* p, const attn_kv8_cache_t* c, const attn_kv8_batch_t* b) {
  if (!p || !b) return ATTN_ERR_INVALID_ARG;
  const attn_status_t st = check_cache(c);
  if (st != ATTN_OK) return st;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  if (dev != p->device) return ATTN_ERR_INVALID_ARG;
  if (c->hkv != p->hkv || c->head_dim != p->d || c->page_size != p->page_size) return ATTN_ERR_INVALID_ARG;
  if (b->batch < 0 || b->total_q < 0 || b->max_pages_per_seq < 1) return ATTN_ERR_INVALID_ARG;
  if (int64_t(b->total_q) * p->hq >= (int64_t(1) << 31)) return ATTN_ERR_INVALID_ARG;
  if (int64_t(b->max_pages_per_seq) * p->page_size >= (int64_t(1) << 31)) return ATTN_ERR_INVALID_ARG;
  if (!b->cu_seqlens_q && b->total_q != b->batch) return ATTN_ERR_INVALID_ARG;
  if (b->total_q == 0 || b->batch == 0) return ATTN_OK;
  if (!b->q || !b->page_table || !b->kv_lens) return ATTN_ERR_INVALID_ARG;
  if (b->q_stride < int64_t(p->hq) * p->d || b->q_stride % 8) return ATTN_ERR_INVALID_ARG;
  if (misaligned(b->q, 16) || misaligned(b->cu_seqlens_q, 4) || misaligned(b->page_table, 4) || misaligned(b->kv_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

template <class... Params, class... Args>
inline attn_status_t launch(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, attn_stream_t stream, Args... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = reinterpret_cast<cudaStream_t>(stream);
  c.attrs = &at;
  c.numAttrs = 1;
  if (cudaLaunchKernelEx(&c, kernel, args...) == cudaSuccess) return ATTN_OK;
  cudaGetLastError();             // the status says it; the caller's next check is not to find it again
  return ATTN_ERR_CUDA;
}

inline Batch batch_of(const attn_kv8_plan_t* p, const attn_kv8_batch_t* b) {
  return Batch{b->page_table, b->kv_lens, b->cu_seqlens_q, b->batch, b->total_q, b->max_pages_per_seq, p->page_shift,
               p->mask, p->window};
}

}  // namespace kv8
