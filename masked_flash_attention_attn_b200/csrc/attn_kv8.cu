// The 8-bit paged K/V cache around its attention (attn_kv8_fwd.cu): page tables and slot maps
// from request lengths, quantising append, gather to bf16, and page selection.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "kv8_common.cuh"

namespace kv8 {
namespace {

// ---- page tables and slot maps ------------------------------------------------------------------
// Every CTA scans the request lengths itself (two int32 per request, from L2 after the first
// CTA), keeps the three prefix sums -- new tokens, pages taken, pages given back -- in shared
// memory and then writes its share of the tokens, table entries and ring entries, each found by a
// binary search in the prefixes. So one launch does it all without a grid-wide wait: nothing
// that a CTA reads is written in the call (table entries below the old page count and the ring's
// occupied part are read, entries from the old page count on and the ring's empty part written).
struct Sums { long long tok; int take, give; };

constexpr int kMaxBatch = 16384;  // 3 prefixes of it in shared memory: 192 KiB

__device__ __forceinline__ int pages_of(int n, int shift) { return int((unsigned(n) + (1u << shift) - 1) >> shift); }

__device__ __forceinline__ Sums add(Sums a, Sums b) { return Sums{a.tok + b.tok, a.take + b.take, a.give + b.give}; }
__device__ __forceinline__ Sums up(Sums a, int o) {
  return Sums{__shfl_up_sync(~0u, a.tok, o), __shfl_up_sync(~0u, a.take, o), __shfl_up_sync(~0u, a.give, o)};
}

// the largest i in [0, n) with a[i] <= x (a non-decreasing, a[0] = 0 <= x)
__device__ __forceinline__ int find(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a[m] <= x) lo = m; else hi = m;
  }
  return lo;
}

__global__ void __launch_bounds__(1024) page_tables_kernel(attn_page_tables_t a, int shift) {
  extern __shared__ int s_prefix[];
  wait_for_previous_kernel();
  const int B = a.batch;
  int* s_tok = s_prefix;
  int* s_take = s_tok + B + 1;
  int* s_give = s_take + B + 1;
  __shared__ Sums s_warp[32];
  __shared__ Sums s_total;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
  const int cap = int(min((long long)(a.max_pages_per_seq) << shift, 0x7fffffffLL));
  const int n = a.num_pages;
  int head = a.free_state[0] % n;
  head = head < 0 ? head + n : head;
  const int count = min(max(a.free_state[1], 0), n);

  auto request = [&](int b, int& old_n, int& new_n) -> bool {
    old_n = min(max(a.old_lens[b], 0), cap);
    new_n = a.new_lens[b];
    const bool valid = new_n >= 0 && new_n <= cap;
    if (!valid) new_n = old_n;
    return valid;
  };
  auto sums = [&](int old_n, int new_n) {
    const int d = pages_of(new_n, shift) - pages_of(old_n, shift);
    return Sums{new_n > old_n ? new_n - old_n : 0, max(d, 0), max(-d, 0)};
  };

  const int per = (B + nt - 1) / nt, b0 = min(B, tid * per), b1 = min(B, b0 + per);
  Sums mine{0, 0, 0};
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    int o, w;
    bad |= !request(b, o, w);
    mine = add(mine, sums(o, w));
  }
  Sums inc = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const Sums x = up(inc, o);
    if (lane >= o) inc = add(inc, x);
  }
  if (lane == 31) s_warp[warp] = inc;
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    Sums w = lane < nw ? s_warp[lane] : Sums{0, 0, 0};
    Sums wi = w;
    for (int o = 1; o < 32; o <<= 1) {
      const Sums x = up(wi, o);
      if (lane >= o) wi = add(wi, x);
    }
    if (lane == 31) s_total = wi;
    s_warp[lane] = Sums{wi.tok - w.tok, wi.take - w.take, wi.give - w.give};
  }
  __syncthreads();
  Sums total = s_total;
  const int status = bad ? 2 : total.tok > a.max_tokens ? 3 : total.take > count ? 1 : 0;
  const int missing = status == 1 ? total.take - count : 0;
  const bool ok = status == 0;
  if (!ok) total.tok = 0, total.take = 0;
  Sums at = s_warp[warp];
  at = Sums{at.tok + inc.tok - mine.tok, at.take + inc.take - mine.take, at.give + inc.give - mine.give};
  for (int b = b0; b < b1; ++b) {
    int o, w;
    request(b, o, w);
    s_tok[b] = ok ? int(at.tok) : 0;
    s_take[b] = ok ? at.take : 0;
    s_give[b] = at.give;
    at = add(at, sums(o, w));
  }
  if (tid == 0) {
    s_tok[B] = int(total.tok);
    s_take[B] = total.take;
    s_give[B] = total.give;
  }
  __syncthreads();

  const int g0 = blockIdx.x * nt + tid, gn = gridDim.x * nt;
  auto ring = [&](int i) {        // head + i modulo the ring, 0 <= i <= 2 n
    unsigned x = unsigned(head) + unsigned(i);
    return x % unsigned(n);
  };
  for (int b = g0; b <= B; b += gn) {
    a.cu_seqlens_q[b] = s_tok[b];
    if (b < B) {
      int o, w;
      request(b, o, w);
      a.kv_lens[b] = ok || w < o ? w : o;
    }
  }
  if (g0 == 0) {
    a.next_state[0] = int(ring(total.take));
    a.next_state[1] = count - total.take + total.give;
    a.next_state[2] = status;
    a.next_state[3] = missing;
  }
  for (int t = g0; t < a.max_tokens; t += gn) {
    int slot = -1, pos = -1;
    if (t < int(total.tok)) {
      const int b = find(s_tok, B, t);
      int o, w;
      request(b, o, w);
      pos = o + t - s_tok[b];
      const int pi = pos >> shift, before = pages_of(o, shift);
      const int pg = pi < before ? a.page_table[int64_t(b) * a.max_pages_per_seq + pi]
                                 : a.free_pages[ring(s_take[b] + pi - before)];
      if (unsigned(pg) < unsigned(n)) slot = (pg << shift) + (pos & ((1 << shift) - 1));
    }
    a.slots[t] = slot;
    if (a.positions) a.positions[t] = pos;
  }
  for (int j = g0; j < total.take; j += gn) {
    const int b = find(s_take, B, j);
    int o, w;
    request(b, o, w);
    a.page_table[int64_t(b) * a.max_pages_per_seq + pages_of(o, shift) + j - s_take[b]] = a.free_pages[ring(j)];
  }
  for (int j = g0; j < total.give; j += gn) {
    const int b = find(s_give, B, j);
    int o, w;
    request(b, o, w);
    a.free_pages[ring(count + j % n)] = a.page_table[int64_t(b) * a.max_pages_per_seq + pages_of(w, shift) + j - s_give[b]];
  }
}

// ---- append ---------------------------------------------------------------------------------------
// One CTA takes the runs (tokens of one page that follow one another) that start among its `span` tokens, for
// one head and K or V. A run's new values stay in registers between the maximum and the
// rounding, so they are read once; a page block's codes are contiguous. HBM-bound: 2 bytes in and 1
// out per value. Power-of-two scales lose nothing with a floating 8-bit format (the
// relative step is the same at every exponent) and make requantising after a growth exact
// but for subnormal codes, so a page filled token by token holds what one call would write.
struct AppendArgs {
  const __nv_bfloat16* x[2];
  int64_t stride[2];
  uint8_t* codes[2];
  float* scale[2];
  int8_t* bounds;
  const int32_t* slots;
  int32_t tokens, span, hkv, d, shift, num_slots;   // span: tokens per CTA
};

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {   // two bf16; a NaN loses
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Four bf16 in two words -> their codes in a unit whose reciprocal inv2 (a power of two, in both
// halves) is exact, so one rounding
__device__ __forceinline__ uint32_t codes_of(uint32_t a, uint32_t b, uint32_t inv2) {
  uint32_t x, y;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(a), "r"(inv2));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(b), "r"(inv2));
  return e4m3x4(low(x), high(x), low(y), high(y));
}
// The rare cases, kept out of the kernel's instruction stream: a unit that a caller chose, and values that are not
// finite (the largest finite |x| of the word; NaN becomes 0).
__device__ __noinline__ uint32_t codes_by_division(uint32_t a, uint32_t b, float unit) {
  return e4m3x4(low(a) / unit, high(a) / unit, low(b) / unit, high(b) / unit);
}
__device__ __noinline__ uint32_t without_nan(uint32_t w, unsigned& top) {
  const unsigned lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  if (lo < 0x7f80u) top = max(top, lo);
  if (hi < 0x7f80u) top = max(top, hi);
  return (lo > 0x7f80u ? 0u : w & 0xffffu) | (hi > 0x7f80u ? 0u : w & 0xffff0000u);
}

// Bounds (largest, smallest code of a channel in steps of 4) after the codes became RN(code * ratio). By powers of two codes
// stay exact, or are subnormal and within one step, so scaling and rounding outwards is right. By another
// ratio RN may go past bound * ratio (code 288, bound 72, ratio 0.95: code 288, 4 * 69 = 276): here the
// bound's own code is rounded as theirs were, and RN is monotone. Only for scales that a caller chose: out of line.
__device__ __noinline__ void round_bounds(int8_t* b, int d, float ratio) {
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    const float2 q = float2_of_e4m3(e4m3x4(float(4 * b[c]) * ratio, float(4 * b[d + c]) * ratio, 0.f, 0.f));
    b[c] = int8_t(__float2int_ru(q.x * 0.25f));
    b[d + c] = int8_t(__float2int_rd(q.y * 0.25f));
  }
}

// The nearest token at or behind t (forward) or at or before it that is not skipped, -1 if there is none; by the
// whole CTA, 8 slots a thread and one barrier a round (16 slots: no faster, and the kernel's registers spill). A captured step
// passes all of its slots, the last of them -1, and tokens that are cached already may be left out in front, so
// runs end and start at such stretches. In a graph, 8 heads of d = 128: 32 tokens in 8192 slots 20.9 us, 18.7 of them for the
// empty CTAs (39.4 us by windows of NT slots and four barriers); behind 8192 skipped slots 21.5 (371 by a walk of one thread).
template <int NT, bool FORWARD>
__device__ __noinline__ int nearest_token(const int32_t* slots, int64_t t, int tokens, unsigned num_slots, int* s_found) {
  constexpr int PER = 8;
  for (int64_t at = t; FORWARD ? at < tokens : at >= 0; at += FORWARD ? NT * PER : -NT * PER) {
    const int left = int(min(FORWARD ? tokens - at : at + 1, int64_t(NT * PER)));
    const int32_t* from = slots + at;
    int s[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {             // without branches, so that the loads overlap
      const int w = min(i * NT + int(threadIdx.x), left - 1);
      s[i] = from[FORWARD ? w : -w];
    }
    int dist = INT_MAX;           // from `at`
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) {
      const int w = i * NT + threadIdx.x;
      if (w < left && unsigned(s[i]) < num_slots) dist = w;
    }
    if (!__syncthreads_or(dist < INT_MAX)) continue;
    dist = __reduce_min_sync(~0u, dist);
    if ((threadIdx.x & 31) == 0) s_found[threadIdx.x >> 5] = dist;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) dist = min(dist, s_found[i]);
    return int(FORWARD ? at + dist : at - dist);
  }
  return -1;
}

// Tokens t .. t + n - 1 hold consecutive places and a skipped token or place follows: lists the run's tokens, up
// to the first of another page, and returns their number; 0 if the n are all.
template <int NT>
__device__ __noinline__ int list_run(const int32_t* slots, int tokens, unsigned num_slots, int shift, int t, int n, int2* s_run,
                                     int& s_stop, int* s_taken) {
  const int tid = threadIdx.x, ps = 1 << shift, pg = slots[t] >> shift;
  const int64_t next = nearest_token<NT, true>(slots, int64_t(t) + n, tokens, num_slots, s_taken);
  if (next < 0 || (slots[next] >> shift) != pg) return 0;
  n = 0;
  for (int64_t w0 = t; w0 >= 0; w0 = nearest_token<NT, true>(slots, w0 + NT, tokens, num_slots, s_taken)) {
    __syncthreads();
    if (tid == 0) s_stop = NT;
    __syncthreads();
    const int64_t w = w0 + tid;
    const int s = w < tokens ? slots[w] : 0;
    const bool valid = w < tokens && unsigned(s) < num_slots;
    if (w >= tokens || (valid && (s >> shift) != pg)) atomicMin(&s_stop, tid);
    __syncthreads();
    const int stop = s_stop;
    const bool take = valid && tid < stop;
    const unsigned m = __ballot_sync(~0u, take);
    if ((tid & 31) == 0) s_taken[tid >> 5] = __popc(m);
    __syncthreads();
    int at = n + __popc(m & ((1u << (tid & 31)) - 1u));
    for (int i = 0; i < NT / 32; ++i) {
      if (i < (tid >> 5)) at += s_taken[i];
      n += s_taken[i];
    }
    if (take && at < ps) s_run[at] = make_int2(int(w), s & (ps - 1));
    if (stop < NT || n >= ps) break;
  }
  __syncthreads();
  return min(n, ps);
}

// CTAs per SM: 9 where a page is few vectors (56 registers; 10.8 K tokens of 8 x 128 in pages of 16 take 34.9 us, 37.7
// with 64 registers and 8 CTAs), 8 and 2 for larger pages, whose values fill the registers.
template <int NT, int NV>
__global__ void __launch_bounds__(NT, NT == 256 ? 2 : NV <= 2 ? 9 : 8) append_kernel(AppendArgs a) {
  constexpr int kEnd = -2;        // slot of the tokens before the first and behind the last; -1: a skipped token
  __shared__ int s_slot[260];     // of the tokens t0 - 1 .. t0 + span + page_size - 1
  __shared__ int s_list[128];
  __shared__ int s_count, s_stop, s_taken[NT / 32];
  __shared__ int2 s_run[128];     // token and place of the run's tokens
  __shared__ unsigned s_max[NT / 32];
  __shared__ int s_hi[256], s_lo[256];
  const int tid = threadIdx.x, h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const __nv_bfloat16* src = is_v ? a.x[1] : a.x[0];
  const int64_t stride = is_v ? a.stride[1] : a.stride[0];
  const int t0 = blockIdx.x * a.span, ps = 1 << a.shift, D = a.d, vd = D >> 3;
  const int vshift = 31 - __clz(vd);
  auto valid = [&](int s) { return unsigned(s) < unsigned(a.num_slots); };
  if (tid == 0) s_count = 0;
  wait_for_previous_kernel();
  for (int j = tid; j <= a.span + ps; j += NT) {
    const int t = t0 - 1 + j;
    const int s = t >= 0 && t < a.tokens ? a.slots[t] : kEnd;
    s_slot[j] = valid(s) ? s : t >= 0 && t < a.tokens ? -1 : kEnd;
  }
  __syncthreads();
  const bool live = tid < a.span && valid(s_slot[tid + 1]);
  int outside = s_slot[0];        // of the last token in front of the CTA's, skipped ones aside
  if (outside == -1) {
    if (!__syncthreads_or(live)) return;
    const int t = nearest_token<NT, false>(a.slots, int64_t(t0) - 2, a.tokens, a.num_slots, s_taken);
    if (t >= 0) outside = a.slots[t];
  }
  if (live) {                     // a run starts where the token before is of another page
    int before = s_slot[tid];
    if (before == -1) {
      int j = tid;
      while (j > 0 && s_slot[j] == -1) --j;
      before = j > 0 ? s_slot[j] : outside;
    }
    if (!valid(before) || (before >> a.shift) != (s_slot[tid + 1] >> a.shift)) s_list[atomicAdd(&s_count, 1)] = tid;
  }
  __syncthreads();
  const int runs = s_count;
  for (int r = 0; r < runs; ++r) {
    const int j0 = s_list[r] + 1, t = t0 + j0 - 1, s0 = s_slot[j0], pg = s0 >> a.shift, off = s0 & (ps - 1);
    const bool bound = !is_v && a.bounds != nullptr;
    if (tid == 0) s_stop = ps - off;
    __syncthreads();
    if (tid < ps - off && s_slot[j0 + tid] != s0 + tid) atomicMin(&s_stop, tid);
    __syncthreads();
    int n = s_stop;               // tokens in consecutive places
    bool whole = n == ps - off || s_slot[j0 + n] == kEnd || (valid(s_slot[j0 + n]) && (s_slot[j0 + n] >> a.shift) != pg);
    if (!whole) {
      const int listed = list_run<NT>(a.slots, a.tokens, a.num_slots, a.shift, t, n, s_run, s_stop, s_taken);
      whole = listed == 0;
      n = whole ? n : listed;
    }
    const int vecs = n << vshift;
    if (bound)
      for (int c = tid; c < D; c += NT) s_hi[c] = -128, s_lo[c] = 127;
    const int64_t block = int64_t(pg) * a.hkv + h;
    float* scale = (is_v ? a.scale[1] : a.scale[0]) + block;
    const float old = off > 0 ? *scale : 0.f;
    // vector v is vector v mod vd of the run's token v / vd; NT is a multiple of vd, so a thread keeps its channels
    uint4 x[NV];
    const __nv_bfloat16* from = src + h * D + (tid & (vd - 1)) * 8;
    if (whole) {
      from += int64_t(t + (tid >> vshift)) * stride;
      const int64_t step = (NT >> vshift) * stride;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        x[i] = tid + i * NT < vecs ? __ldg(reinterpret_cast<const uint4*>(from + i * step)) : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * NT;
        x[i] = v < vecs ? __ldg(reinterpret_cast<const uint4*>(from + s_run[v >> vshift].x * stride)) : make_uint4(0, 0, 0, 0);
      }
    }
    unsigned two = 0;             // the largest |x| as bf16 bits, of even and of odd channels
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      two = __vmaxu2(two, __vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu));
      two = __vmaxu2(two, __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
    }
    unsigned top = __reduce_max_sync(~0u, max(two & 0xffffu, two >> 16));
    if ((tid & 31) == 0) s_max[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) top = max(top, s_max[i]);
    bool nan = top > 0x7f80u;
    if (top >= 0x7f80u) {         // infinities or NaN among them: the largest finite |x|
      top = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        x[i].x = without_nan(x[i].x, top), x[i].y = without_nan(x[i].y, top);
        x[i].z = without_nan(x[i].z, top), x[i].w = without_nan(x[i].w, top);
      }
      __syncthreads();
      top = __reduce_max_sync(~0u, top);
      if ((tid & 31) == 0) s_max[tid >> 5] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NT / 32; ++i) top = max(top, s_max[i]);
    }

    // 448 = 1.75 * 2^8: the exponent of top less 8, plus one when its significand is above 1.75
    const int e = max(-126, int(top >> 7) - 127 - 8 + ((top & 127u) > 96u ? 1 : 0));
    nan |= old != old;            // a NaN stays with its page until place 0 is written again
    const float unit = __int_as_float((e + 127) << 23), now = nan ? unit : fmaxf(old, unit);
    const float ratio = nan ? 1.f : old / now;
    uint8_t* codes = (is_v ? a.codes[1] : a.codes[0]) + block * (int64_t(ps) * D);
    float bound_ratio = ratio;
    if (off > 0 && ratio < 1.f) { // the codes before, in the new unit
      if (bound && (__float_as_int(old) & 0x7fffff)) {    // not a power of two (the loop below has the same channels per thread)
        round_bounds(a.bounds + block * (2 * D), D, ratio);
        bound_ratio = 1.f;
      }
      for (int v = tid; v < off * D / 16; v += NT) {
        uint4* p = reinterpret_cast<uint4*>(codes) + v;
        const uint4 c = *p;
        uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 lo = float2_of_e4m3(w[j]), hi = float2_of_e4m3(w[j] >> 16);
          w[j] = e4m3x4(lo.x * ratio, lo.y * ratio, hi.x * ratio, hi.y * ratio);
        }
        *p = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    // a power of two has an exact reciprocal (2^-120 .. 2^126); a scale that a caller wrote may be another
    const bool pow2 = (__float_as_int(now) & 0x7fffff) == 0;
    const uint32_t inv = __float_as_uint(1.f / now) >> 16, inv2 = inv | (inv << 16);
    auto convert = [&](uint32_t p, uint32_t q) { return pow2 ? codes_of(p, q, inv2) : codes_by_division(p, q, now); };
    if (pow2 && whole) {          // the usual case: one page's codes in a row
      uint2* to = reinterpret_cast<uint2*>(codes + off * D) + tid;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (tid + i * NT < vecs) to[i * NT] = make_uint2(codes_of(x[i].x, x[i].y, inv2), codes_of(x[i].z, x[i].w, inv2));
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * NT;
        if (v < vecs) {
          const int at = whole ? off * D + v * 8 : s_run[v >> vshift].y * D + (v & (vd - 1)) * 8;
          *reinterpret_cast<uint2*>(codes + at) = make_uint2(convert(x[i].x, x[i].y), convert(x[i].z, x[i].w));
        }
      }
    }
    // extremes of the thread's eight channels
    uint32_t hi2[4], lo2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) hi2[j] = 0xff80ff80u, lo2[j] = 0x7f807f80u;
    if (bound) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (tid + i * NT < vecs) {
          const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) hi2[j] = max2(hi2[j], w[j]), lo2[j] = min2(lo2[j], w[j]);
        }
      }
    }
    if (bound) {
      for (int o = vd; o < 32; o <<= 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          hi2[j] = max2(hi2[j], __shfl_xor_sync(~0u, hi2[j], o));
          lo2[j] = min2(lo2[j], __shfl_xor_sync(~0u, lo2[j], o));
        }
      }
      if ((tid & 31) < vd && (tid & ~31) < vecs) {   // rounding is monotone: the extreme's code is the extreme code
        const int c = (tid & (vd - 1)) * 8;
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const uint32_t h4 = convert(hi2[j], hi2[j + 1]), l4 = convert(lo2[j], lo2[j + 1]);
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const float2 hq = float2_of_e4m3(h4 >> (8 * k)), lq = float2_of_e4m3(l4 >> (8 * k));
            atomicMax(&s_hi[c + 2 * j + k], __float2int_ru(hq.x * 0.25f));
            atomicMax(&s_hi[c + 2 * j + k + 1], __float2int_ru(hq.y * 0.25f));
            atomicMin(&s_lo[c + 2 * j + k], __float2int_rd(lq.x * 0.25f));
            atomicMin(&s_lo[c + 2 * j + k + 1], __float2int_rd(lq.y * 0.25f));
          }
        }
      }
      __syncthreads();
      int8_t* b = a.bounds + block * (2 * D);
      for (int c = tid; c < D; c += NT) {
        int hi = s_hi[c], lo = s_lo[c];
        if (off > 0) {
          hi = max(hi, __float2int_ru(float(b[c]) * bound_ratio));
          lo = min(lo, __float2int_rd(float(b[D + c]) * bound_ratio));
        }
        b[c] = int8_t(hi);
        b[D + c] = int8_t(lo);
      }
    }
    __syncthreads();              // every thread has read the old scale
    if (tid == 0) *scale = nan ? __int_as_float(0x7fffffff) : now;
  }
}

// ---- gather -----------------------------------------------------------------------------------------
// HBM-bound: 1 byte in and 2 out per value. A CTA takes 8 rows (16: a second wave that is nearly empty at
// the sizes of a prompt chunk; 30.3 against 26.5 us for 22 K rows of 8 x 128, floor 20.8); their
// pages are looked up once.
constexpr int kGatherRows = 8;

struct GatherArgs {
  const uint8_t* codes[2];
  const float* scale[2];
  __nv_bfloat16* out[2];
  const int32_t* page_table;
  const int32_t* cu_k;
  int64_t total_k;
  int32_t batch, max_pages, num_pages, hkv, d, shift;
};

__global__ void __launch_bounds__(256) gather_kernel(GatherArgs a) {
  __shared__ int s_page[kGatherRows], s_off[kGatherRows];
  const int tid = threadIdx.x;
  const int64_t row0 = int64_t(blockIdx.x) * kGatherRows;
  wait_for_previous_kernel();
  if (tid < kGatherRows) {
    const int64_t row = row0 + tid;
    int pg = -2, off = 0;         // -2: no row, -1: a page outside the cache
    if (row < a.total_k) {
      int x = 0, y = a.batch;     // the largest b with cu[b] <= row
      while (y - x > 1) {
        const int m = (x + y) >> 1;
        if (a.cu_k[m] <= row) x = m; else y = m;
      }
      const int64_t j = row - a.cu_k[x];
      const int64_t pi = j >> a.shift;
      if (j >= 0 && row < a.cu_k[x + 1]) {      // tokens past the table's row are zeros, as those of pages outside the cache
        pg = pi < a.max_pages ? a.page_table[int64_t(x) * a.max_pages + pi] : -1;
        if (unsigned(pg) >= unsigned(a.num_pages)) pg = -1;
        off = int(j) & ((1 << a.shift) - 1);
      }
    }
    s_page[tid] = pg;
    s_off[tid] = off;
  }
  __syncthreads();
  // Heads outermost: a warp reads 256 contiguous bytes of a block (2 rows of 128 channels) and writes 512.
  // (16 bytes in and 32 out a lane, in two half-sector stores, measured 27.4 us against 26.5.)
  const int vs = 31 - __clz(a.d >> 3), vd = 1 << vs;
#pragma unroll 4
  for (int i = tid; i < (kGatherRows * a.hkv) << vs; i += 256) {
    const int v = i & (vd - 1), r = (i >> vs) & (kGatherRows - 1), h = (i >> vs) / kGatherRows;
    const int pg = s_page[r];
    if (pg == -2) continue;
    const int64_t block = int64_t(max(pg, 0)) * a.hkv + h;
    uint2 w[2];
    float sc[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      w[z] = pg >= 0 ? __ldg(reinterpret_cast<const uint2*>(a.codes[z] + ((block << a.shift) + s_off[r]) * a.d) + v) : make_uint2(0, 0);
      sc[z] = pg >= 0 ? __ldg(a.scale[z] + block) : 0.f;
    }
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const uint32_t in[2] = {w[z].x, w[z].y};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = float2_of_e4m3(in[j >> 1] >> (16 * (j & 1)));
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * sc[z], f.y * sc[z]);
        o[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *(reinterpret_cast<uint4*>(a.out[z] + ((row0 + r) * a.hkv + h) * a.d) + v) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ---- page selection -----------------------------------------------------------------------------------
// Scores. sum_c (qi > 0 ? qi hi_c : qi lo_c) is the dot product of [max(qi, 0), min(qi, 0)] with
// [hi, lo]: an int8 matrix product of 2 d bound bytes per page with the query heads, on mma.sync
// m16n8k32 (16 pages, 8 heads). The order of channels is free, so lane (g, t) loads bytes 64 i + 16 t of
// pages g and g + 8, its operands. HBM-bound: 2 d bytes per page and KV head. (4-way int8 dot
// products took five times the instructions.)
constexpr int kScorePages = 128;  // pages per CTA
constexpr int kMaxGroup = 64;

struct SelectArgs {
  Batch b;
  const __nv_bfloat16* q;
  int64_t q_stride;
  const int8_t* bounds;
  const float* k_scale;
  int32_t num_pages, hkv, group;
  int32_t sink, recent, k;
  float* scores;
  int32_t* selected;
};

// D += A B, A 16x32 (rows g, g + 8; bytes 4t .. 4t + 3 | 16 more), B 32x8, s8 with s32 accumulators
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The queries of a token and head h in int8: s_q [heads in eights][2 D], s_unit as many units (-inf: no head)
template <int D>
struct Queries {
  static constexpr int PITCH = 2 * D / 16 + 4;   // vectors; neighbouring heads half a line apart: no bank conflicts
  uint4* s_q;
  float* s_unit;
  int eights;
  __device__ __forceinline__ Queries(const SelectArgs& a, uint4* smem) {
    eights = (a.group + 7) >> 3;
    s_q = smem;
    s_unit = reinterpret_cast<float*>(smem + eights * 8 * PITCH);
  }
  __device__ __forceinline__ void quantise(const SelectArgs& a, int tok, int h, int warps) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    for (int r = threadIdx.x >> 5; r < 8 * eights; r += warps) {
      int8_t* dst = reinterpret_cast<int8_t*>(s_q + r * PITCH) + lane * E;
      const bool live = r < a.group;
      const __nv_bfloat16* q = a.q + int64_t(tok) * a.q_stride + int64_t(h * a.group + (live ? r : 0)) * D + lane * E;
      float f[E];
      unsigned top = 0;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        f[j] = live ? __bfloat162float(q[j]) : 0.f;
        const unsigned m = (__float_as_uint(f[j]) >> 16) & 0x7fffu;
        if (m < 0x7f80u) top = max(top, m);
      }
      top = __reduce_max_sync(~0u, top);
      // 127 = 1.984375 * 2^6: significand 126 / 128 over 1
      const int e = max(-126, int(top >> 7) - 127 - 6 + ((top & 127u) > 126u ? 1 : 0));
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int qi = min(127, max(-127, __float2int_rn(f[j] * __int_as_float((127 - e) << 23))));   // NaN converts to 0
        dst[j] = int8_t(max(qi, 0));
        dst[D + j] = int8_t(min(qi, 0));
      }
      if (lane == 0) s_unit[r] = live ? __int_as_float((e + 127) << 23) : -INFINITY;
    }
  }
};

// Bounds of the pages pg[0], pg[1] that lane (g, t) has (g = 0 .. 7: sixteen pages a warp), and their scores
template <int D>
struct PagePair {
  static constexpr int VEC = D / 32;             // 16-byte vectors per lane and page
  uint4 w[2][VEC];
  float ks[2];
  __device__ __forceinline__ void load(const SelectArgs& a, int h, const int* pg, int t) {
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const bool in = unsigned(pg[z]) < unsigned(a.num_pages);
      const int64_t block = in ? int64_t(pg[z]) * a.hkv + h : 0;
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        w[z][i] = in ? __ldg(reinterpret_cast<const uint4*>(a.bounds + block * (2 * D)) + 4 * i + t) : make_uint4(0, 0, 0, 0);
      ks[z] = in ? __ldg(a.k_scale + block) : 0.f;
    }
  }
  __device__ __forceinline__ void score(const SelectArgs& a, const Queries<D>& q, const int* pg, int g, int t, float (&s)[2]) const {
    float best[2] = {-INFINITY, -INFINITY};
    for (int e = 0; e < q.eights; ++e) {
      int dot[4] = {0, 0, 0, 0};  // pages g, g, g + 8, g + 8 and heads 2t, 2t + 1, 2t, 2t + 1
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const uint4 c = q.s_q[(8 * e + g) * Queries<D>::PITCH + 4 * i + t];
        mma_s8(dot, w[0][i].x, w[1][i].x, w[0][i].y, w[1][i].y, c.x, c.y);
        mma_s8(dot, w[0][i].z, w[1][i].z, w[0][i].w, w[1][i].w, c.z, c.w);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float unit = q.s_unit[8 * e + 2 * t + j];
#pragma unroll
        for (int z = 0; z < 2; ++z)
          best[z] = fmaxf(best[z], unit > 0.f ? float(dot[2 * z + j]) * unit : -INFINITY);
      }
    }
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      best[z] = fmaxf(best[z], __shfl_xor_sync(~0u, best[z], 1));
      best[z] = fmaxf(best[z], __shfl_xor_sync(~0u, best[z], 2));
      // finite, so that the pages that are always selected stay above it; a page that holds a NaN
      // comes first of the others, so that the NaN shows
      float x = best[z] * (4.f * ks[z]);
      x = x != x ? 3.402823466e38f : fminf(fmaxf(x, -3.402823466e38f), 3.402823466e38f);
      s[z] = unsigned(pg[z]) < unsigned(a.num_pages) ? x + 0.f : -INFINITY;
    }
  }
};

template <int D>
__global__ void __launch_bounds__(128) page_score_kernel(SelectArgs a) {
  extern __shared__ uint4 s_q[];
  constexpr int ROUNDS = kScorePages / 64;
  Queries<D> queries(a, s_q);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int tok = blockIdx.x / a.hkv, h = blockIdx.x - tok * a.hkv;
  const int p0 = blockIdx.y * kScorePages;
  wait_for_previous_kernel();
  int b, pos, len;
  if (!a.b.token_by_warp(tok, b, pos, len)) return;
  const int n = (a.b.hi(pos, len) + (1 << a.b.page_shift) - 1) >> a.b.page_shift;
  if (p0 >= n) return;
  // the lane's pages are p0 + 64 r + 16 warp + g and 8 more; looked up before the queries are quantised
  const int first = p0 + 16 * warp + g;
  int pages[2 * ROUNDS];
#pragma unroll
  for (int r = 0; r < 2 * ROUNDS; ++r) {
    const int p = first + 64 * (r >> 1) + 8 * (r & 1);
    pages[r] = p < n ? __ldg(a.b.page_table + int64_t(b) * a.b.max_pages + p) : -1;
  }
  queries.quantise(a, tok, h, 4);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    PagePair<D> x;
    x.load(a, h, pages + 2 * r, t);
    float s[2];
    x.score(a, queries, pages + 2 * r, g, t, s);
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int p = first + 64 * r + 8 * z;
      if (t == 0 && p < n) a.scores[(int64_t(tok) * a.hkv + h) * a.b.max_pages + p] = s[z];
    }
  }
}

// The k largest of n scores with ties to the lower page: the k-th largest key by four 8-bit
// radix passes at most (a pass ends the search when the k-th largest is the last of its bin), then the
// pages above it and the first of those equal to it, in ascending order.
// One CTA per token and KV head. A thread keeps its KEYS keys (0: reads them again in every pass,
// for rows of any length). Bound by the latency of its passes; 512 threads, or adding up the lanes
// that meet in a bin first, measured 0.5 us slower.
constexpr int kSelectThreads = 256;
// Scores and selection are one launch, by one CTA a row, where that CTA's part is short or there are rows for
// all SMs; else the scores are spread over more CTAs. Measured (8 rows to a token, d = 128; one launch, two):
//   tokens x pages   1 x 64: 3.8 us, 5.6   1 x 512: 6.8, 7.0   1 x 1000: 10.0, 7.8   8 x 1000: 10.2, 9.4
//                    16 x 1000: 10.8, 12.2   32 x 1000: 18.5, 21.7   1024 x 128: 92, 112
constexpr int kFuse = 512;                // pages of a table row that one launch takes with any number of rows,
constexpr int kFuseRows = 96;             // rows from which on it takes 4 kSelectThreads

// the CTA's share: the pages of one token and head into `out`; load(p) is the key of page p
template <int KEYS, class Load>
__device__ __forceinline__ void pick_pages(int n, int k, int32_t* out, int (&s_hist)[4][256], Load load) {
  constexpr int W = kSelectThreads / 32;
  __shared__ int s_eq[2][W], s_gt[2][W];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t keys[KEYS ? KEYS : 1];
  if constexpr (KEYS > 0) {
#pragma unroll
    for (int i = 0; i < KEYS; ++i) keys[i] = tid + i * kSelectThreads < n ? load(tid + i * kSelectThreads) : 0u;
  }
  auto each = [&](auto f) {       // f(round, page, key) for every round, by all threads
    if constexpr (KEYS > 0) {
#pragma unroll
      for (int i = 0; i < KEYS; ++i) f(i, tid + i * kSelectThreads, keys[i]);
    } else {
      for (int i = 0; i * kSelectThreads < n; ++i) {
        const int p = tid + i * kSelectThreads;
        f(i, p, p < n ? load(p) : 0u);
      }
    }
  };
  uint32_t prefix = 0, fixed = 0;
  int rem = k;                    // how many of the keys that match the prefix are taken
  __syncthreads();
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    int* hist = s_hist[pass];
    each([&](int, int p, uint32_t u) {
      const bool in = p < n && (u & fixed) == prefix;
      if (in) atomicAdd(&hist[(u >> shift) & 255u], 1);
    });
    __syncthreads();
    // every warp looks for the digit of the k-th largest: lane l holds bins 255 - 8 l down to 248 - 8 l
    int c[8], sum = 0, digit = 0, over = 0, count = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += c[j] = hist[255 - 8 * lane - j];
    int inc = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += x;
    }
    int above = inc - sum;
    const bool mine = above < rem && inc >= rem;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (above < rem && above + c[j] >= rem) digit = 255 - 8 * lane - j, over = above, count = c[j];
      above += c[j];
    }
    const int who = __ffs(__ballot_sync(~0u, mine)) - 1;
    digit = __shfl_sync(~0u, digit, who);
    rem -= __shfl_sync(~0u, over, who);
    prefix |= uint32_t(digit) << shift;
    fixed |= 255u << shift;
    if (__shfl_sync(~0u, count, who) == rem) break;   // every key that matches is taken
  }
  int eq0 = 0, gt0 = 0;           // counts before the current 256 pages
  each([&](int i, int p, uint32_t u) {
    if (i * kSelectThreads >= n) return;
    const bool gt = p < n && (u & fixed) > prefix, eq = p < n && (u & fixed) == prefix;
    const unsigned mg = __ballot_sync(~0u, gt), me = __ballot_sync(~0u, eq);
    if (lane == 0) s_gt[i & 1][warp] = __popc(mg), s_eq[i & 1][warp] = __popc(me);
    __syncthreads();
    int g = gt0, e = eq0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int x = s_gt[i & 1][w], y = s_eq[i & 1][w];
      if (w < warp) g += x, e += y;
      gt0 += x, eq0 += y;
    }
    const unsigned below = (1u << lane) - 1u;
    g += __popc(mg & below);
    e += __popc(me & below);
    if (gt || (eq && e < rem)) out[g + min(e, rem)] = p;
  });
}

// larger scores have larger keys; the pages that are always selected have the largest
__device__ __forceinline__ uint32_t key_of(const SelectArgs& a, int n, int p, float score) {
  if (p < a.sink || p >= n - a.recent) return 0xffffffffu;
  const uint32_t u = __float_as_uint(score);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// all of n <= k pages, and the rest of the list; true if that was all
__device__ __forceinline__ bool few_pages(const SelectArgs& a, int n, int32_t* out) {
  for (int i = threadIdx.x; i < a.k; i += kSelectThreads)
    if (i >= n || n <= a.k) out[i] = i < n ? i : -1;
  return n <= a.k;
}

template <int KEYS>
__global__ void __launch_bounds__(kSelectThreads) page_select_kernel(SelectArgs a) {
  __shared__ int s_hist[4][256];
  for (int i = threadIdx.x; i < 4 * 256; i += kSelectThreads) s_hist[0][i] = 0;
  wait_for_previous_kernel();
  const int tok = blockIdx.x / a.hkv, h = blockIdx.x - tok * a.hkv;
  int b, pos, len;
  if (!a.b.token_by_warp(tok, b, pos, len)) return;
  const int n = (a.b.hi(pos, len) + (1 << a.b.page_shift) - 1) >> a.b.page_shift;
  const float* scores = a.scores + (int64_t(tok) * a.hkv + h) * a.b.max_pages;
  int32_t* out = a.selected + (int64_t(tok) * a.hkv + h) * a.k;
  if (few_pages(a, n, out)) return;
  pick_pages<KEYS>(n, a.k, out, s_hist, [&](int p) { return key_of(a, n, p, scores[p]); });
}

// Both steps in one launch, for rows of at most 256 KEYS pages
template <int D, int KEYS>
__global__ void __launch_bounds__(kSelectThreads, D == 256 ? 2 : 4) page_score_select_kernel(SelectArgs a) {
  constexpr int W = kSelectThreads / 32;
  extern __shared__ uint4 s_q[];
  __shared__ int s_hist[4][256];
  __shared__ float s_score[KEYS * kSelectThreads];
  Queries<D> queries(a, s_q);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  for (int i = tid; i < 4 * 256; i += kSelectThreads) s_hist[0][i] = 0;
  const int tok = blockIdx.x / a.hkv, h = blockIdx.x - tok * a.hkv;
  wait_for_previous_kernel();
  int b, pos, len;
  if (!a.b.token_by_warp(tok, b, pos, len)) return;
  const int n = (a.b.hi(pos, len) + (1 << a.b.page_shift) - 1) >> a.b.page_shift;
  const int32_t* table = a.b.page_table + int64_t(b) * a.b.max_pages;
  float* scores = a.scores + (int64_t(tok) * a.hkv + h) * a.b.max_pages;
  int32_t* out = a.selected + (int64_t(tok) * a.hkv + h) * a.k;
  auto look_up = [&](int p) { return p < n ? __ldg(table + p) : -1; };
  // the lane's pages of a round: p and p + 8. The next round's are looked up while this one's bounds come
  int p = 16 * warp + g, next[2] = {look_up(p), look_up(p + 8)};
  queries.quantise(a, tok, h, W);
  __syncthreads();
  for (; p - g < n; p += 16 * W) {
    const int now[2] = {next[0], next[1]};
    PagePair<D> x;
    x.load(a, h, now, t);
    next[0] = look_up(p + 16 * W), next[1] = look_up(p + 16 * W + 8);
    float s[2];
    x.score(a, queries, now, g, t, s);
#pragma unroll
    for (int z = 0; z < 2; ++z)
      if (t == 0 && p + 8 * z < n) scores[p + 8 * z] = s_score[p + 8 * z] = s[z];
  }
  if (few_pages(a, n, out)) return;
  __syncthreads();
  pick_pages<KEYS>(n, a.k, out, s_hist, [&](int p) { return key_of(a, n, p, s_score[p]); });
}

}  // namespace
}  // namespace kv8

using namespace kv8;

extern "C" {

attn_status_t attn_page_tables(const attn_page_tables_t* t, attn_stream_t stream) {
  if (!t) return ATTN_ERR_INVALID_ARG;
  const int shift = shift_of(t->page_size);
  if (shift < 0 || t->batch > kMaxBatch) return ATTN_ERR_UNSUPPORTED;
  if (t->batch < 0 || t->max_pages_per_seq < 1 || t->num_pages < 1 || t->max_tokens < 0) return ATTN_ERR_INVALID_ARG;
  if (int64_t(t->batch) * t->max_pages_per_seq >= (int64_t(1) << 31) ||
      int64_t(t->num_pages) * t->page_size >= (int64_t(1) << 31))
    return ATTN_ERR_INVALID_ARG;
  if (!t->free_pages || !t->free_state || !t->next_state || !t->cu_seqlens_q) return ATTN_ERR_INVALID_ARG;
  if (t->batch && (!t->page_table || !t->old_lens || !t->new_lens || !t->kv_lens)) return ATTN_ERR_INVALID_ARG;
  if (t->max_tokens && !t->slots) return ATTN_ERR_INVALID_ARG;
  // every array of its own, but that old_lens and new_lens (only read) may be one
  const struct { const void* p; int64_t n; } all[] = {
      {t->old_lens, t->batch}, {t->new_lens, t->batch}, {t->free_state, 4}, {t->next_state, 4}, {t->kv_lens, t->batch},
      {t->cu_seqlens_q, int64_t(t->batch) + 1}, {t->slots, t->max_tokens}, {t->positions, t->max_tokens},
      {t->free_pages, t->num_pages}, {t->page_table, int64_t(t->batch) * t->max_pages_per_seq}};
  for (int i = 0; i < 10; ++i) {
    if (misaligned(all[i].p, 4)) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (!(i == 1 && j == 0) && overlap(all[i].p, 4 * all[i].n, all[j].p, 4 * all[j].n)) return ATTN_ERR_INVALID_ARG;
  }
  const int work = std::max(t->batch + 1, t->max_tokens);
  const int threads = work <= 256 ? 256 : 1024;
  const int grid = std::min(148, (work + threads - 1) / threads);
  const size_t smem = size_t(3) * (t->batch + 1) * sizeof(int);
  // The 48 KiB that need no opt-in hold the kernel's static arrays too. Always the same maximum, that of the
  // largest batch, so that a call never takes back what another thread's launch needs.
  if (smem > 32 * 1024 && cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               int(3 * (kMaxBatch + 1) * sizeof(int))) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_CUDA;
  }
  return launch(page_tables_kernel, dim3(grid), threads, smem, stream, *t, shift);
}

attn_status_t attn_kv8_append(const attn_kv8_cache_t* c, const void* k_new, int64_t k_stride, const void* v_new,
                              int64_t v_stride, const int32_t* slots, int32_t num_tokens, attn_stream_t stream) {
  const attn_status_t st = check_cache(c);
  if (st != ATTN_OK) return st;
  if (num_tokens < 0) return ATTN_ERR_INVALID_ARG;
  if (num_tokens == 0) return ATTN_OK;
  const int64_t row = int64_t(c->hkv) * c->head_dim;
  if (!k_new || !v_new || !slots || misaligned(k_new, 16) || misaligned(v_new, 16) || misaligned(slots, 4))
    return ATTN_ERR_INVALID_ARG;
  if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8) return ATTN_ERR_INVALID_ARG;
  const int64_t blocks = int64_t(c->num_pages) * c->hkv, codes = blocks * c->page_size * c->head_dim;
  if (overlap(c->k, codes, c->v, codes) || overlap(c->k_scale, blocks * 4, c->v_scale, blocks * 4)) return ATTN_ERR_INVALID_ARG;
  AppendArgs a{};
  a.x[0] = static_cast<const __nv_bfloat16*>(k_new);
  a.x[1] = static_cast<const __nv_bfloat16*>(v_new);
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.codes[0] = static_cast<uint8_t*>(c->k);
  a.codes[1] = static_cast<uint8_t*>(c->v);
  a.scale[0] = c->k_scale;
  a.scale[1] = c->v_scale;
  a.bounds = c->k_bounds;
  a.slots = slots;
  a.tokens = num_tokens;
  a.hkv = c->hkv;
  a.d = c->head_dim;
  a.shift = shift_of(c->page_size);
  a.num_slots = c->num_pages * c->page_size;
  // tokens per CTA: enough that the grid is about one wave of 148 x 16 CTAs, at most half a page (a CTA then has
  // one run or none: 17.5 us for 10.8 K tokens of 8 x 128 against 18.3 with whole pages, floor 10.2)
  int span = 1;
  while (2 * span < c->page_size && int64_t(num_tokens) * c->hkv * 2 >= int64_t(2 * span) * 148 * 16) span *= 2;
  a.span = span;
  const dim3 grid((num_tokens + span - 1) / span, c->hkv, 2);
  switch (c->page_size * c->head_dim / 8) {         // 16-byte vectors of a full page
    case 128: return launch(append_kernel<128, 1>, grid, 128, 0, stream, a);
    case 256: return launch(append_kernel<128, 2>, grid, 128, 0, stream, a);
    case 512: return launch(append_kernel<128, 4>, grid, 128, 0, stream, a);
    case 1024: return launch(append_kernel<128, 8>, grid, 128, 0, stream, a);
    case 2048: return launch(append_kernel<256, 8>, grid, 256, 0, stream, a);
    default: return launch(append_kernel<256, 16>, grid, 256, 0, stream, a);
  }
}

attn_status_t attn_kv8_gather(const attn_kv8_cache_t* c, const int32_t* page_table, int32_t max_pages_per_seq,
                              const int32_t* cu_seqlens_k, int32_t batch, int64_t total_k, void* k_out, void* v_out,
                              attn_stream_t stream) {
  const attn_status_t st = check_cache(c);
  if (st != ATTN_OK) return st;
  if (batch < 0 || total_k < 0 || max_pages_per_seq < 1) return ATTN_ERR_INVALID_ARG;
  if (batch == 0 || total_k == 0) return ATTN_OK;
  if (!page_table || !cu_seqlens_k || !k_out || !v_out || total_k >= (int64_t(1) << 31)) return ATTN_ERR_INVALID_ARG;
  if (misaligned(k_out, 16) || misaligned(v_out, 16) || misaligned(page_table, 4) || misaligned(cu_seqlens_k, 4))
    return ATTN_ERR_INVALID_ARG;
  const int64_t bytes = total_k * c->hkv * c->head_dim * 2;
  if (overlap(k_out, bytes, v_out, bytes)) return ATTN_ERR_INVALID_ARG;
  GatherArgs a{};
  a.codes[0] = static_cast<const uint8_t*>(c->k);
  a.codes[1] = static_cast<const uint8_t*>(c->v);
  a.scale[0] = c->k_scale;
  a.scale[1] = c->v_scale;
  a.out[0] = static_cast<__nv_bfloat16*>(k_out);
  a.out[1] = static_cast<__nv_bfloat16*>(v_out);
  a.page_table = page_table;
  a.cu_k = cu_seqlens_k;
  a.total_k = total_k;
  a.batch = batch;
  a.max_pages = max_pages_per_seq;
  a.num_pages = c->num_pages;
  a.hkv = c->hkv;
  a.d = c->head_dim;
  a.shift = shift_of(c->page_size);
  const unsigned grid = unsigned((total_k + kGatherRows - 1) / kGatherRows);
  return launch(gather_kernel, dim3(grid), 256, 0, stream, a);
}

attn_status_t attn_kv8_select(const attn_kv8_plan_t* p, const attn_kv8_cache_t* c, const attn_kv8_batch_t* b,
                              int32_t sink, int32_t recent, float* scores, int32_t* selected, int32_t n_selected,
                              attn_stream_t stream) {
  const attn_status_t st = check_batch(p, c, b);
  if (st != ATTN_OK) return st;
  if (p->mask == ATTN_MASK_SLIDING_WINDOW || p->hq / p->hkv > kMaxGroup) return ATTN_ERR_UNSUPPORTED;
  if (sink < 0 || recent < 1 || int64_t(sink) + recent > n_selected) return ATTN_ERR_INVALID_ARG;
  if (b->total_q == 0 || b->batch == 0) return ATTN_OK;
  if (!c->k_bounds || !scores || !selected || misaligned(scores, 4) || misaligned(selected, 4)) return ATTN_ERR_INVALID_ARG;
  const int64_t rows = int64_t(b->total_q) * p->hkv;
  const int64_t chunks = (int64_t(b->max_pages_per_seq) + kScorePages - 1) / kScorePages;
  if (rows >= (int64_t(1) << 31) || chunks > 65535) return ATTN_ERR_INVALID_ARG;
  if (overlap(scores, rows * b->max_pages_per_seq * 4, selected, rows * n_selected * 4)) return ATTN_ERR_INVALID_ARG;
  SelectArgs a{};
  a.b = batch_of(p, b);
  a.q = static_cast<const __nv_bfloat16*>(b->q);
  a.q_stride = b->q_stride;
  a.bounds = c->k_bounds;
  a.k_scale = c->k_scale;
  a.num_pages = c->num_pages;
  a.hkv = p->hkv;
  a.group = p->hq / p->hkv;
  a.sink = sink;
  a.recent = recent;
  a.k = n_selected;
  a.scores = scores;
  a.selected = selected;
  const dim3 grid{unsigned(rows), unsigned(chunks)}, each{unsigned(rows)};
  const size_t smem = size_t((a.group + 7) / 8 * 8) * (2 * p->d + 64 + 4);
  const int pages = b->max_pages_per_seq;
  if (pages <= kFuse || (pages <= 4 * kSelectThreads && rows >= kFuseRows)) {
    return p->d == 64    ? launch(page_score_select_kernel<64, 4>, each, kSelectThreads, smem, stream, a)
           : p->d == 128 ? launch(page_score_select_kernel<128, 4>, each, kSelectThreads, smem, stream, a)
                         : launch(page_score_select_kernel<256, 4>, each, kSelectThreads, smem, stream, a);
  }
  const attn_status_t scored = p->d == 64    ? launch(page_score_kernel<64>, grid, 128, smem, stream, a)
                               : p->d == 128 ? launch(page_score_kernel<128>, grid, 128, smem, stream, a)
                                             : launch(page_score_kernel<256>, grid, 128, smem, stream, a);
  if (scored != ATTN_OK) return scored;
  if (pages <= 4 * kSelectThreads) return launch(page_select_kernel<4>, each, kSelectThreads, 0, stream, a);
  if (pages <= 16 * kSelectThreads) return launch(page_select_kernel<16>, each, kSelectThreads, 0, stream, a);
  return launch(page_select_kernel<0>, each, kSelectThreads, 0, stream, a);
}

}  // extern "C"
