// Attention of a few query tokens per request over the 8-bit paged K/V cache.
//
// Mathematics. Per request, KV head h and query row n (a token and a query head of h's group):
//     s_j = scale k_scale[page(j)] (q_n . code_j),  p_j = 2^(s_j log2 e - m_n),
//     out = sum_j p_j v_scale[page(j)] code_j / sum_j p_j,  lse = m_n ln 2 + ln sum_j p_j
// with m_n near the running maximum. e4m3 codes convert to fp16 exactly and q is scaled by a power of
// two per row into fp16 range, so the products are exact (of q values from 2^-31 of the row's largest on); both matrix products run on
// mma.sync m16n8k16 with fp32 accumulators, transposed: S^T = K Q^T and O^T = V^T P^T, keys or
// channels on the 16-row side and 8 query rows on the other, so the eight rows of a grouped
// decode step fill a tile (as the 128-row side of a tcgen05 MMA they would use 6 % of it).
//
// What bounds it: HBM. 2 d bytes per key and KV head are read once; at the measured copy rate
// an SM receives ~23 bytes per clock. Next come the issue slots: ~250 instructions of a warp per 16
// keys of 128 channels (4 KiB), of which 64 convert codes (cvt.f16x2.e4m3x2).
//
// Layout. A step is 16 keys (a page holds a whole number of them): 16 d contiguous bytes of K and
// of V. A warp copies them by cp.async, 512 contiguous bytes per instruction, into its own ring
// of stages (no barrier but __syncwarp). Copying straight into fragment order instead (each
// lane the bytes it needs, 64-byte pieces) measured 5.0 TB/s against 6.8 TB/s for this order. The
// order of channels in the dot product and of output channels over the tile rows is free, so
// every read is of 16 bytes that are one lane's fragments: K: lane (g, t) bytes 64 i + 16 t of keys g
// and g + 8; V: bytes 16 g (+ 128) of keys 2t, 2t+1, 2t+8, 2t+9. 16-byte chunks of a row are swizzled
// so that both reads are free of bank conflicts. P passes from the accumulator layout of S^T to
// the operand layout of P^T by movmatrix.
//
// Work. Every persistent CTA scans the lengths itself. The keys of an item (request, KV head, row
// tile) come in chunks of kWarps steps; within a CTA the warps take alternate steps and merge in
// shared memory. Two ways to share the chunks out:
//   one piece each: an item of c chunks is cut into ceil(c / T) equal pieces, T the least tried at
//     which no more pieces than CTAs are made. Taken when T is within kPiece chunks of the mean.
//   one line: the chunks of all items in a row (the start of an item counts kStart chunks), cut
//     evenly, so that a CTA has the end of one item, whole ones, and the start of another.
// A second piece costs a CTA about 7 chunks (profiled: 32 x 0.5-4 K tokens on a line, CTAs with one
// piece are done at 28 us, with two at 36). Equal pieces handed out by a ticket measured slower at
// any size. An item that several CTAs share is joined by the last of them to arrive (an atomic
// counter that it resets), in the order of the keys: results do not depend on timing, nothing waits.
// (One release-acquire atomic, and the join's first loads ahead of its weights, against two full fences
// and loads behind them: 32 x 0.5-4 K tokens 39.7 -> 37.6 us.)

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <new>

#include "kv8_common.cuh"

namespace kv8 {
namespace {

constexpr int kStep = 16;                 // keys per step
constexpr int kStart = 3;                 // chunks that starting on an item is worth in the line
constexpr int kPiece = 6;                 // chunks over the mean that one piece each may take
constexpr int kTries = 8;                 // lengths of a piece that are tried, 1/16 of the mean apart
constexpr float kNone = -3.402823466e38f;  // reference of a row that has seen no key; finite, so differences are never NaN
// P is 2^(s - m) in fp16, m the row's reference. When P of a step's largest key would leave 2^(+-kRange), m moves to kHead
// below that key, down as well as up: fp16 keeps 11 bits down to 2^-14, so the rounding of a P is at most 2^-11 of the
// largest of its 16 keys, however far those are below the row's maximum. (With the running maximum as reference,
// keys 17 nats below a sink lost a third of their sum.) Downwards until the row's sum is 2^kGrow, far from the
// end of fp32 for the products too: keys up to 65 nats below the maximum.
// (With the maximum as reference / so: 32 x 2-4 K keys at d = 128 with 4 rows 42.3 / 42.4 us, 16 rows 50.9 / 52.7,
// 32 rows 76.8 / 79.3; 16 verifications at d = 256 46.5 / 46.9. Both ends in one compare of |x - m|: two compares 1-2 % more.)
constexpr float kHead = 6.f;
constexpr float kRange = 14.f;
constexpr int kGrow = 80;

struct FwdArgs {
  Batch b;
  const __nv_bfloat16* q;
  int64_t q_stride;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  int32_t num_pages, hkv, group;
  float scale_log2;
  const int32_t* selected;
  int32_t n_selected;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;
  float* part_ml;
  uint32_t* counters;
};

// A CTA of W warps. Merging the warps and starting on the next item cost about as many instructions as
// 27 steps in a CTA of 8 warps, in proportion less in one of 2; many warps leave fewer parts of few
// long items to join. So CTAs of 2 warps from kManyItems items on (requests, or tokens with selected pages, times
// KV heads); the lengths are on the device, so the rule cannot see them. us with 8 (d = 256, or more than 8 rows: 4) warps
// / with 2, 8 KV heads, requests x keys:
//                    64 x 2-4 K  150 x 8-16 K  150 x 2-4 K  300 x 1-2 K  600 x 300-600  1024 x 150-300
//   d = 128,  4 rows   92 /  98   586 /  616    170 / 184    177 / 184     154 / 133      186 / 133
//   d =  64,  4 rows   56 /  54   330 /  328    109 / 104    123 / 108     120 /  88      150 /  98
//   d = 256,  2 rows  161 / 158  1153 / 1157    315 / 317    309 / 317     223 / 209      250 / 205
//   d = 128, 16 rows  102 / 100   653 /  633    203 / 193    225 / 208     208 / 175      260 / 203
//   d = 128, 32 rows  150 / 152  1043 / 1061    315 / 311    360 / 347     343 / 307      431 / 367
//   d = 256,  8 rows  158 / 174  1153 / 1159    320 / 326    326 / 328     246 / 225      283 / 229
//   d =  64, 32 rows  106 / 100   719 /  705    227 / 214    250 / 225     246 / 205      319 / 238
// Many long items lose up to 8 % by it (decode at d = 128), short ones gain up to a third.
constexpr int kManyItems = 1200;

template <int D, int NG, int W>
struct Cfg {
  static constexpr int ROWS = 8 * NG;
  static constexpr bool NARROW = NG == 1 && D <= 128;  // 128 registers: 16 warps per SM, else 8
  static constexpr int WARPS = W;
  static constexpr int STAGES = NG >= 4 ? 4 : 3;       // >= NG: the merge overlays the ring
  static constexpr int CTAS = (NARROW ? 16 : 8) / W;   // per SM
  static constexpr int KI = D / 64;                    // 16-byte K vectors per lane and key
  static constexpr int VB = D / 8;                     // V bytes per lane and key
  static constexpr int STAGE_BYTES = 32 * D;           // 16 keys of K and of V
  static constexpr int RING = WARPS * STAGES * STAGE_BYTES;
  static constexpr int MERGE = WARPS * ROWS * D * 4;
  static constexpr bool QREGS = NG * KI <= 4;          // query fragments: at most 32 registers, else shared memory
  static constexpr int OFF_Q = RING > MERGE ? RING : MERGE;
  static constexpr int OFF_META = OFF_Q + (QREGS ? 0 : NG * KI * 1024);
  static constexpr int OFF_SCALE = OFF_META + WARPS * 64 * 8;    // [warp][stage] k_scale, v_scale
  static constexpr int OFF_ML = OFF_SCALE + WARPS * STAGES * 8;
  static constexpr int SMEM = OFF_ML + WARPS * ROWS * 8;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }

// `bytes` of the source are read, the rest of the 16 (or 4) are zeros
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// D = A B + C, A 16x16 (rows g, g+8; columns 2t, 2t+1 | +8), B 16x8, fp32 accumulators
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (d0, d1) += s (x0, x1) in one instruction
__device__ __forceinline__ void fma2(float s, float x0, float x1, float& d0, float& d1) {
  uint64_t a, b, c;
  asm("mov.b64 %0, {%1, %1};" : "=l"(a) : "f"(s));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(x0), "f"(x1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(d0), "f"(d1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d0), "=f"(d1) : "l"(c));
}

// A unit of the work line: a request, or with selected pages a query token.
struct Unit {
  int tok0, nq;     // first token and tokens
  int b, pos0, len; // request, position of the first token, keys
  int key0, steps;  // first key (a multiple of 16) and 16-key steps; selected pages: steps of the list
  int tiles;        // row tiles
  int chunks;       // groups of kWarps steps (at least one, so that empty rows are written)
};

template <int ROWS, int WARPS>
__device__ __forceinline__ Unit unit_of(const FwdArgs& a, int u) {
  Unit x;
  if (a.selected) {
    x.tok0 = u;
    x.nq = a.b.token(u, x.b, x.pos0, x.len) ? 1 : 0;
    if (x.nq == 0) x.b = 0, x.pos0 = 0, x.len = 0;
    x.key0 = 0;
    const int pages = (a.b.hi(x.pos0, x.len) + (1 << a.b.page_shift) - 1) >> a.b.page_shift;
    x.steps = min(pages, a.n_selected) << (a.b.page_shift - 4);
  } else {
    x.b = u;
    x.tok0 = a.b.cu_q ? a.b.cu(u) : u;
    x.nq = a.b.cu_q ? max(0, a.b.cu(u + 1) - x.tok0) : 1;
    x.len = a.b.len(u);
    x.pos0 = x.len - x.nq;
    const int lo = a.b.lo(x.pos0), hi = a.b.hi(x.len - 1, x.len);
    x.key0 = lo & ~(kStep - 1);
    x.steps = hi > lo ? (hi - x.key0 + kStep - 1) / kStep : 0;
  }
  x.tiles = int((int64_t(x.nq) * a.group + ROWS - 1) / ROWS);
  x.chunks = max(1, (x.steps + WARPS - 1) / WARPS);
  return x;
}

template <int D, int NG, int W>
__global__ void __launch_bounds__(32 * W, Cfg<D, NG, W>::CTAS) kv8_fwd_kernel(FwdArgs a) {
  using C = Cfg<D, NG, W>;
  constexpr int ROWS = C::ROWS, KI = C::KI, S = C::STAGES, kWarps = C::WARPS, kThreads = 32 * kWarps;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_scan[kWarps], s_off;
  __shared__ int s_sum[kTries][kWarps];
  __shared__ int s_unit, s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t base = smem_addr(smem);
  const int ps = 1 << a.b.page_shift;

  wait_for_previous_kernel();
  if (tid == 0) s_unit = 0, s_off = 0;
  // ---- this CTA's part [line0, line1) of the line of places (T > 0: pieces, else chunks and starts) ----
  const int units = a.selected ? a.b.total_q : a.b.batch;
  const int per = (units + kThreads - 1) / kThreads, u0 = min(units, tid * per), u1 = min(units, u0 + per);
  // (64-bit division is slow)
  auto divide = [](long long x, long long y) { return (x | y) >> 31 ? x / y : (long long)(unsigned(x) / unsigned(y)); };
  const Unit unit0 = unit_of<ROWS, kWarps>(a, min(u0, units - 1));
  auto my_unit = [&](int u) { return u == u0 ? unit0 : unit_of<ROWS, kWarps>(a, u); };
  int T = 0;
  auto length_of = [&](const Unit& x) { return T ? (x.chunks + T - 1) / T : x.chunks + kStart; };   // places of an item
  auto line_of = [&](const Unit& x) { return (long long)length_of(x) * (x.tiles * a.hkv); };
  long long first = 0, mine = 0, total = 0;       // where this thread's units begin in the line, their places
  auto scan = [&] {
    mine = 0;
    for (int u = u0; u < u1; ++u) mine += line_of(my_unit(u));
    long long inc = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    first = inc - mine, total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) first += s_scan[w];
      total += s_scan[w];
    }
  };
  for (int pass = 0;; ++pass) {                   // a loop, so that the scan is there once
    scan();
    const int mean = int(min(divide(total, gridDim.x), 0x10000LL));
    if (pass == 1 || total <= gridDim.x || units > int(gridDim.x) || mean == 0x10000) break;
    int sum[kTries] = {};                         // pieces at each length
    for (int u = u0; u < u1; ++u) {
      const Unit x = my_unit(u);
      // in floating point: an estimate one off only moves a piece to a CTA that has one
      const float items = float(x.tiles) * float(a.hkv);
#pragma unroll
      for (int j = 0; j < kTries; ++j) {
        const float len = float(mean + 1 + mean * j / 16);
        sum[j] += int(fminf(items * ceilf(__fdividef(float(x.chunks), len)), 1e6f));
      }
    }
#pragma unroll
    for (int j = 0; j < kTries; ++j) {
      sum[j] = __reduce_add_sync(~0u, sum[j]);
      if (lane == 0) s_sum[j][warp] = sum[j];
    }
    __syncthreads();
    // lane j looks at length j
    int pieces = 0;
    if (lane < kTries)
#pragma unroll
      for (int w = 0; w < kWarps; ++w) pieces += s_sum[lane][w];
    const int len = mean + 1 + mean * lane / 16;
    const unsigned fits = __ballot_sync(~0u, lane < kTries && pieces <= int(gridDim.x) && len <= mean + kPiece);
    if (fits) T = __shfl_sync(~0u, len, __ffs(fits) - 1);
    if (T == 0) break;
  }
  const int G = int(min((long long)gridDim.x, total));
  if (int(blockIdx.x) >= G) return;
  // the first `more` CTAs take part + 1 places, the others part
  const long long part = divide(total, G);
  const int more = int(total - part * G);
  auto start_of = [&](int c) { return c * part + min(c, more); };
  auto cta_of = [&](long long x) {                // the CTA whose part holds x
    const long long wide = more * (part + 1);
    return int(x < wide ? divide(x, part + 1) : more + divide(x - wide, part));
  };
  const long long line0 = start_of(blockIdx.x), line1 = start_of(blockIdx.x + 1);
  if (first <= line0 && line0 < first + mine) {
    for (int u = u0; u < u1; ++u) {
      const long long n = line_of(my_unit(u));
      if (line0 < first + n) {
        s_unit = u;
        s_off = line0 - first;
        break;
      }
      first += n;
    }
  }
  __syncthreads();
  int unit = s_unit;
  long long off = s_off;                          // chunk offset inside the unit

  int2* s_meta = reinterpret_cast<int2*>(smem + C::OFF_META) + warp * 64;
  const float2* s_scale = reinterpret_cast<const float2*>(smem + C::OFF_SCALE) + warp * S;
  const uint32_t scale_addr = base + C::OFF_SCALE + warp * (S * 8) + (lane & 1) * 4;
  float2* s_ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
  float2* s_o = reinterpret_cast<float2*>(smem);
  // Chunk c (16 bytes) of a stage's row r lies at chunk c ^ s(r), s(r) = (((r >> 1) & 3) ^ ((r & 1) << 1)) << 1
  // (rows of 64 bytes: c ^ ((r >> 1) & 3)): of the eight lanes of one shared-memory phase, the K reads
  // have two neighbouring rows and four neighbouring chunks, the V reads four rows two apart and two
  // neighbouring chunks; both hit all eight chunks of a 128-byte line (64-byte rows: V two ways).
  const uint32_t ring = base + warp * (S * C::STAGE_BYTES);
  const int wr = lane / (D / 16), wc = lane % (D / 16);   // copies: row (of 512 bytes) and chunk of the lane
  const uint32_t copy_to = ring + wr * D + ((D == 64 ? wc ^ ((wr >> 1) & 3) : wc ^ ((((wr >> 1) & 3) ^ ((wr & 1) << 1)) << 1)) << 4);
  const uint32_t k_at = ring + g * D + ((D == 64 ? t ^ ((g >> 1) & 3) : t ^ ((((g >> 1) & 3) ^ ((g & 1) << 1)) << 1)) << 4);
  const uint32_t v_at = ring + 16 * D + 2 * t * D + (D == 64 ? (((g >> 1) ^ t) << 4) + (g & 1) * 8 : (g ^ (t << 1)) << 4);
  const uint32_t q_at = base + C::OFF_Q + lane * 16;

  for (long long line = line0; line < line1;) {
    const Unit x = unit_of<ROWS, kWarps>(a, unit);
    const long long unit_chunks = line_of(x);
    if (off >= unit_chunks) {                     // a unit without tokens, or done with
      if (++unit >= units) break;                 // (only if the lengths change while the kernel runs)
      off = 0;
      continue;
    }
    const int length = length_of(x), lead = T ? 0 : kStart;   // places that stand for the item's start
    const int item = int(divide(off, length)), p0 = int(off - (long long)item * length);
    const int p1 = int(min((long long)length, p0 + (line1 - line)));
    const int c0 = T ? int(divide((long long)x.chunks * p0, length)) : max(0, p0 - lead);
    const int c1 = T ? int(divide((long long)x.chunks * p1, length)) : max(0, p1 - lead);
    const long long item0 = line - p0;
    const bool at_start = line == line0;
    line += p1 - p0;
    off += p1 - p0;
    if (c0 == c1) continue;
    const int h = item / x.tiles, tile = item - h * x.tiles;
    const int row0 = tile * ROWS, rows = min(ROWS, x.nq * a.group - row0);
    const bool whole = c0 == 0 && c1 == x.chunks;

    // ---- the warp's steps: the i-th is step (c0 + i) kWarps + warp of the unit ----
    const int i0 = row0 / a.group, i1 = (row0 + rows - 1) / a.group;
    const int hi_all = a.b.hi(x.pos0 + i0, x.len), hi_any = a.b.hi(x.pos0 + i1, x.len);
    const int lo_any = a.b.lo(x.pos0 + i0), lo_all = a.b.lo(x.pos0 + i1);
    const int count = c1 - c0;
    // ---- queries: lane (g, t) takes channels 64 i + 16 t + 0 .. 15 of row g of each group, its fragments,
    // scaled by a power of two per row to below 2^15 in fp16. fac: score factor of rows 2t, 2t + 1
    // (the loads go before the keys', behind which they would wait)
    uint4 qw[NG][2 * KI];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const int r = row0 + 8 * n + g;
      const bool live = 8 * n + g < rows;
      const int i = live ? r / a.group : 0, head = live ? r - i * a.group : 0;
      const uint4* q = reinterpret_cast<const uint4*>(a.q + int64_t(x.tok0 + i) * a.q_stride + int64_t(h * a.group + head) * D + 16 * t);
#pragma unroll
      for (int j = 0; j < 2 * KI; ++j) qw[n][j] = live ? __ldg(q + (j >> 1) * 8 + (j & 1)) : make_uint4(0, 0, 0, 0);
    }
    // first key (-1: skip the step) and page (-1: outside the cache, zeros) of the 32 steps from i on
    auto load_meta = [&](int i) {
      const int st = (c0 + i + lane) * kWarps + warp;
      int key = -1, pg = -1;
      if (i + lane < count && st < x.steps) {
        int page, inner;
        if (a.selected) {
          const int j = st >> (a.b.page_shift - 4);
          page = __ldg(a.selected + (int64_t(x.tok0) * a.hkv + h) * a.n_selected + j);
          inner = (st << 4) & (ps - 1);
        } else {
          const int kk = x.key0 + st * kStep;
          page = kk >> a.b.page_shift;
          inner = kk & (ps - 1);
        }
        if (unsigned(page) < unsigned(a.b.max_pages)) {
          key = (page << a.b.page_shift) + inner;
          if (key >= hi_any || key + kStep <= lo_any) {
            key = -1;
          } else {
            pg = __ldg(a.b.page_table + int64_t(x.b) * a.b.max_pages + page);
            if (unsigned(pg) >= unsigned(a.num_pages)) pg = -1;
          }
        }
      }
      s_meta[(i + lane) & 63] = make_int2(key, pg);
      __syncwarp();
    };
    uint32_t put = 0, get = 0;                    // stage that the next copies go to, that the next step is in
    auto issue = [&](int i) {
      if (i < count) {
        if ((i & 31) == 0) load_meta(i);
        const int2 m = s_meta[i & 63];
        if (m.x >= 0) {
          const int bytes = m.y >= 0 ? 16 : 0;
          const int64_t block = int64_t(max(m.y, 0)) * a.hkv + h;
          const int64_t o = (block << a.b.page_shift) + (m.x & (ps - 1));
          const uint8_t* kp = a.k + o * D + lane * 16;
          const uint8_t* vp = a.v + o * D + lane * 16;
          const uint32_t st = put * C::STAGE_BYTES;
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {      // s() of the rows that the j-th 512 bytes hold
            const uint32_t flip = D == 128 ? (j & 1) * 64 : D == 256 ? (j & 3) * 32 : 0;
            cp16((copy_to ^ flip) + st + j * 512, kp + j * 512, bytes);
            cp16((copy_to ^ flip) + st + 16 * D + j * 512, vp + j * 512, bytes);
          }
          if (lane < 2) cp4(scale_addr + put * 8, (lane ? a.v_scale : a.k_scale) + block, bytes >> 2);
        }
      }
      cp_commit();
      put = put == S - 1 ? 0 : put + 1;
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(i);

    uint32_t qf[C::QREGS ? NG * KI * 8 : 1];
    float fac[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const bool live = 8 * n + g < rows;
      unsigned top = 0;
#pragma unroll
      for (int j = 0; j < 2 * KI; ++j) {
        const uint4 w = qw[n][j];
        const uint32_t v4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) top = __vmaxu2(top, v4[c] & 0x7fff7fffu);
      }
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(~0u, top, 1));
      top = max(top, __shfl_xor_sync(~0u, top, 2));
      // |q| < 2^(exponent + 1) -> below 2^15; infinities and NaN go through as they are
      const int e = top >= 0x7f80u ? 0 : min(100, 14 - (int(top >> 7) - 127));
      const float up = __int_as_float((127 + e) << 23);
      const float f = live ? a.scale_log2 * __int_as_float((127 - e) << 23) : 0.f;
      fac[n][0] = __shfl_sync(~0u, f, 8 * t);
      fac[n][1] = __shfl_sync(~0u, f, 8 * t + 4);
#pragma unroll
      for (int j = 0; j < 2 * KI; ++j) {
        uint32_t d[4];
        const uint4 w = qw[n][j];
        const uint32_t v4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float q0 = __uint_as_float(v4[2 * c] << 16), q1 = __uint_as_float(v4[2 * c] & 0xffff0000u);
          const float q2 = __uint_as_float(v4[2 * c + 1] << 16), q3 = __uint_as_float(v4[2 * c + 1] & 0xffff0000u);
          d[2 * c] = pack_half2(q0 * up, q1 * up);
          d[2 * c + 1] = pack_half2(q2 * up, q3 * up);
        }
        if constexpr (C::QREGS) {
#pragma unroll
          for (int c = 0; c < 4; ++c) qf[(n * 2 * KI + j) * 4 + c] = d[c];
        } else {                                  // every warp writes the same; a lane reads back its own
          *reinterpret_cast<uint4*>(smem + C::OFF_Q + (n * 2 * KI + j) * 512 + lane * 16) = make_uint4(d[0], d[1], d[2], d[3]);
        }
      }
    }
    auto sees = [&](int r, int& hi, int& lo) {    // keys of row r of the tile
      const int i = (row0 + r) / a.group;
      hi = r < rows ? a.b.hi(x.pos0 + i, x.len) : 0;
      lo = a.b.lo(x.pos0 + i);
    };

    float o[D / 16][NG][4];
    float m[NG][2], l[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      m[n][0] = m[n][1] = kNone;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.f;
    }

    for (int i = 0; i < count; ++i) {
      cp_wait<S - 2>();                           // this lane's copies of step i are there,
      __syncwarp();                               // every lane's are, and step i - 1 has been read
      issue(i + S - 1);
      const int key = s_meta[i & 63].x;
      const uint32_t st = get * C::STAGE_BYTES;
      const float2 scale = s_scale[get];
      get = get == S - 1 ? 0 : get + 1;
      if (key < 0) continue;

      // S^T = K Q^T
      float s[NG][4];
#pragma unroll
      for (int n = 0; n < NG; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int j = 0; j < KI; ++j) {
        const uint32_t kaddr = (k_at ^ ((j & 1) * 64)) + st + (j >> 1) * 128;
        const uint4 ka = lds128(kaddr), kb = lds128(kaddr + 8 * D);
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
        uint32_t frag[4][4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          frag[c][0] = half2_of_e4m3(wa[c]);
          frag[c][1] = half2_of_e4m3(wb[c]);
          frag[c][2] = half2_of_e4m3(wa[c] >> 16);
          frag[c][3] = half2_of_e4m3(wb[c] >> 16);
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          uint32_t b[8];
          if constexpr (C::QREGS) {
#pragma unroll
            for (int c = 0; c < 8; ++c) b[c] = qf[(n * KI + j) * 8 + c];
          } else {
            const uint4 q0 = lds128(q_at + (n * KI + j) * 1024), q1 = lds128(q_at + (n * KI + j) * 1024 + 512);
            b[0] = q0.x, b[1] = q0.y, b[2] = q0.z, b[3] = q0.w, b[4] = q1.x, b[5] = q1.y, b[6] = q1.z, b[7] = q1.w;
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) mma(s[n], frag[c], b[2 * c], b[2 * c + 1]);
        }
      }

      // scores in log2 units, masked; accumulator rows are keys key + g and key + g + 8
      const float ks = scale.x, vs = scale.y;
      const bool partial = key + kStep > hi_all || key < lo_all;
      bool out_of_range = false;                  // of a lane's two keys: it may be only these
#pragma unroll
      for (int n = 0; n < NG; ++n) {
#pragma unroll
        for (int c = 0; c < 4; ++c) s[n][c] *= fac[n][c & 1] * ks;
        if (partial) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            int hi, lo;
            sees(8 * n + 2 * t + c, hi, lo);
            if (key + g >= hi || key + g < lo) s[n][c] = -INFINITY;
            if (key + g + 8 >= hi || key + g + 8 < lo) s[n][c + 2] = -INFINITY;
          }
        }
        out_of_range |= (fabsf(fmaxf(s[n][0], s[n][2]) - m[n][0]) > kRange) | (fabsf(fmaxf(s[n][1], s[n][3]) - m[n][1]) > kRange);
      }
      if (__any_sync(~0u, out_of_range)) {        // move the references and rescale
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x2 = fmaxf(s[n][c], s[n][c + 2]);
            x2 = fmaxf(x2, __shfl_xor_sync(~0u, x2, 4));
            x2 = fmaxf(x2, __shfl_xor_sync(~0u, x2, 8));
            x2 = fmaxf(x2, __shfl_xor_sync(~0u, x2, 16));
            float sum = l[n][c];
            sum += __shfl_xor_sync(~0u, sum, 4);
            sum += __shfl_xor_sync(~0u, sum, 8);
            sum += __shfl_xor_sync(~0u, sum, 16);
            const bool low = x2 < m[n][c] - kRange && x2 > -INFINITY;
            float to = x2 - kHead;
            if (low) to = fmaxf(to, m[n][c] - max(0, kGrow - ((__float_as_int(sum) >> 23) - 127)));
            if (low || to > m[n][c]) {
              const float r = ex2(m[n][c] - to);
              m[n][c] = to;
              l[n][c] *= r;
#pragma unroll
              for (int j = 0; j < D / 16; ++j) {
                o[j][n][c] *= r;
                o[j][n][c + 2] *= r;
              }
            }
          }
      }
      uint32_t p0[NG], p1[NG];
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const float e0 = ex2(s[n][0] - m[n][0]), e1 = ex2(s[n][1] - m[n][1]);
        const float e2 = ex2(s[n][2] - m[n][0]), e3 = ex2(s[n][3] - m[n][1]);
        l[n][0] += e0 + e2;
        l[n][1] += e1 + e3;
        p0[n] = transpose8(pack_half2(e0, e1));
        p1[n] = transpose8(pack_half2(e2, e3));
      }

      // O^T += v_scale V^T P^T. The page's scale multiplies the fp32 products, so P keeps its 11
      // bits whatever the scales of the pages are.
      uint32_t vw[4][C::VB / 4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (D == 64) {
          const uint2 w = lds64(v_at + st + ((j & 1) + (j >> 1) * 8) * D);
          vw[j][0] = w.x, vw[j][1] = w.y;
        } else {
#pragma unroll
          for (int v = 0; v < C::VB / 16; ++v) {
            const uint4 w = lds128((v_at ^ ((j & 1) * 64)) + st + ((j & 1) + (j >> 1) * 8) * D + v * 128);
            vw[j][4 * v] = w.x, vw[j][4 * v + 1] = w.y, vw[j][4 * v + 2] = w.z, vw[j][4 * v + 3] = w.w;
          }
        }
      }
      if (partial) {
        // a slot behind the request's last token may hold any byte, and 0 * NaN would spread
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (key + 2 * t + (j & 1) + (j >> 1) * 8 >= hi_any)
#pragma unroll
            for (int w = 0; w < C::VB / 4; ++w) vw[j][w] = 0u;
      }
      if (vs != vs) {                             // a page that holds a NaN: for the rows that see a key of the step
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            int hi, lo;
            sees(8 * n + 2 * t + c, hi, lo);
            if (min(hi, key + kStep) > max(lo, key))
#pragma unroll
              for (int j = 0; j < D / 16; ++j) o[j][n][c] = o[j][n][c + 2] = vs;
          }
        continue;
      }
#pragma unroll
      for (int w = 0; w < C::VB / 4; ++w) {
        // bytes 4w .. 4w+3 of the lane's channels: rows g and g + 8 of tiles 2w and 2w + 1
        uint32_t f0[4], f1[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {             // keys 2t, 2t+1, then 2t+8, 2t+9
          const uint32_t c01 = __byte_perm(vw[2 * j][w], vw[2 * j + 1][w], 0x5140);
          const uint32_t c23 = __byte_perm(vw[2 * j][w], vw[2 * j + 1][w], 0x7362);
          f0[2 * j] = half2_of_e4m3(c01), f0[2 * j + 1] = half2_of_e4m3(c01 >> 16);
          f1[2 * j] = half2_of_e4m3(c23), f1[2 * j + 1] = half2_of_e4m3(c23 >> 16);
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
          mma(x0, f0, p0[n], p1[n]);
          mma(x1, f1, p0[n], p1[n]);
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            fma2(vs, x0[c], x0[c + 1], o[2 * w][n][c], o[2 * w][n][c + 1]);
            fma2(vs, x1[c], x1[c + 1], o[2 * w + 1][n][c], o[2 * w + 1][n][c + 1]);
          }
        }
      }
    }
    cp_wait<0>();

    // ---- merge the warps in shared memory (over the ring). Channel pair p of row r lies at p ^ y, y from
    // the writing lane's t and g, so that a warp's 8-byte writes take two phases, the least
    __syncthreads();
    const int y = D == 64 ? t : 2 * t + ((g >> 1) & 1);
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[n][c];
        sum += __shfl_xor_sync(~0u, sum, 4);
        sum += __shfl_xor_sync(~0u, sum, 8);
        sum += __shfl_xor_sync(~0u, sum, 16);
        const int r = 8 * n + 2 * t + c;
        if (g == 0) s_ml[warp * ROWS + r] = make_float2(m[n][c], sum);
        float2* dst = s_o + (warp * ROWS + r) * (D / 2);
#pragma unroll
        for (int j = 0; j < D / 16; ++j)          // channels 4w + 2 (j & 1) of the lane, w = j / 2; 16 of each 128
          dst[(g * (D == 64 ? 4 : 8) + (j >> 3) * 64 + (j & 7)) ^ y] = make_float2(o[j][n][c], o[j][n][c + 2]);
      }
    __syncthreads();

    auto finish = [&](int r, int d4, float4 acc, float M, float Z) {
      const int i = (row0 + r) / a.group;
      const int64_t orow = int64_t(x.tok0 + i) * (a.group * a.hkv) + h * a.group + (row0 + r - i * a.group);
      const float inv = Z > 0.f || Z != Z ? 1.f / Z : 0.f;
      const __nv_bfloat162 lo2 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi2 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(a.out + orow * D + d4 * 4) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo2), *reinterpret_cast<const uint32_t*>(&hi2));
      if (a.lse && d4 == 0) a.lse[orow] = Z == 0.f ? -INFINITY : (M + log2f(Z)) * 0.6931471805599453f;
    };
    for (int idx = tid; idx < rows * (D / 4); idx += kThreads) {
      const int r = idx / (D / 4), d4 = idx % (D / 4);
      const int gg = D == 64 ? 0 : (d4 >> 2) & 7, yy = D == 64 ? (r >> 1) & 3 : 2 * ((r >> 1) & 3) + ((gg >> 1) & 1);
      float M = kNone;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w * ROWS + r].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float Z = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = s_ml[w * ROWS + r];
        const float e = ex2(ml.x - M);
        const float2* src = s_o + (w * ROWS + r) * (D / 2);
        const float2 v0 = src[(2 * d4) ^ yy], v1 = src[(2 * d4 + 1) ^ yy];
        Z = fmaf(e, ml.y, Z);
        acc.x = fmaf(e, v0.x, acc.x), acc.y = fmaf(e, v0.y, acc.y), acc.z = fmaf(e, v1.x, acc.z), acc.w = fmaf(e, v1.y, acc.w);
      }
      if (whole) {
        finish(r, d4, acc, M, Z);
      } else {
        // a CTA has at most two parts of items: one at the start of its line, one at the end
        const int64_t slot = 2 * blockIdx.x + (at_start ? 0 : 1);
        __stcg(reinterpret_cast<float4*>(a.part_o + (slot * ROWS + r) * D + d4 * 4), acc);
        if (d4 == 0) __stcg(reinterpret_cast<float2*>(a.part_ml + (slot * ROWS + r) * 2), make_float2(M, Z));
      }
    }
    if (!whole) {                                 // the last CTA of the item to arrive joins the parts
      const int fc = cta_of(item0 + lead), n = cta_of(item0 + length - 1) - fc + 1;
      __syncthreads();
      if (tid == 0) {                             // releases this CTA's part, acquires the others'
        uint32_t old;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(a.counters + fc) : "memory");
        s_last = old == uint32_t(n - 1);
        if (s_last) a.counters[fc] = 0u;
      }
      __syncthreads();
      if (s_last) {
        // parts at slots 2 c, but the first one's where it is not the start of its CTA's line
        const int odd = start_of(fc) >= item0 ? 0 : 1;
        const float2* pml = reinterpret_cast<const float2*>(a.part_ml) + int64_t(2 * fc) * ROWS;
        const float4* po = reinterpret_cast<const float4*>(a.part_o + int64_t(2 * fc) * (ROWS * D));
        // the 32 lanes of a warp (D = 64: each 16) hold one row: lane c the weight of part c
        constexpr int PW = D == 64 ? 16 : 32, N = (ROWS * D / 4 + kThreads - 1) / kThreads;
        // The first P parts are on their way while the weights are worked out. One at d = 256 (16 verifications:
        // 48.8 us, 51.0 without), none in the tile of 32 rows, whose registers spill (96 rows of 32 requests: 203, 196)
        constexpr int P = N <= 2 ? 8 / N : D == 256 ? 1 : 0;
        float M[N], Z[N], w[N];
        float4 acc[N];
#pragma unroll
        for (int k = 0; k < N; ++k) M[k] = kNone, Z[k] = 0.f, acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int b0 = 0; b0 < n; b0 += PW) {
          const int mc = b0 + (lane & (PW - 1)), nb = min(PW, n - b0);
          auto part = [&](int c, int k) {
            const int slot = b0 + c == 0 ? odd : 2 * (b0 + c);
            return __ldcg(po + slot * (ROWS * D / 4) + min(ROWS * D / 4 - 1, tid + k * kThreads));
          };
          float4 early[P ? P : 1][N];
#pragma unroll
          for (int c = 0; c < P; ++c)
#pragma unroll
            for (int k = 0; k < N; ++k)
              if (c < nb) early[c][k] = part(c, k);
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const int r = min(ROWS - 1, (tid + k * kThreads) / (D / 4));
            float2 ml = make_float2(kNone, 0.f);
            if (mc < n) ml = __ldcg(pml + (mc == 0 ? odd : 2 * mc) * ROWS + r);
            float Mn = ml.x;
#pragma unroll
            for (int o2 = PW / 2; o2; o2 >>= 1) Mn = fmaxf(Mn, __shfl_xor_sync(~0u, Mn, o2));
            Mn = fmaxf(Mn, M[k]);
            w[k] = ex2(ml.x - Mn);
            float zs = w[k] * ml.y;
#pragma unroll
            for (int o2 = PW / 2; o2; o2 >>= 1) zs += __shfl_xor_sync(~0u, zs, o2);
            const float e0 = ex2(M[k] - Mn);
            M[k] = Mn;
            Z[k] = fmaf(Z[k], e0, zs);
            acc[k].x *= e0, acc[k].y *= e0, acc[k].z *= e0, acc[k].w *= e0;
          }
          auto add = [&](int c, int k, const float4& v) {
            const float e = __shfl_sync(~0u, w[k], c, PW);
            acc[k].x = fmaf(e, v.x, acc[k].x), acc[k].y = fmaf(e, v.y, acc[k].y);
            acc[k].z = fmaf(e, v.z, acc[k].z), acc[k].w = fmaf(e, v.w, acc[k].w);
          };
#pragma unroll
          for (int c = 0; c < P; ++c)
#pragma unroll
            for (int k = 0; k < N; ++k)
              if (c < nb) add(c, k, early[c][k]);
#pragma unroll(N == 1 ? 8 : 4)
          for (int c = P; c < nb; ++c)
#pragma unroll
            for (int k = 0; k < N; ++k) add(c, k, part(c, k));
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const int idx = tid + k * kThreads;
          if (idx / (D / 4) < rows) finish(idx / (D / 4), idx % (D / 4), acc[k], M[k], Z[k]);
        }
      }
    }
    __syncthreads();                              // the next item writes the ring
  }
}

using Kernel = void (*)(FwdArgs);

struct Choice {
  Kernel kernel;
  int smem, ctas, threads;
};

template <int D, int NG>
Choice pick(bool many) {
  constexpr int FEW = Cfg<D, NG, 2>::NARROW ? 8 : 4;
  if (many) return {kv8_fwd_kernel<D, NG, 2>, Cfg<D, NG, 2>::SMEM, Cfg<D, NG, 2>::CTAS, 64};
  return {kv8_fwd_kernel<D, NG, FEW>, Cfg<D, NG, FEW>::SMEM, Cfg<D, NG, FEW>::CTAS, 32 * FEW};
}

// head_dim 256: at most 16 rows (the accumulators of 32 would take every register)
Choice choice_of(int d, int ng, bool many) {
  if (d == 64) return ng == 1 ? pick<64, 1>(many) : ng == 2 ? pick<64, 2>(many) : pick<64, 4>(many);
  if (d == 128) return ng == 1 ? pick<128, 1>(many) : ng == 2 ? pick<128, 2>(many) : pick<128, 4>(many);
  return ng == 1 ? pick<256, 1>(many) : pick<256, 2>(many);
}

}  // namespace
}  // namespace kv8

using namespace kv8;

extern "C" {

attn_status_t attn_kv8_plan(const attn_kv8_problem_t* problem, attn_kv8_plan_t** out_plan) {
  if (!problem || !out_plan) return ATTN_ERR_INVALID_ARG;
  *out_plan = nullptr;
  const attn_kv8_problem_t& p = *problem;
  if (p.hq < 1 || p.hkv < 1 || p.hq % p.hkv || p.hq > 65535 || p.max_q_len < 1) return ATTN_ERR_INVALID_ARG;
  if (p.head_dim != 64 && p.head_dim != 128 && p.head_dim != 256) return ATTN_ERR_UNSUPPORTED;
  const int shift = shift_of(p.page_size);
  if (shift < 0) return ATTN_ERR_UNSUPPORTED;
  if (!(p.scale == p.scale)) return ATTN_ERR_INVALID_ARG;
  if (p.mask == ATTN_MASK_SLIDING_WINDOW) {
    if (p.window < 1) return ATTN_ERR_INVALID_ARG;
  } else if (p.mask != ATTN_MASK_FULL && p.mask != ATTN_MASK_CAUSAL) {
    return ATTN_ERR_UNSUPPORTED;
  }
  attn_kv8_plan_t* pl = new (std::nothrow) attn_kv8_plan_t;
  if (!pl) return ATTN_ERR_OOM;
  pl->hq = p.hq;
  pl->hkv = p.hkv;
  pl->d = p.head_dim;
  pl->page_size = p.page_size;
  pl->page_shift = shift;
  pl->scale = p.scale > 0.f ? p.scale : p.head_dim == 64 ? 0.125f : p.head_dim == 128 ? 0.08838834764831845f : 0.0625f;
  pl->mask = p.mask;
  pl->window = p.window;
  const int64_t rows = int64_t(p.hq / p.hkv) * p.max_q_len;
  pl->ng = rows <= 8 ? 1 : rows <= 16 || p.head_dim == 256 ? 2 : 4;
  int sms = 0;
  cudaError_t e = cudaGetDevice(&pl->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, pl->device);
  for (int many = 0; many < 2; ++many) {
    const Choice c = choice_of(pl->d, pl->ng, many);
    int fit = 0;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(c.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, c.smem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, c.kernel, c.threads, c.smem);
    pl->grid[many] = sms * std::max(1, std::min(fit, c.ctas));
  }
  const int grid = std::max(pl->grid[0], pl->grid[1]);
  const size_t tile = size_t(8) * pl->ng, slots = size_t(2) * grid;
  const size_t bytes_o = slots * tile * pl->d * 4, bytes_ml = slots * tile * 8, bytes_c = size_t(grid) * 4;
  if (e == cudaSuccess) {
    e = cudaMalloc(&pl->ws, bytes_o + bytes_ml + bytes_c);
    if (e == cudaSuccess) {
      char* w = static_cast<char*>(pl->ws);
      pl->part_o = reinterpret_cast<float*>(w);
      pl->part_ml = reinterpret_cast<float*>(w + bytes_o);
      pl->counters = reinterpret_cast<uint32_t*>(w + bytes_o + bytes_ml);
      e = cudaMemset(pl->counters, 0, bytes_c);
      if (e == cudaSuccess) e = cudaDeviceSynchronize();
    }
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    if (pl->ws) cudaFree(pl->ws);
    delete pl;
    return e == cudaErrorMemoryAllocation ? ATTN_ERR_OOM : ATTN_ERR_CUDA;
  }
  *out_plan = pl;
  return ATTN_OK;
}

attn_status_t attn_kv8_plan_destroy(attn_kv8_plan_t* plan) {
  if (!plan) return ATTN_OK;
  const cudaError_t e = plan->ws ? cudaFree(plan->ws) : cudaSuccess;
  delete plan;
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_kv8_fwd(const attn_kv8_plan_t* p, const attn_kv8_cache_t* c, const attn_kv8_batch_t* b,
                           const int32_t* selected, int32_t n_selected, void* out, float* lse, attn_stream_t stream) {
  const attn_status_t st = check_batch(p, c, b);
  if (st != ATTN_OK) return st;
  if (selected && (n_selected < 1 || int64_t(n_selected) * p->page_size >= (int64_t(1) << 31) || misaligned(selected, 4)))
    return ATTN_ERR_INVALID_ARG;
  if (b->total_q == 0 || b->batch == 0) return ATTN_OK;
  if (!out || misaligned(out, 16) || misaligned(lse, 4)) return ATTN_ERR_INVALID_ARG;
  const int64_t row = int64_t(p->hq) * p->d;
  if (overlap(b->q, (int64_t(b->total_q - 1) * b->q_stride + row) * 2, out, int64_t(b->total_q) * row * 2)) return ATTN_ERR_INVALID_ARG;
  if (overlap(out, int64_t(b->total_q) * row * 2, lse, int64_t(b->total_q) * p->hq * 4)) return ATTN_ERR_INVALID_ARG;
  FwdArgs a{};
  a.b = batch_of(p, b);
  a.q = static_cast<const __nv_bfloat16*>(b->q);
  a.q_stride = b->q_stride;
  a.k = static_cast<const uint8_t*>(c->k);
  a.v = static_cast<const uint8_t*>(c->v);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.num_pages = c->num_pages;
  a.hkv = p->hkv;
  a.group = p->hq / p->hkv;
  a.scale_log2 = p->scale * 1.4426950408889634f;
  a.selected = selected;
  a.n_selected = n_selected;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.part_o = p->part_o;
  a.part_ml = p->part_ml;
  a.counters = p->counters;
  const int many = int64_t(selected ? b->total_q : b->batch) * p->hkv >= kManyItems;
  const Choice k = choice_of(p->d, p->ng, many);
  return launch(k.kernel, dim3(p->grid[many]), k.threads, k.smem, stream, a);
}

}  // extern "C"
