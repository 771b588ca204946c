// Attention of a few query tokens per request over the 8-bit paged K/V cache.
//
// Mathematics. Per request, KV head h and query row n (a token and a query head of h's group):
//     s_j = scale k_scale[page(j)] (q_n . code_j),  p_j = 2^(s_j log2 e - m_n),
//     out = sum_j p_j v_scale[page(j)] code_j / sum_j p_j,  lse = m_n ln 2 + ln sum_j p_j
// with the running maximum m_n. e4m3 codes convert to fp16 exactly and q is scaled by a power of
// two per row into fp16 range, so the products are exact; both matrix products run on
// mma.sync m16n8k16 with fp32 accumulators, transposed: S^T = K Q^T and O^T = V^T P^T, keys or
// channels on the 16-row side and 8 query rows on the other, so the eight rows of a grouped
// decode step fill a tile (as the 128-row side of a tcgen05 MMA they would use 6 % of it).
//
// What bounds it: HBM. 2 d bytes per key and KV head are read once; at the measured copy rate
// an SM receives ~23 bytes per clock. The conversion comes next: cvt.f16x2.e4m3x2 measured ~4 clocks
// of the SM per warp instruction (profiled: the XU pipe 73 % busy at 3.1 TB/s, nothing else above
// 27 %), which alone caps the stream at 16 bytes per clock. So K and half of V are converted by
// shifts and logic: the code's sign, exponent and mantissa moved into an fp16 give code / 256,
// exactly (subnormals too), and the factor goes into the scales.
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
// Work. The steps of all (request, KV head, row tile) items form one line, cut into equal
// parts for the persistent CTAs (each scans the lengths itself); within a CTA the warps take
// alternate steps of an item and merge in shared memory. An item whose chunks several CTAs share
// is joined by the last of them to arrive (an atomic counter that it resets), in
// CTA order, so results do not depend on timing and nothing waits.

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

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 16;                 // keys per step
constexpr float kLazy = 8.f;              // log2 units a score may exceed the running maximum by

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

template <int D, int NG>
struct Cfg {
  static constexpr int ROWS = 8 * NG;
  static constexpr int STAGES = NG >= 4 ? 4 : 3;       // >= NG: the merge overlays the ring
  static constexpr int CTAS = NG == 1 ? (D == 256 ? 2 : 4) : 2;   // per SM
  static constexpr int KI = D / 64;                    // 16-byte K vectors per lane and key
  static constexpr int VB = D / 8;                     // V bytes per lane and key
  static constexpr int STAGE_BYTES = 32 * D;           // 16 keys of K and of V
  static constexpr int RING = kWarps * STAGES * STAGE_BYTES;
  static constexpr int MERGE = kWarps * ROWS * D * 4;
  static constexpr int QPITCH = D + 8;                 // halves; the pad spreads rows over banks
  static constexpr int OFF_Q = RING > MERGE ? RING : MERGE;
  static constexpr int OFF_META = OFF_Q + ROWS * QPITCH * 2;
  static constexpr int OFF_SCALE = OFF_META + kWarps * 64 * 8;    // [warp][stage] k_scale, v_scale
  static constexpr int OFF_ML = OFF_SCALE + kWarps * STAGES * 8;
  static constexpr int OFF_ROW = OFF_ML + kWarps * ROWS * 8;      // [ROWS] factor, hi, lo, out row
  static constexpr int SMEM = OFF_ROW + ROWS * 16;
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

// The codes in the odd / even bytes of w as two halves (lower byte first) of code / 256: the
// sign stays on top, exponent and mantissa move down by one bit (fp16 has a fifth exponent bit).
__device__ __forceinline__ uint32_t half2_of_odd(uint32_t w) { return (w & 0x80008000u) | ((w >> 1) & 0x3f803f80u); }
__device__ __forceinline__ uint32_t half2_of_even(uint32_t w) { return ((w << 8) & 0x80008000u) | ((w << 7) & 0x3f803f80u); }

// A unit of the work line: a request, or with selected pages a query token.
struct Unit {
  int tok0, nq;     // first token and tokens
  int b, pos0, len; // request, position of the first token, keys
  int key0, steps;  // first key (a multiple of 16) and 16-key steps; selected pages: steps of the list
  int tiles;        // row tiles
  int chunks;       // groups of kWarps steps (at least one, so that empty rows are written)
};

template <int ROWS>
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
  x.chunks = max(1, (x.steps + kWarps - 1) / kWarps);
  return x;
}

template <int D, int NG>
__global__ void __launch_bounds__(kThreads, Cfg<D, NG>::CTAS) kv8_fwd_kernel(FwdArgs a) {
  using C = Cfg<D, NG>;
  constexpr int ROWS = C::ROWS, KI = C::KI, S = C::STAGES;
  constexpr bool kQRegs = NG * KI <= 4;           // Q fragments: at most 32 registers, else from shared memory
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_scan[kWarps], s_found;
  __shared__ int s_unit, s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t base = smem_addr(smem);
  const int ps = 1 << a.b.page_shift;

  // ---- this CTA's part [line0, line1) of the line of chunks ----
  const int units = a.selected ? a.b.total_q : a.b.batch;
  auto line_of = [&](const Unit& x) { return (long long)x.chunks * x.tiles * a.hkv; };
  const int per = (units + kThreads - 1) / kThreads, u0 = min(units, tid * per), u1 = min(units, u0 + per);
  long long mine = 0;
  for (int u = u0; u < u1; ++u) mine += line_of(unit_of<ROWS>(a, u));
  long long inc = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_scan[warp] = inc;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const int G = int(min((long long)gridDim.x, total));
  if (int(blockIdx.x) >= G) return;
  // the first `more` CTAs take part + 1 chunks, the others part
  auto divide = [](long long x, long long y) { return (x | y) >> 31 ? x / y : (long long)(unsigned(x) / unsigned(y)); };
  const long long part = divide(total, G);
  const int more = int(total - part * G);
  auto start_of = [&](int c) { return c * part + min(c, more); };
  auto cta_of = [&](long long x) {                // the CTA whose part holds x
    const long long wide = more * (part + 1);
    return int(x < wide ? divide(x, part + 1) : more + divide(x - wide, part));
  };
  const long long line0 = start_of(blockIdx.x), line1 = start_of(blockIdx.x + 1);
  long long first = before + inc - mine;          // the line where this thread's units begin
  if (first <= line0 && line0 < first + mine) {
    for (int u = u0; u < u1; ++u) {
      const long long n = line_of(unit_of<ROWS>(a, u));
      if (line0 < first + n) {
        s_unit = u;
        s_found = line0 - first;
        break;
      }
      first += n;
    }
  }
  __syncthreads();
  int unit = s_unit;
  long long off = s_found;                        // chunk offset inside the unit

  __half* s_q = reinterpret_cast<__half*>(smem + C::OFF_Q);
  int2* s_meta = reinterpret_cast<int2*>(smem + C::OFF_META) + warp * 64;
  const float2* s_scale = reinterpret_cast<const float2*>(smem + C::OFF_SCALE) + warp * S;
  const uint32_t scale_addr = base + C::OFF_SCALE + warp * (S * 8) + (lane & 1) * 4;
  float2* s_ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
  int4* s_row = reinterpret_cast<int4*>(smem + C::OFF_ROW);
  float* s_o = reinterpret_cast<float*>(smem);
  // Chunk c (16 bytes) of a stage's row r lies at chunk c ^ s(r), s(r) = (((r >> 1) & 3) ^ ((r & 1) << 1)) << 1
  // (rows of 64 bytes: c ^ ((r >> 1) & 3)): of the eight lanes of one shared-memory phase, the K reads
  // have two neighbouring rows and four neighbouring chunks, the V reads four rows two apart and two
  // neighbouring chunks; both hit all eight chunks of a 128-byte line (64-byte rows: V two ways).
  const uint32_t ring = base + warp * (S * C::STAGE_BYTES);
  const int wr = lane / (D / 16), wc = lane % (D / 16);   // copies: row (of 512 bytes) and chunk of the lane
  const uint32_t copy_to = ring + wr * D + ((D == 64 ? wc ^ ((wr >> 1) & 3) : wc ^ ((((wr >> 1) & 3) ^ ((wr & 1) << 1)) << 1)) << 4);
  const uint32_t k_at = ring + g * D + ((D == 64 ? t ^ ((g >> 1) & 3) : t ^ ((((g >> 1) & 3) ^ ((g & 1) << 1)) << 1)) << 4);
  const uint32_t v_at = ring + 16 * D + 2 * t * D + (D == 64 ? (((g >> 1) ^ t) << 4) + (g & 1) * 8 : (g ^ (t << 1)) << 4);

  for (long long line = line0; line < line1;) {
    const Unit x = unit_of<ROWS>(a, unit);
    const long long unit_chunks = line_of(x);
    if (off >= unit_chunks) {                     // a unit without tokens
      ++unit;
      off = 0;
      continue;
    }
    const int item = int(off / x.chunks), c0 = int(off - (long long)item * x.chunks);
    const int c1 = int(min((long long)x.chunks, c0 + (line1 - line)));
    const int h = item / x.tiles, tile = item - h * x.tiles;
    const int rows = int(min((long long)ROWS, (long long)x.nq * a.group - (long long)tile * ROWS));

    // ---- the warp's steps: the i-th is step (c0 + i) kWarps + warp of the unit ----
    const int i0 = int(int64_t(tile) * ROWS / a.group), i1 = int((int64_t(tile) * ROWS + rows - 1) / a.group);
    const int hi_all = a.b.hi(x.pos0 + i0, x.len), hi_any = a.b.hi(x.pos0 + i1, x.len);
    const int lo_any = a.b.lo(x.pos0 + i0), lo_all = a.b.lo(x.pos0 + i1);
    const int count = c1 - c0;
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
          const uint32_t st = uint32_t(i % S) * C::STAGE_BYTES;
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {      // s() of the rows that the j-th 512 bytes hold
            const uint32_t flip = D == 128 ? (j & 1) * 64 : D == 256 ? (j & 3) * 32 : 0;
            cp16((copy_to ^ flip) + st + j * 512, kp + j * 512, bytes);
            cp16((copy_to ^ flip) + st + 16 * D + j * 512, vp + j * 512, bytes);
          }
          if (lane < 2) cp4(scale_addr + uint32_t(i % S) * 8, (lane ? a.v_scale : a.k_scale) + block, bytes >> 2);
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(i);

    // ---- rows of the tile: query in fp16, score factor, visible keys ----
    for (int r = warp; r < ROWS; r += kWarps) {
      constexpr int E = D / 32;
      float f[E];
      unsigned top = 0;
      int hi = 0, lo = 0, orow = -1;
#pragma unroll
      for (int j = 0; j < E; ++j) f[j] = 0.f;
      if (r < rows) {
        const int64_t rr = int64_t(tile) * ROWS + r;
        const int i = int(rr / a.group), head = h * a.group + int(rr - int64_t(i) * a.group);
        const __nv_bfloat16* q = a.q + int64_t(x.tok0 + i) * a.q_stride + int64_t(head) * D + lane * E;
        uint32_t w[(E + 1) / 2];
        if constexpr (E == 2) w[0] = __ldg(reinterpret_cast<const uint32_t*>(q));
        else if constexpr (E == 4) *reinterpret_cast<uint2*>(w) = __ldg(reinterpret_cast<const uint2*>(q));
        else *reinterpret_cast<uint4*>(w) = __ldg(reinterpret_cast<const uint4*>(q));
#pragma unroll
        for (int j = 0; j < E; ++j) {
          f[j] = __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
          top = max(top, (__float_as_uint(f[j]) >> 16) & 0x7fffu);
        }
        hi = a.b.hi(x.pos0 + i, x.len);
        lo = a.b.lo(x.pos0 + i);
        orow = (x.tok0 + i) * (a.group * a.hkv) + head;
      }
      top = __reduce_max_sync(~0u, top);
      // |q| < 2^(exponent + 1) -> below 2^15; infinities and NaN go through as they are
      const int e = top >= 0x7f80u ? 0 : min(100, 14 - (int(top >> 7) - 127));
      const float f2 = __int_as_float((127 + e) << 23);
      __half* dst = s_q + r * C::QPITCH + lane * E;
      // channels 0 1 2 3 of each four are stored as 1 3 0 2, the order in which the K codes convert
      if constexpr (E == 2) {
        const uint32_t two = pack_half2(f[0] * f2, f[1] * f2);
        __half* d4 = s_q + r * C::QPITCH + (lane >> 1) * 4 + (lane & 1);
        *reinterpret_cast<uint16_t*>(d4 + 2) = uint16_t(two);
        *reinterpret_cast<uint16_t*>(d4) = uint16_t(two >> 16);
      } else {
#pragma unroll
        for (int j = 0; j < E; j += 4)
          *reinterpret_cast<uint2*>(dst + j) =
              make_uint2(pack_half2(f[j + 1] * f2, f[j + 3] * f2), pack_half2(f[j] * f2, f[j + 2] * f2));
      }
      // 256: the K codes convert to code / 256
      if (lane == 0)
        s_row[r] = make_int4(__float_as_int(r < rows ? 256.f * a.scale_log2 * __int_as_float((127 - e) << 23) : 0.f), hi, lo, orow);
    }
    __syncthreads();

    uint32_t qf[kQRegs ? NG * KI * 8 : 1];
    const uint32_t qaddr = base + C::OFF_Q + g * (C::QPITCH * 2) + t * 32;
    if constexpr (kQRegs) {
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int i = 0; i < KI; ++i) {
          const uint4 q0 = lds128(qaddr + n * (8 * C::QPITCH * 2) + i * 128), q1 = lds128(qaddr + n * (8 * C::QPITCH * 2) + i * 128 + 16);
          uint32_t* d = qf + (n * KI + i) * 8;
          d[0] = q0.x, d[1] = q0.y, d[2] = q0.z, d[3] = q0.w, d[4] = q1.x, d[5] = q1.y, d[6] = q1.z, d[7] = q1.w;
        }
    }
    float fac[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      fac[n][0] = __int_as_float(s_row[8 * n + 2 * t].x);
      fac[n][1] = __int_as_float(s_row[8 * n + 2 * t + 1].x);
    }

    float o[D / 16][NG][4];
    float m[NG][2], l[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.f;
    }
    for (int i = 0; i < count; ++i) {
      cp_wait<S - 2>();                           // this lane's copies of step i are there,
      __syncwarp();                               // every lane's are, and step i - 1 has been read
      issue(i + S - 1);
      const int key = s_meta[i & 63].x;
      if (key < 0) continue;
      const float2 scale = s_scale[i % S];
      const uint32_t st = uint32_t(i % S) * C::STAGE_BYTES;

      // S^T = K Q^T
      float s[NG][4];
#pragma unroll
      for (int n = 0; n < NG; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int j = 0; j < KI; ++j) {
        const uint32_t at = (k_at ^ ((j & 1) * 64)) + st + (j >> 1) * 128;
        const uint4 ka = lds128(at), kb = lds128(at + 8 * D);
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
        uint32_t frag[4][4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          frag[c][0] = half2_of_odd(wa[c]);
          frag[c][1] = half2_of_odd(wb[c]);
          frag[c][2] = half2_of_even(wa[c]);
          frag[c][3] = half2_of_even(wb[c]);
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          uint32_t b[8];
          if constexpr (kQRegs) {
#pragma unroll
            for (int c = 0; c < 8; ++c) b[c] = qf[(n * KI + j) * 8 + c];
          } else {
            const uint4 q0 = lds128(qaddr + n * (8 * C::QPITCH * 2) + j * 128), q1 = lds128(qaddr + n * (8 * C::QPITCH * 2) + j * 128 + 16);
            b[0] = q0.x, b[1] = q0.y, b[2] = q0.z, b[3] = q0.w, b[4] = q1.x, b[5] = q1.y, b[6] = q1.z, b[7] = q1.w;
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) mma(s[n], frag[c], b[2 * c], b[2 * c + 1]);
        }
      }

      // scores in log2 units, masked; accumulator rows are keys key + g and key + g + 8
      const float ks = scale.x, vs = scale.y;
      const bool partial = key + kStep > hi_all || key < lo_all;
      bool over = false;
#pragma unroll
      for (int n = 0; n < NG; ++n) {
#pragma unroll
        for (int c = 0; c < 4; ++c) s[n][c] *= fac[n][c & 1] * ks;
        if (partial) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int4 row = s_row[8 * n + 2 * t + (c & 1)];
            const int kk = key + g + 8 * (c >> 1);
            if (kk >= row.y || kk < row.z) s[n][c] = -INFINITY;
          }
        }
        over |= fmaxf(s[n][0], s[n][2]) > m[n][0] + kLazy || fmaxf(s[n][1], s[n][3]) > m[n][1] + kLazy;
      }
      if (__any_sync(~0u, over)) {                // raise the maxima and rescale
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x2 = fmaxf(s[n][c], s[n][c + 2]);
            x2 = fmaxf(x2, __shfl_xor_sync(~0u, x2, 4));
            x2 = fmaxf(x2, __shfl_xor_sync(~0u, x2, 8));
            x2 = fmaxf(x2, __shfl_xor_sync(~0u, x2, 16));
            if (x2 > m[n][c]) {
              const float r = ex2(m[n][c] - x2);
              m[n][c] = x2;
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
        const float ma = m[n][0] == -INFINITY ? 0.f : m[n][0], mb = m[n][1] == -INFINITY ? 0.f : m[n][1];
        const float e0 = ex2(s[n][0] - ma), e1 = ex2(s[n][1] - mb), e2 = ex2(s[n][2] - ma), e3 = ex2(s[n][3] - mb);
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
            const int4 row = s_row[8 * n + 2 * t + c];
            if (min(row.y, key + kStep) > max(row.z, key))
#pragma unroll
              for (int j = 0; j < D / 16; ++j) o[j][n][c] = o[j][n][c + 2] = vs;
          }
        continue;
      }
#pragma unroll
      for (int w = 0; w < C::VB / 4; ++w) {
        // bytes 4w .. 4w+3 of the lane's channels: rows g and g + 8 of tiles 2w and 2w + 1. Every other
        // word converts on the XU pipe, which is idle otherwise.
        uint32_t f0[4], f1[4];
        const bool xu = w & 1;
        const float vw_scale = xu ? vs * (1.f / 256.f) : vs;   // the accumulators hold out / 256
#pragma unroll
        for (int j = 0; j < 2; ++j) {             // keys 2t, 2t+1, then 2t+8, 2t+9
          const uint32_t lo = vw[2 * j][w], hi = vw[2 * j + 1][w];
          if (xu) {
            const uint32_t c01 = __byte_perm(lo, hi, 0x5140), c23 = __byte_perm(lo, hi, 0x7362);
            f0[2 * j] = half2_of_e4m3(c01), f0[2 * j + 1] = half2_of_e4m3(c01 >> 16);
            f1[2 * j] = half2_of_e4m3(c23), f1[2 * j + 1] = half2_of_e4m3(c23 >> 16);
          } else {
            const uint32_t c01 = __byte_perm(lo, hi, 0x5410), c23 = __byte_perm(lo, hi, 0x7632);
            f0[2 * j] = half2_of_even(c01), f0[2 * j + 1] = half2_of_odd(c01);
            f1[2 * j] = half2_of_even(c23), f1[2 * j + 1] = half2_of_odd(c23);
          }
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
          mma(x0, f0, p0[n], p1[n]);
          mma(x1, f1, p0[n], p1[n]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            o[2 * w][n][c] = fmaf(vw_scale, x0[c], o[2 * w][n][c]);
            o[2 * w + 1][n][c] = fmaf(vw_scale, x1[c], o[2 * w + 1][n][c]);
          }
        }
      }
    }
    cp_wait<0>();

    // ---- merge the warps in shared memory (over the ring) ----
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float y = l[n][c];
        y += __shfl_xor_sync(~0u, y, 4);
        y += __shfl_xor_sync(~0u, y, 8);
        y += __shfl_xor_sync(~0u, y, 16);
        const int r = 8 * n + 2 * t + c;
        if (g == 0) s_ml[warp * ROWS + r] = make_float2(m[n][c], y);
        float* dst = s_o + (warp * ROWS + r) * D + g * (D == 64 ? 8 : 16);
#pragma unroll
        for (int j = 0; j < D / 16; ++j)          // channels 4w + 2 (j & 1) of the lane, w = j / 2; 16 of each 128
          *reinterpret_cast<float2*>(dst + (j >> 3) * 128 + (j & 7) * 2) = make_float2(o[j][n][c], o[j][n][c + 2]);
      }
    __syncthreads();

    const bool whole = c0 == 0 && c1 == x.chunks;
    const int slot = 2 * blockIdx.x + (line == line0 ? 0 : 1);
    auto finish = [&](int r, int d4, float4 acc, float M, float L) {
      const int orow = s_row[r].w;
      const float inv = L > 0.f || L != L ? 256.f / L : 0.f;
      const __nv_bfloat162 lo2 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi2 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(a.out + int64_t(orow) * D + d4 * 4) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo2), *reinterpret_cast<const uint32_t*>(&hi2));
      if (a.lse && d4 == 0) a.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    };
    for (int idx = tid; idx < rows * (D / 4); idx += kThreads) {
      const int r = idx / (D / 4), d4 = idx % (D / 4);
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w * ROWS + r].x);
      const float Ms = M == -INFINITY ? 0.f : M;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = s_ml[w * ROWS + r];
        const float e = ex2(ml.x - Ms);
        const float4 y = *reinterpret_cast<const float4*>(s_o + (w * ROWS + r) * D + d4 * 4);
        L = fmaf(e, ml.y, L);
        acc.x = fmaf(e, y.x, acc.x), acc.y = fmaf(e, y.y, acc.y), acc.z = fmaf(e, y.z, acc.z), acc.w = fmaf(e, y.w, acc.w);
      }
      if (whole) {
        finish(r, d4, acc, M, L);
      } else {
        *reinterpret_cast<float4*>(a.part_o + (int64_t(slot) * ROWS + r) * D + d4 * 4) = acc;
        if (d4 == 0) *reinterpret_cast<float2*>(a.part_ml + (int64_t(slot) * ROWS + r) * 2) = make_float2(M, L);
      }
    }
    if (!whole) {
      // the last CTA of the item to arrive joins the parts
      const long long item0 = line - c0;
      const int fc = int(cta_of(item0)), lc = int(cta_of(item0 + x.chunks - 1));
      __syncthreads();
      if (tid == 0) {
        __threadfence();                          // this CTA's part before its arrival
        const uint32_t old = atomicAdd(a.counters + fc, 1u);
        s_last = old == uint32_t(lc - fc);
        if (s_last) a.counters[fc] = 0u;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        const int slot0 = 2 * fc + (start_of(fc) == item0 ? 0 : 1);
        for (int idx = tid; idx < rows * (D / 4); idx += kThreads) {
          const int r = idx / (D / 4), d4 = idx % (D / 4);
          float M = -INFINITY, L = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int c = fc; c <= lc; ++c) {
            const int64_t sl = c == fc ? slot0 : 2 * c;
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml + (sl * ROWS + r) * 2));
            const float4 y = __ldcg(reinterpret_cast<const float4*>(a.part_o + (sl * ROWS + r) * D + d4 * 4));
            const float Mn = fmaxf(M, ml.x), Ms = Mn == -INFINITY ? 0.f : Mn;
            const float e0 = ex2(M - Ms), e1 = ex2(ml.x - Ms);
            M = Mn;
            L = L * e0 + ml.y * e1;
            acc.x = acc.x * e0 + y.x * e1, acc.y = acc.y * e0 + y.y * e1;
            acc.z = acc.z * e0 + y.z * e1, acc.w = acc.w * e0 + y.w * e1;
          }
          finish(r, d4, acc, M, L);
        }
      }
    }
    __syncthreads();                              // the next item writes the rows and the ring
    line += c1 - c0;
    off += c1 - c0;
    if (off == unit_chunks) {
      ++unit;
      off = 0;
    }
  }
}

using Kernel = void (*)(FwdArgs);

template <int D, int NG>
void pick(Kernel& k, int& smem, int& ctas) {
  k = kv8_fwd_kernel<D, NG>;
  smem = Cfg<D, NG>::SMEM;
  ctas = Cfg<D, NG>::CTAS;
}

// head_dim 256: at most 16 rows (the accumulators of 32 would take every register)
bool kernel_of(int d, int ng, Kernel& k, int& smem, int& ctas) {
  if (d == 64) ng == 1 ? pick<64, 1>(k, smem, ctas) : ng == 2 ? pick<64, 2>(k, smem, ctas) : pick<64, 4>(k, smem, ctas);
  else if (d == 128) ng == 1 ? pick<128, 1>(k, smem, ctas) : ng == 2 ? pick<128, 2>(k, smem, ctas) : pick<128, 4>(k, smem, ctas);
  else ng == 1 ? pick<256, 1>(k, smem, ctas) : pick<256, 2>(k, smem, ctas);
  return k != nullptr;
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
  Kernel k = nullptr;
  int smem = 0, ctas = 0, sms = 0;
  kernel_of(pl->d, pl->ng, k, smem, ctas);
  cudaError_t e = cudaGetDevice(&pl->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, pl->device);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) {
    int fit = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, k, kThreads, smem);
    pl->grid = sms * std::max(1, std::min(fit, ctas));
  }
  const size_t tile = size_t(8) * pl->ng, slots = size_t(2) * pl->grid;
  const size_t bytes_o = slots * tile * pl->d * 4, bytes_ml = slots * tile * 8, bytes_c = size_t(pl->grid) * 4;
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
  Kernel k = nullptr;
  int smem = 0, ctas = 0;
  kernel_of(p->d, p->ng, k, smem, ctas);
  k<<<p->grid, kThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
