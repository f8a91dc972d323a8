// fm_paged.cu — attention of new tokens over the paged cache: the plan (units
// and CTA ranges), the kernel for few query rows a KV head, and the joining of
// partial results.
//
// O = softmax(scale Q K^T + M) V over the keys a query sees, by the online
// softmax (running maximum m, running sum l, O rescaled when m moves); a row
// that sees no key gives O = 0, LSE = -inf. Position p sees key j < kv_len iff
// (not causal or j <= p) and (no window W, or j > p - W, or j < sinks).
//
// few_kernel, one unit = 16 query rows of a KV head (a token's query heads of
// the group, then the next token's): bound by memory, each key and value byte
// is read once for all query heads of its group and 16 rows cost few
// operations, so the design is about loads in flight. A producer warp brings
// tiles of 64 keys in by TMA, page by page, into a ring of 96 KB a CTA (two
// CTAs an SM, 192 KB in flight an SM); four warps take 16 keys of a tile each,
// so every byte in shared memory is read once, and keep their own running
// (m, l, O) in registers (m16n8k16 products), joined at a segment's end. The
// tensor-memory path has nothing to offer here: its smallest tile is 64 rows.
// P goes into the second product as two bf16 terms (p and what its rounding
// left), so P's rounding adds nothing to O's own; the products are a small part
// of the time either way.
//
// e4m3 caches: e4m3 is exact in fp16, one conversion for two values, so the
// products run in fp16 on the stored values and the rows' power-of-two scales
// stay outside: a key's on its score, a value's in its weight, 2^(score +
// exponent - mo) with a running maximum mo of its own, so that the weight of
// the largest summand is near 1 whatever the rows' scales are. One fp16 term
// (2^-12 of a weight; weights below 2^-14 of the largest are off by 2^-25 of it
// at most) is finer than bf16's 2^-9. Measured at 32 sequences of 4K to 16K keys, 32 / 8 heads, d = 128: 258 us
// with the values widened to bf16 by integer operations (867 instructions for 16 keys).
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>
#include <cuda.h>
#include <cuda_bf16.h>
#include "fm_internal.h"
#include "paged.cuh"
#include "sm100.cuh"

namespace fm {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kLn2F = 0.69314718055994530942f;

// ------------------------------------------------------------------ the plan
struct PlanParams {
  PagedShape s;
  const int32_t* q_off;
  const int32_t* kv_len;
  PagedWork w;
  int* err;
};

constexpr int kPlanThreads = 1024;

template <typename V>
__device__ __forceinline__ V block_scan(V v, V* warp_sums) {  // inclusive
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const V x = __shfl_up_sync(kAll, v, m);
    if (lane >= m) v += x;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    V t = warp_sums[lane];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const V x = __shfl_up_sync(kAll, t, m);
      if (lane >= m) t += x;
    }
    warp_sums[lane] = t;
  }
  __syncthreads();
  if (warp > 0) v += warp_sums[warp - 1];
  return v;
}

// new tokens of sequence r: [s, e), kept inside [0, T] whatever q_off holds
__device__ __forceinline__ void span_of(const PlanParams& p, int r, int& s, int& e, bool& bad) {
  const int a = p.q_off[r], b = p.q_off[r + 1];
  s = min(max(a, 0), p.s.T);
  e = min(max(b, s), p.s.T);
  bad = a != s || b != e;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  __shared__ long long sums[32];
  __shared__ long long carry;
  const PagedShape& s = p.s;
  const int tid = threadIdx.x;
  grid_launch_dependents();
  bool bad = false;
  // units of each sequence
  if (tid == 0) {
    carry = 0;
    p.w.first[0] = 0;
  }
  __syncthreads();
  for (int r0 = 0; r0 < s.R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    long long n = 0;
    if (r < s.R) {
      int a, b;
      bool x;
      span_of(p, r, a, b, x);
      bad |= x;
      n = ((long long)(b - a) * s.G + s.step - 1) / s.step;
    }
    const long long in = block_scan(n, sums) + carry;
    if (r < s.R) p.w.first[r + 1] = (int)min(in, s.max_units);
    __syncthreads();
    if (tid == kPlanThreads - 1) carry = in;
    __syncthreads();
  }
  const int units = (int)min(carry, s.max_units);
  bad |= carry > s.max_units;  // spans that overlap
  __syncthreads();
  if (tid == 0) carry = 0;
  __syncthreads();
  // every unit's rows and key tiles, and the running sum of the work
  for (int u0 = 0; u0 < units; u0 += kPlanThreads) {
    const int u = u0 + tid;
    long long work = 0;
    if (u < units) {
      int lo = 0, hi = s.R - 1;  // last r with first[r] <= u
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.w.first[mid] <= u)
          lo = mid;
        else
          hi = mid - 1;
      }
      int a, b;
      bool x;
      span_of(p, lo, a, b, x);
      const int n = b - a;
      const int L0 = p.kv_len[lo];
      const int L = min(max(L0, 0), s.width * s.page);
      bad |= L0 != L;
      const long long row0 = (long long)(u - p.w.first[lo]) * s.step;
      PagedUnit q;
      q.r = lo;
      q.tok = a + (int)(row0 / s.G);
      q.g0 = (int)(row0 % s.G);
      q.nrows = (int)min((long long)s.step, (long long)n * s.G - row0);
      q.pos = L - n + (int)(row0 / s.G);
      q.kv_len = L;
      const int last = q.pos + (q.g0 + q.nrows - 1) / s.G;
      q.hi = s.causal ? min(max(last + 1, 0), L) : L;
      q.lo = s.window > 0 ? max(0, q.pos - s.window + 1) : 0;
      const int all = (q.hi + s.tile - 1) / s.tile;
      q.ns = s.window > 0 ? min((s.sinks + s.tile - 1) / s.tile, all) : 0;
      q.w0 = max(q.ns, min(q.lo / s.tile, all));
      q.ntiles = q.ns + max(0, all - q.w0);
      q.pad = 0;
      p.w.units[u] = q;
      work = (long long)max(q.ntiles, 1) * s.H_kv;
    }
    const long long in = block_scan(work, sums) + carry;
    if (u < units) p.w.sum[u] = in - work;
    __syncthreads();
    if (tid == kPlanThreads - 1) carry = in;
    __syncthreads();
  }
  const long long total = carry;
  if (tid == 0) p.w.sum[units] = total;
  __syncthreads();
  // each CTA's range: [c total / ctas, (c + 1) total / ctas)
  for (int c = tid; c < s.ctas; c += kPlanThreads) {
    const long long f = total * c / s.ctas, g = total * (c + 1) / s.ctas;
    PagedStart st = {0, 0, 0, (int)(g - f)};
    if (st.count > 0) {
      int lo = 0, hi = units - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.w.sum[mid] <= f)
          lo = mid;
        else
          hi = mid - 1;
      }
      const long long rem = f - p.w.sum[lo];
      const int nt = max(p.w.units[lo].ntiles, 1);
      st.u = lo;
      st.h = (int)(rem / nt);
      st.kt = (int)(rem - (long long)st.h * nt);
    }
    p.w.starts[c] = st;
  }
  if (bad) record_error(p.err, FM_DEV_ERR_RANGE);
}

// -------------------------------------------------------------- few query rows
constexpr int kFewThreads = 160;  // four computing warps and the producer
constexpr int kFewRows = 16;
constexpr int kTileKeys = 64;

template <int D, bool F8>
struct FewCfg {
  static constexpr int ES = F8 ? 1 : 2;
  static constexpr int ROW = D * ES < 128 ? D * ES : 128;  // bytes of a row inside a box
  static constexpr int BOXES = D * ES / ROW;
  static constexpr int BOX = kTileKeys * ROW;
  static constexpr int TILE = BOXES * BOX;  // K or V of one stage
  static constexpr int EXP = F8 ? 2 * kTileKeys : 0;
  static constexpr int STAGE = 2 * TILE + 0;
  static constexpr int STAGES = D == 256 ? (F8 ? 6 : 3) : D == 128 ? (F8 ? 6 : 3) : (F8 ? 8 : 6);
  static constexpr int PER_SM = D == 256 ? 1 : 2;
  static constexpr int MERGE_OFF = STAGES * STAGE;
  static constexpr int EXP_OFF = MERGE_OFF + kFewRows * D * 4;
  static constexpr int BAR_OFF = EXP_OFF + STAGES * EXP;
  static constexpr int ML_OFF = BAR_OFF + 2 * STAGES * 8;
  static constexpr int BYTES = ML_OFF + 4 * kFewRows * 2 * 4 + 16;
  static constexpr int SMEM = BYTES + 1024;
  static constexpr int KSTEPS = D / 16;
  static constexpr int CHUNKS = ROW / 64;         // 16-byte chunks a thread reads of a box's row
  static constexpr int SPC = F8 ? 4 : 2;          // k-steps of a chunk
};

struct FewParams {
  PagedShape s;
  PagedWork w;
  const char* q;
  int64_t q_st, q_sh;
  PagedOut out;
  const uint8_t* k_exp;
  const uint8_t* v_exp;
  const int32_t* table;
  float scale_log2;
  int* err;
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// four e4m3 values as two fp16 pairs (exact)
__device__ __forceinline__ void e4m3_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
// 2^(e - 127), NaN for e = 255
__device__ __forceinline__ float scale_of(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7fc00000u : e == 0u ? 0x00400000u : e << 23);
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

template <int D, bool F8>
__global__ void __launch_bounds__(kFewThreads, FewCfg<D, F8>::PER_SM)
    few_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const FewParams p) {
  using C = FewCfg<D, F8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  float* ml = reinterpret_cast<float*>(smem + C::ML_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::ML_OFF + 4 * kFewRows * 2 * 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  FM_DEBUG_BEGIN();
  if (threadIdx.x == 0) {
    *abort_flag = timeout_pending(p.err) ? 1 : 0;
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    fence_mbar_init();
  }
  if (warp == 4 && lane == 0) {
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  const PagedStart st = p.w.starts[blockIdx.x];
  const int G = p.s.G;
  bool ok = *abort_flag == 0;
  PagedWalk walk(p.w.units, st, p.s.H_kv);
  uint32_t it = 0;  // tiles so far

  if (warp == 4) {
    // ------------------------------------------------------------- producer
    const int P = p.s.page, rows = min(P, kTileKeys), per = kTileKeys / rows;  // box rows, boxes along the keys
    const int zmax = p.s.n_pages * p.s.H_kv;
    PageWindow pages;
    for (; walk.more() && ok; walk.next()) {
      const PagedUnit& u = walk.u;
      pages.reset(p.table, u.r, p.s.width);
      for (int j = 0; j < walk.n && ok; ++j, ++it) {
        const int key0 = tile_of(u, walk.kt + j) * kTileKeys;
        const int pg0 = key0 / P;
        pages.hold(pg0, per, lane);
        const int stage = it % C::STAGES;
        ok = __all_sync(kAll, mbar_wait(&empty[stage], ((it / C::STAGES) & 1u) ^ 1u, abort_flag, p.err));
        if (!ok) break;
        // boxes whose first key is held: the rest of the tile is never read
        const int boxes = min(per, (u.kv_len - key0 + rows - 1) / rows);
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], boxes * rows * (2 * D * C::ES + (F8 ? 2 : 0)));
        __syncwarp();
        constexpr int OPS = 2 * C::BOXES + (F8 ? 2 : 0);  // copies of one page's part
        for (int i0 = 0; i0 < boxes * OPS; i0 += 32) {
          const int i = i0 + lane;
          const int b = min(i / OPS, boxes - 1), op = i % OPS;
          const int pg = __shfl_sync(kAll, pages.held, pg0 + b - pages.base);
          if (i >= boxes * OPS) continue;
          const bool good = pg >= 0 && pg < p.s.n_pages;
          if (!good) record_error(p.err, FM_DEV_ERR_RANGE);
          const int z = good ? pg * p.s.H_kv + walk.h : zmax;  // zmax: out of range, reads as zero
          const int y = key0 - pg0 * P;
          uint8_t* at = smem + stage * C::STAGE + b * rows * C::ROW;
          if (op < 2 * C::BOXES) {
            const int v = op >= C::BOXES, x = op - v * C::BOXES;
            tma_load_3d(at + v * C::TILE + x * C::BOX, v ? &tv : &tk, &full[stage], x * (C::ROW / C::ES), y, z);
          } else {
            const int v = op - 2 * C::BOXES;
            bulk_load(smem + C::EXP_OFF + stage * C::EXP + v * kTileKeys + b * rows,
                      (v ? p.v_exp : p.k_exp) + (int64_t)(good ? z : walk.h) * P + y, rows, &full[stage]);
          }
        }
      }
    }
    if (!ok) {
      // leave with no copy in flight: every stage handed out has landed, or a second bound passed
      volatile int none = 0;
      for (uint32_t s = it > C::STAGES ? it - C::STAGES : 0; s < it; ++s)
        mbar_wait(&full[s % C::STAGES], (s / C::STAGES) & 1u, &none, p.err);
    }
  } else {
    // ------------------------------------------------------------ computing
    const int g = lane >> 2, t = lane & 3;
    float* merge = reinterpret_cast<float*>(smem + C::MERGE_OFF);
    const float sl2 = p.scale_log2;
    for (; walk.more(); walk.next()) {
      const PagedUnit& u = walk.u;
      // this thread's rows g and g + 8: their positions (-1: no such row), their Q
      int pos[2];
      uint32_t qf[C::KSTEPS][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = g + 8 * i, x = u.g0 + row;
        const bool live = row < u.nrows;
        pos[i] = live ? (p.s.causal ? u.pos + x / G : u.kv_len - 1) : -1;
        const char* src = p.q + 2 * ((int64_t)(u.tok + x / G) * p.q_st + (int64_t)(walk.h * G + x % G) * p.q_sh);
#pragma unroll
        for (int b = 0; b < C::BOXES; ++b)
#pragma unroll
          for (int c = 0; c < C::CHUNKS; ++c) {
            // the elements of the chunk that this thread reads of a key's row
            const int e0 = (b * C::ROW + (C::CHUNKS * t + c) * 16) / C::ES;
#pragma unroll
            for (int x4 = 0; x4 < C::SPC / 2; ++x4) {
              uint4 v = make_uint4(0, 0, 0, 0);
              if (live && ok && walk.n > 0) v = *reinterpret_cast<const uint4*>(src + 2 * (e0 + 8 * x4));
              const int k = (b * C::CHUNKS + c) * C::SPC + 2 * x4;
              qf[k][i] = v.x;
              qf[k][2 + i] = v.y;
              qf[k + 1][i] = v.z;
              qf[k + 1][2 + i] = v.w;
            }
          }
      }
      const int plo = u.pos + u.g0 / G, phi = u.pos + (u.g0 + u.nrows - 1) / G;  // the unit's first and last position
      float sc[2] = {sl2, sl2};  // per row: scores to log2 units
      if constexpr (F8) {
        // Q in fp16, each row times the power of two that puts its largest value at
        // the top of fp16's range: values down to 2^-29 of it keep all their bits
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < C::KSTEPS; ++k)
            top = __vmaxu2(top, __vmaxu2(qf[k][i] & 0x7fff7fffu, qf[k][2 + i] & 0x7fff7fffu));
          top = __vmaxu2(top, __shfl_xor_sync(kAll, top, 1));
          top = __vmaxu2(top, __shfl_xor_sync(kAll, top, 2));
          const int E = (int)(max(top & 0xffffu, top >> 16) >> 7);
          // 2^(142 - E), kept finite; a row of zeros, infinities or NaN stays as it is
          const int up = (E == 0 || E == 255) ? 0 : min(142 - E, 126);
          const float f = __uint_as_float((uint32_t)(127 + up) << 23);
          sc[i] = sl2 * __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
          for (int k = 0; k < C::KSTEPS; ++k)
#pragma unroll
            for (int x = i; x < 4; x += 2)
              qf[k][x] = pack_f16x2(__uint_as_float(qf[k][x] << 16) * f, __uint_as_float(qf[k][x] & 0xffff0000u) * f);
        }
      }
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      float mo[2] = {-INFINITY, -INFINITY};  // e4m3: the running maximum of score + exponent of the value's scale
      float o[D / 8][4];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

      for (int j = 0; j < walk.n; ++j, ++it) {
        const int stage = it % C::STAGES;
        if (ok) ok = __all_sync(kAll, mbar_wait(&full[stage], (it / C::STAGES) & 1u, abort_flag, p.err));
        const int key0 = tile_of(u, walk.kt + j) * kTileKeys + warp * 16;
        // keys of this warp that some row sees: below hi, and from lo on or sinks
        if (ok && key0 < u.hi && (key0 + 16 > u.lo || key0 < p.s.sinks)) {
          const uint32_t kb = smem_u32(smem + stage * C::STAGE), vb = kb + C::TILE;
          const uint32_t eb = smem_u32(smem + C::EXP_OFF + stage * C::EXP) + warp * 16;
          float s[2][4];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
            const int row = warp * 16 + 8 * n + g;
#pragma unroll
            for (int b = 0; b < C::BOXES; ++b)
#pragma unroll
              for (int c = 0; c < C::CHUNKS; ++c) {
                const uint4 v = lds128(kb + b * C::BOX + in_box<C::ROW>(row, C::CHUNKS * t + c));
                const int k = (b * C::CHUNKS + c) * C::SPC;
                if constexpr (F8) {
                  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    uint32_t b0, b1;
                    e4m3_to_f16(w[x], b0, b1);
                    mma16816_f16(s[n], qf[k + x], b0, b1);
                  }
                } else {
                  mma16816(s[n], qf[k], v.x, v.y);
                  mma16816(s[n], qf[k + 1], v.z, v.w);
                }
              }
          }
          float ve[2][2];  // e4m3: the exponents of the values' scales
          if constexpr (F8) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const uint32_t ek = lds16(eb + 8 * n + 2 * t), ev = lds16(eb + kTileKeys + 8 * n + 2 * t);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float f = scale_of((ek >> (8 * x)) & 255u);
                s[n][x] *= f * sc[0];
                s[n][2 + x] *= f * sc[1];
                const uint32_t e = (ev >> (8 * x)) & 255u;
                ve[n][x] = e == 255u ? NAN : (float)((int)e - 127);
              }
            }
          } else {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int x = 0; x < 4; ++x) s[n][x] *= sl2;
          }
          // masked scores: a tile whose 16 keys all rows see is left as it is
          const bool part = key0 + 16 > u.hi || (p.s.causal && key0 + 15 > plo) ||
                            (p.s.window > 0 && key0 <= phi - p.s.window);
          if (part) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int key = key0 + 8 * n + 2 * t + (x & 1), ps = pos[x >> 1];
                const bool see = key <= ps && key < u.kv_len &&
                                 (p.s.window == 0 || key > ps - p.s.window || key < p.s.sinks);
                s[n][x] = see ? s[n][x] : -INFINITY;
              }
          }
          // a running maximum moves only when it is passed by more than 8 (weights stay below 2^8)
          float f[2];
          bool moved = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
            x = fmaxf(x, __shfl_xor_sync(kAll, x, 1));
            x = fmaxf(x, __shfl_xor_sync(kAll, x, 2));
            f[i] = 1.f;
            if (x > m[i] + 8.f) {
              const float y = ex2_approx(m[i] - x);
              l[i] *= y;
              m[i] = x;
              if (!F8) {
                f[i] = y;
                moved = true;
              }
            }
            if constexpr (F8) {
              float z = fmaxf(fmaxf(s[0][2 * i] + ve[0][0], s[0][2 * i + 1] + ve[0][1]),
                              fmaxf(s[1][2 * i] + ve[1][0], s[1][2 * i + 1] + ve[1][1]));
              z = fmaxf(z, __shfl_xor_sync(kAll, z, 1));
              z = fmaxf(z, __shfl_xor_sync(kAll, z, 2));
              if (z > mo[i] + 8.f) {
                f[i] = ex2_approx(mo[i] - z);
                mo[i] = z;
                moved = true;
              }
            }
          }
          if (__any_sync(kAll, moved)) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              o[i][0] *= f[0];
              o[i][1] *= f[0];
              o[i][2] *= f[1];
              o[i][3] *= f[1];
            }
          }
          // weights: bf16 in two terms (p and what its rounding left), fp16 in one
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float base = m[i] == -INFINITY ? 0.f : m[i];
              const float a = ex2_approx(s[n][2 * i] - base), b = ex2_approx(s[n][2 * i + 1] - base);
              l[i] += a + b;
              if constexpr (F8) {
                const float bo = mo[i] == -INFINITY ? 0.f : mo[i];
                // a masked score stays masked whatever its key's exponent byte holds
                const float x = s[n][2 * i] == -INFINITY ? 0.f : ex2_approx(s[n][2 * i] + (ve[n][0] - bo));
                const float y = s[n][2 * i + 1] == -INFINITY ? 0.f : ex2_approx(s[n][2 * i + 1] + (ve[n][1] - bo));
                hi[2 * n + i] = pack_f16x2(x, y);
              } else {
                const uint32_t h = pack_bf16x2(a, b);
                hi[2 * n + i] = h;
                lo[2 * n + i] = pack_bf16x2(a - __uint_as_float(h << 16), b - __uint_as_float(h & 0xffff0000u));
              }
            }
          auto product = [&](auto masked) {
            // values of keys no row sees (past the sequence's end: anything may lie there) count as zero
            uint32_t vz[2] = {0xffffffffu, 0xffffffffu};
            if constexpr (masked.value) {
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const int key = key0 + 8 * n + 2 * t + x;
                  if (!(key < u.hi && (key >= u.lo || key < p.s.sinks))) vz[n] &= x ? 0x0000ffffu : 0xffff0000u;
                }
            }
            if constexpr (F8) {
              const int r0 = warp * 16 + 2 * t;
#pragma unroll
              for (int cg = 0; cg < D / 32; ++cg) {
                // four columns 32 cg + 4 g + i of keys 2t, 2t + 1, 2t + 8, 2t + 9
                const int box = cg / (C::ROW / 32), ch = (cg % (C::ROW / 32)) * 2 + (g >> 2);
                uint32_t w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  w[x] = lds32(vb + box * C::BOX + in_box<C::ROW>(r0 + (x & 1) + 8 * (x >> 1), ch) + 4 * (g & 3));
                uint32_t b0[4], b1[4];
                e4m3_to_f16(__byte_perm(w[0], w[1], 0x5140), b0[0], b0[1]);
                e4m3_to_f16(__byte_perm(w[0], w[1], 0x7362), b0[2], b0[3]);
                e4m3_to_f16(__byte_perm(w[2], w[3], 0x5140), b1[0], b1[1]);
                e4m3_to_f16(__byte_perm(w[2], w[3], 0x7362), b1[2], b1[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) mma16816_f16(o[4 * cg + i], hi, b0[i] & vz[0], b1[i] & vz[1]);
              }
            } else {
#pragma unroll
              for (int c = 0; c < D / 8; c += 2) {
                uint32_t r[4];
                const int ch = c + (lane >> 4);
                ldmatrix4_trans(vb + (ch >> 3) * C::BOX + in_box<128>(warp * 16 + (lane & 15), ch & 7), r);
                mma16816(o[c], hi, r[0] & vz[0], r[1] & vz[1]);
                mma16816(o[c + 1], hi, r[2] & vz[0], r[3] & vz[1]);
                mma16816(o[c], lo, r[0] & vz[0], r[1] & vz[1]);
                mma16816(o[c + 1], lo, r[2] & vz[0], r[3] & vz[1]);
              }
            }
          };
          if (part)
            product(std::true_type{});
          else
            product(std::false_type{});
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&empty[stage]);
      }

      // join the four warps' (m, l, O): a common maximum, then the sums in warp order
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (F8) {
          // O in units of l's: 2^mo of its scores-and-exponents to 2^m of the scores
          const float y = m[i] == -INFINITY ? 0.f : ex2_approx(mo[i] - m[i]);
#pragma unroll
          for (int x = 0; x < D / 8; ++x) {
            o[x][2 * i] *= y;
            o[x][2 * i + 1] *= y;
          }
        }
        l[i] += __shfl_xor_sync(kAll, l[i], 1);
        l[i] += __shfl_xor_sync(kAll, l[i], 2);
        if (t == 0) {
          ml[(warp * kFewRows + g + 8 * i) * 2] = m[i];
          ml[(warp * kFewRows + g + 8 * i) * 2 + 1] = l[i];
        }
      }
      named_bar_sync(1, 128);
      float top[2], sum[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = -INFINITY;
        for (int w = 0; w < 4; ++w) top[i] = fmaxf(top[i], ml[(w * kFewRows + g + 8 * i) * 2]);
        sum[i] = 0.f;
        const float base = top[i] == -INFINITY ? 0.f : top[i];
        for (int w = 0; w < 4; ++w)
          sum[i] += ex2_approx(ml[(w * kFewRows + g + 8 * i) * 2] - base) * ml[(w * kFewRows + g + 8 * i) * 2 + 1];
        const float f = ex2_approx(m[i] - base);
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
          o[x][2 * i] *= f;
          o[x][2 * i + 1] *= f;
        }
      }
      for (int w = 0; w < 4; ++w) {
        if (warp == w) {
#pragma unroll
          for (int x = 0; x < D / 8; ++x) {
            float4* at = reinterpret_cast<float4*>(merge) + x * 32 + lane;
            if (w > 0) {
              const float4 v = *at;
              o[x][0] += v.x;
              o[x][1] += v.y;
              o[x][2] += v.z;
              o[x][3] += v.w;
            }
            if (w < 3) *at = make_float4(o[x][0], o[x][1], o[x][2], o[x][3]);
          }
        }
        named_bar_sync(1, 128);
      }
      if (warp == 3 && ok) {
        const bool whole = walk.whole();
        float* part = p.w.part + p.w.part_floats * (2 * (size_t)blockIdx.x + walk.slot());
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = g + 8 * i, x = u.g0 + row;
          if (row >= u.nrows) continue;
          const int64_t tok = u.tok + x / G;
          const int head = walk.h * G + x % G;
          if (whole) {
            const float inv = sum[i] > 0.f ? 1.f / sum[i] : (sum[i] == 0.f ? 0.f : sum[i]);
            char* dst = p.out.o + 2 * (tok * p.out.st + head * p.out.sh);
            if constexpr (F8) {
#pragma unroll
              for (int cg = 0; cg < D / 32; ++cg) {
                uint32_t v[4];
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                  for (int z = 0; z < 2; ++z)
                    v[2 * y + z] = pack_bf16x2(o[4 * cg + 2 * z][2 * i + y] * inv, o[4 * cg + 2 * z + 1][2 * i + y] * inv);
                *reinterpret_cast<uint4*>(dst + 2 * (32 * cg + 8 * t)) = make_uint4(v[0], v[1], v[2], v[3]);
              }
            } else {
#pragma unroll
              for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint32_t*>(dst + 2 * (8 * c + 2 * t)) =
                    pack_bf16x2(o[c][2 * i] * inv, o[c][2 * i + 1] * inv);
            }
            if (t == 0)
              p.out.lse[tok * p.out.H_q + head] = sum[i] == 0.f ? -INFINITY : top[i] * kLn2F + logf(sum[i]);
          } else {
            float* dst = part + (size_t)row * D;
            if constexpr (F8) {
#pragma unroll
              for (int cg = 0; cg < D / 32; ++cg)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  *reinterpret_cast<float4*>(dst + 32 * cg + 8 * t + 4 * y) =
                      make_float4(o[4 * cg][2 * i + y], o[4 * cg + 1][2 * i + y], o[4 * cg + 2][2 * i + y],
                                  o[4 * cg + 3][2 * i + y]);
            } else {
#pragma unroll
              for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<float2*>(dst + 8 * c + 2 * t) = make_float2(o[c][2 * i], o[c][2 * i + 1]);
            }
            if (t == 0) {
              part[(size_t)kFewRows * D + 2 * row] = top[i];
              part[(size_t)kFewRows * D + 2 * row + 1] = sum[i];
            }
          }
        }
      }
    }
  }
  __syncthreads();
  FM_DEBUG_END(p.err);
}

// ------------------------------------------------------------------- joining
struct JoinParams {
  PagedWork w;
  PagedOut out;
  int ctas, G, rows;  // rows of a slot
};

// Block (c, y): if CTA c's range begins inside a unit that no earlier CTA's
// range begins inside of, the unit's pieces are joined, 8 rows a block.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const JoinParams p) {
  grid_dependency_wait();
  const int c = blockIdx.x + 1;
  const PagedStart st = p.w.starts[c];
  if (st.count <= 0 || st.kt == 0) return;
  // the CTA before it that has work holds the piece before this one
  int b = c - 1;
  while (b > 0 && p.w.starts[b].count <= 0) --b;
  const PagedStart before = p.w.starts[b];
  if (before.u == st.u && before.h == st.h && before.kt > 0) return;
  const PagedUnit u = p.w.units[st.u];
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= u.nrows) return;
  const float* first = p.w.part + p.w.part_floats * (2 * (size_t)b + 1);
  const size_t ml = (size_t)p.rows * D + 2 * row;
  int end = c;  // one past the unit's last CTA
  while (end < p.ctas) {
    const PagedStart x = p.w.starts[end];
    if (x.count > 0 && !(x.u == st.u && x.h == st.h)) break;
    ++end;
  }
  auto slot = [&](int i) { return i < c ? first : p.w.part + p.w.part_floats * (2 * (size_t)i); };
  float top = -INFINITY;
  for (int i = c - 1 + lane; i < end; i += 32)
    if (i < c || p.w.starts[i].count > 0) top = fmaxf(top, slot(i)[ml]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, x));
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f, acc[D / 32];
#pragma unroll
  for (int x = 0; x < D / 32; ++x) acc[x] = 0.f;
  for (int i = c - 1; i < end; ++i) {
    if (i >= c && p.w.starts[i].count <= 0) continue;
    const float* s = slot(i);
    const float f = ex2_approx(s[ml] - base);
    sum += f * s[ml + 1];
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
      const float2 v = *reinterpret_cast<const float2*>(s + (size_t)row * D + 64 * x + 2 * lane);
      acc[2 * x] += f * v.x;
      acc[2 * x + 1] += f * v.y;
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  const int x0 = u.g0 + row;
  const int64_t tok = u.tok + x0 / p.G;
  const int head = st.h * p.G + x0 % p.G;
  char* dst = p.out.o + 2 * (tok * p.out.st + head * p.out.sh);
#pragma unroll
  for (int x = 0; x < D / 64; ++x)
    *reinterpret_cast<uint32_t*>(dst + 2 * (64 * x + 2 * lane)) = pack_bf16x2(acc[2 * x] * inv, acc[2 * x + 1] * inv);
  if (lane == 0) p.out.lse[tok * p.out.H_q + head] = sum == 0.f ? -INFINITY : top * kLn2F + logf(sum);
}

template <int D>
cudaError_t launch_join(const PagedShape& s, const PagedWork& w, const PagedOut& out, int rows, cudaStream_t st) {
  JoinParams j{w, out, s.ctas, s.G, rows};
  const dim3 grid((unsigned)(s.ctas - 1), (unsigned)((rows + 7) / 8));
  if (s.ctas < 2) return cudaSuccess;
  count_launches(1);
  return launch_dependent(join_kernel<D>, grid, 256, 0, st, j);
}

template <int D, bool F8>
cudaError_t launch_few(const PagedShape& s, const PagedWork& w, const fm_kv_cache& c, const fm_paged_batch& b,
                       const fm_rows& q, const PagedOut& out, float scale, cudaStream_t st, int* err) {
  using C = FewCfg<D, F8>;
  static_assert(C::PER_SM * (C::SMEM + 1024) <= 233472, "few_kernel: shared memory of an SM");
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(few_kernel<D, F8>), C::SMEM, ready);
  if (e != cudaSuccess) return e;
  CUtensorMap tk, tv;
  const int rows = std::min(s.page, kTileKeys);
  if (!make_tmap_pages(&tk, c.k, c, rows, C::ROW) || !make_tmap_pages(&tv, c.v, c, rows, C::ROW))
    return cudaErrorInvalidValue;
  FewParams p{s, w, static_cast<const char*>(q.ptr), q.st, q.sh, out, c.k_exp, c.v_exp, b.page_table,
              scale * 1.4426950408889634f, err};
  count_launches(1);
  return launch_dependent(few_kernel<D, F8>, dim3((unsigned)s.ctas), kFewThreads, C::SMEM, st, tk, tv, p);
}

// Which kernel: chunk_kernel's tiles of 128 rows once the sequences have more
// than 16 rows a KV head on average (few_kernel would read the keys again for
// every 16), few_kernel otherwise, and where the other has no form: d = 256,
// groups of more than 128 heads, queries that are broadcast (a TMA map has no
// stride of zero).
bool use_chunk(const fm_kv_cache& c, const fm_paged_batch& b, int T, int H_q, const fm_rows* q) {
  const int G = H_q / c.H_kv;
  if (c.d == 256 || G > 128) return false;
  if (q && ((T > 1 && q->st <= 0) || (H_q > 1 && q->sh <= 0))) return false;
  return (long long)T * G > 16ll * b.R;
}

PagedShape shape_of(const fm_kv_cache& c, const fm_paged_batch& b, int T, int H_q, int causal, int window, int sinks,
                    bool chunk) {
  PagedShape s = {};
  s.T = T;
  s.R = b.R;
  s.H_q = H_q;
  s.H_kv = c.H_kv;
  s.G = H_q / c.H_kv;
  s.d = c.d;
  s.width = b.width;
  s.page = c.page_size;
  s.n_pages = c.n_pages;
  s.causal = causal;
  // positions stay below 2^30: larger windows and sinks hide nothing more
  s.window = std::min(window, 1 << 30);
  s.sinks = window > 0 ? std::min(sinks, 1 << 30) : 0;
  s.step = chunk ? 2 * (128 / s.G) * s.G : kFewRows;
  s.tile = chunk ? 128 : kTileKeys;
  s.ctas = sm_count() * (chunk || c.d == 256 ? 1 : 2);
  s.max_units = ((long long)T * s.G + s.step - 1) / s.step + b.R;
  return s;
}

}  // namespace

size_t paged_ws_bytes(const fm_kv_cache& c, const fm_paged_batch& b, int T, int H_q) {
  // of either kernel: which one runs goes by the queries' strides too
  size_t bytes = paged_work(shape_of(c, b, T, H_q, 1, 0, 0, false), kFewRows, nullptr).bytes;
  if (use_chunk(c, b, T, H_q, nullptr))
    bytes = std::max(bytes, paged_work(shape_of(c, b, T, H_q, 1, 0, 0, true), kChunkRows, nullptr).bytes);
  return bytes;
}

cudaError_t launch_paged(const fm_kv_cache& c, const fm_paged_batch& b, int T, int H_q, const fm_rows& q,
                         const fm_rows& o, float* lse, float scale, int causal, int window, int sinks, void* ws,
                         cudaStream_t st, int* err) {
  const bool chunk = use_chunk(c, b, T, H_q, &q);
  const int rows = chunk ? kChunkRows : kFewRows;
  const PagedShape s = shape_of(c, b, T, H_q, causal, window, sinks, chunk);
  const PagedWork w = paged_work(s, rows, ws);
  const PagedOut out{static_cast<char*>(o.ptr), o.st, o.sh, lse, H_q};
  PlanParams pp{s, b.q_off, b.kv_len, w, err};
  plan_kernel<<<1, kPlanThreads, 0, st>>>(pp);
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const bool f8 = c.k_exp != nullptr;
  if (chunk)
    e = launch_paged_chunk(s, w, c, b, q, out, scale, st, err);
  else if (c.d == 64)
    e = f8 ? launch_few<64, true>(s, w, c, b, q, out, scale, st, err)
           : launch_few<64, false>(s, w, c, b, q, out, scale, st, err);
  else if (c.d == 128)
    e = f8 ? launch_few<128, true>(s, w, c, b, q, out, scale, st, err)
           : launch_few<128, false>(s, w, c, b, q, out, scale, st, err);
  else
    e = f8 ? launch_few<256, true>(s, w, c, b, q, out, scale, st, err)
           : launch_few<256, false>(s, w, c, b, q, out, scale, st, err);
  if (e != cudaSuccess) return e;
  return c.d == 64    ? launch_join<64>(s, w, out, rows, st)
         : c.d == 128 ? launch_join<128>(s, w, out, rows, st)
                      : launch_join<256>(s, w, out, rows, st);
}

}  // namespace fm
