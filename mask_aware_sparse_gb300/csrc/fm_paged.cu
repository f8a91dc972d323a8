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
// operations, so the design is about loads in flight. Each of a CTA's warps
// takes its share of the segment's key tiles (32 keys) and brings them in itself,
// 16 bytes a lane and copy, into a ring of its own (keys and values as entries of
// their own; about 200 KB an SM), with its own running (m, l, O) in
// registers (m16n8k16 products): every byte in shared memory is read once, and
// no warp waits for another before a segment's end, where they are joined.
// Measured against TMA boxes issued by a producer warp (e4m3, pages of 64, loads
// alone, nothing computed): boxes of 32 rows and the exponents' own bulk copies
// reach 3.9 TB/s; the copies also cost the same for pages of any size, and fill
// with zeros where a page ends. The tensor-memory path has nothing to offer
// here: its smallest tile is 64 rows.
// P goes into the second product as two bf16 terms (p and what its rounding
// left), so P's rounding adds nothing to O's own; the products are a small part
// of the time either way.
//
// e4m3 caches: e4m3 is exact in fp16, one conversion for two values, so the
// products run in fp16 on the stored values and the rows' power-of-two scales
// stay outside: a key's on its score, a value's in its weight, 2^(score +
// exponent - mo) with a running maximum of its own less 7 as mo, so that the weight
// of the largest summand lies near the top of fp16's range (2^7 to 2^15) whatever the
// rows' scales are. One fp16 term (2^-11 of a weight; weights below 2^-21 of the
// largest are off by 2^-32 of it at most) is finer than bf16's 2^-8. Measured at 32 ragged sequences of up to 16384
// keys, 32 / 8 heads, d = 128 (bytes alone 99 us): 112 us; 261 with the values widened
// to bf16 by integer operations, whose instructions bounded it.
#include <algorithm>
#include <cfloat>
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

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  __shared__ long long sums[32];
  __shared__ long long carry;
  const PagedShape& s = p.s;
  const int tid = threadIdx.x;
  grid_dependency_wait();
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
      int a, k, L;
      bad |= sequence_at(s, p.q_off, p.kv_len, r, a, k, L);
      n = ((long long)k * s.G + s.step - 1) / s.step;
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
      int a, n, L;
      sequence_at(s, p.q_off, p.kv_len, lo, a, n, L);
      const PagedUnit q = unit_at(s, lo, a, n, L, u - p.w.first[lo]);
      p.w.units[u] = q;
      work = (long long)max(q.ntiles, 1) * s.H_kv;
    }
    const long long in = block_scan(work, sums) + carry;
    if (u < units) p.w.sum[u] = in - work;
    __syncthreads();
    if (tid == kPlanThreads - 1) carry = in;
    __syncthreads();
  }
  const PagedDivision<long long> div(s, carry, units);
  const long long ex = div.extra * s.H_kv;
  for (int c = tid; c < s.ctas; c += kPlanThreads) {
    PagedStart st = {};
    if (c < div.used && div.total > 0) {
      const long long f = div.begin(c);
      int lo = 0, hi = units - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.w.sum[mid] + mid * ex <= f)
          lo = mid;
        else
          hi = mid - 1;
      }
      const long long from = p.w.sum[lo] + lo * ex;
      st.unit = p.w.units[lo];
      const long long nt = max(st.unit.ntiles, 1);
      st.u = lo;
      st.h = (int)((f - from) / (nt + div.extra));
      div.set(st, c, from + st.h * (nt + div.extra), nt);
    }
    p.w.starts[c] = st;
  }
  if (bad) record_error(p.err, FM_DEV_ERR_RANGE);
}

// -------------------------------------------------------------- few query rows
constexpr int kFewRows = 16;
constexpr int kTileKeys = 32;
constexpr float kTopBits = 7.f;  // e4m3: weights go up to 2^(7 + 8)

constexpr int few_warps(int d, bool f8) { return d == 256 && f8 ? 8 : 4; }
constexpr int few_ctas(int d, bool f8) { return d == 256 ? 1 : d == 64 && f8 ? 3 : 2; }

template <int D, bool F8>
struct FewCfg {
  static constexpr int ES = F8 ? 1 : 2;
  static constexpr int RB = D * ES;                  // bytes of a row
  static constexpr int ROW = RB < 128 ? RB : 128;    // of them in one swizzled box
  static constexpr int BOXES = RB / ROW;
  static constexpr int BOX = kTileKeys * ROW;
  static constexpr int TILE = BOXES * BOX;           // one ring entry: a tile's keys, or its values
  static constexpr int EXP = F8 ? kTileKeys : 0;
  // Warps, CTAs an SM and entries of a warp's ring: what fills shared memory with
  // loads in flight. e4m3 rows are short for the work on each, so more warps help
  // where registers allow: d = 64 three CTAs (step of 32 sequences 77 us, with two
  // 91), d = 256 eight warps (271 us, with four 355).
  static constexpr int WARPS = few_warps(D, F8), THREADS = 32 * WARPS;
  static constexpr int PER_SM = few_ctas(D, F8);
  static constexpr int RING = D == 256 ? 3 : D == 64 ? (F8 ? 8 : 6) : (F8 ? 6 : 3);
  static constexpr int ENTRIES = WARPS * RING;
  static constexpr int EXP_OFF = ENTRIES * TILE;
  static constexpr int ML_OFF = EXP_OFF + ENTRIES * EXP;
  static constexpr int SMEM = ML_OFF + WARPS * kFewRows * 16 + 1024;
  // entries that hold a warp's O at a segment's end, and those free for the next segment's first loads
  static constexpr int MERGE = (kFewRows * D * 4 + TILE - 1) / TILE, AHEAD = RING - MERGE;
  static_assert(AHEAD >= 1, "the ring is more than what the join needs");
  static constexpr int KSTEPS = D / 16;
  static constexpr int CHUNKS = ROW / 64;  // 16-byte chunks a thread reads of a box's row
  static constexpr int SPC = F8 ? 4 : 2;   // k-steps of a chunk
  // loading: CPR lanes a row, RPI rows an instruction
  static constexpr int CPR = RB / 16, RPI = 32 / CPR, LOADS = kTileKeys / RPI;
};

struct FewParams {
  PagedShape s;
  PagedWork w;
  const char* q;
  int64_t q_st, q_sh;
  PagedOut out;
  const char* kv[2];
  const uint8_t* exps[2];
  const int32_t* q_off;
  const int32_t* kv_len;
  const int32_t* table;
  float scale_log2;
  int* err;
};

// 16 bytes from global to shared memory without a register between; zeros where !live
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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
// 2^(e - 127), and e - 127 (bytes 1 .. 254: rows without a scale, 255, hold NaN already)
__device__ __forceinline__ float scale_of(uint32_t e) { return __uint_as_float(e << 23); }
__device__ __forceinline__ float exponent_of(uint32_t e) { return __uint_as_float(0x4b000000u | e) - 8388735.f; }
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

template <int D, bool F8>
__global__ void __launch_bounds__(FewCfg<D, F8>::THREADS, FewCfg<D, F8>::PER_SM) few_kernel(const FewParams p) {
  using C = FewCfg<D, F8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float4* ml = reinterpret_cast<float4*>(smem + C::ML_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ PagedStart start;
  __shared__ int4 seq[kLocalSeqs];
  __shared__ uint16_t first[kLocalSeqs + 1], order[kWholeUnits];
  grid_dependency_wait();
  grid_launch_dependents();
  if (p.s.whole) {
    plan_whole(p.s, p.q_off, p.kv_len, seq, first, order, reinterpret_cast<uint16_t*>(smem), &start, p.err);
  } else if (p.s.local) {
    plan_locally(p.s, p.q_off, p.kv_len, seq, reinterpret_cast<unsigned*>(smem), &start, p.err);
    if (threadIdx.x == 0) p.w.starts[blockIdx.x] = start;  // for join_kernel
  } else {
    if (threadIdx.x == 0) start = p.w.starts[blockIdx.x];
    __syncthreads();
  }
  const int G = p.s.G, P = p.s.page;
  PagedWalk walk(p.s, p.w.units, seq, first, order, start);
  const int g = lane >> 2, t = lane & 3;
  const float sl2 = p.scale_log2;
  const uint32_t ring = smem_u32(smem) + warp * C::RING * C::TILE;
  const uint32_t ring_exp = smem_u32(smem + C::EXP_OFF) + warp * C::RING * C::EXP;
  // this thread's place in a tile. Keys: row 8 n + g, chunk CHUNKS t; swizzled, so
  // that chunk + c is an exclusive or of c
  const uint32_t k_at = in_box<C::ROW>(g, C::CHUNKS * t);
  // values, bf16: row lane % 16 of 16 keys, chunk lane / 16; e4m3: keys 2 t and
  // 2 t + 1, 8 bytes from column 8 g on
  const uint32_t v_at0 = F8 ? in_box<C::ROW>(2 * t, g >> 1) + 8 * (g & 1) : in_box<C::ROW>(lane & 15, lane >> 4);
  const uint32_t v_at1 = F8 ? in_box<C::ROW>(2 * t + 1, g >> 1) + 8 * (g & 1) : 0u;
  // loading: row lane / CPR of RPI rows, chunk lane % CPR
  const int l_row = lane / C::CPR, l_chunk = lane % C::CPR;
  const uint32_t l_at = (l_chunk * 16 / C::ROW) * C::BOX + in_box<C::ROW>(l_row, l_chunk % (C::ROW / 16));
  PageWindow pages;
  // The warp's tiles of the segment: [j0, j0 + nt), its entries 0 .. 2 nt - 1 (keys
  // and values in turn), RING of them in the ring or on their way. A segment's
  // first AHEAD entries are asked for before the last segment's results are joined
  // (200 sequences of 64 keys, five segments a CTA: 34 us instead of 62).
  int j0 = 0, nt = 0;
  int64_t src_a = 0, src_b = 0;  // rows of the cache: the tile's first 16 (or all) keys, its last 16
  bool bad_a = false, bad_b = false;
  auto begin = [&] {
    j0 = walk.n * warp / C::WARPS;
    nt = walk.n * (warp + 1) / C::WARPS - j0;
    pages.reset(p.table, walk.u.r, p.s.width);
  };
  auto issue = [&](int e, int slot) {
    const PagedUnit& u = walk.u;
    if (e < 2 * nt) {
      const int key0 = tile_of(u, walk.kt + j0 + (e >> 1)) * kTileKeys;
      const int which = e & 1;
      if (which == 0) {
        const int pg0 = key0 >> p.s.page_log, per = P < kTileKeys ? 2 : 1;
        pages.hold(pg0, per, lane);
        const int a = __shfl_sync(kAll, pages.held, pg0 - pages.base);
        const int b = __shfl_sync(kAll, pages.held, pg0 + per - 1 - pages.base);
        const bool see_a = per == 1 || any_seen(p.s, u, key0, key0 + 16);
        const bool see_b = per == 2 && any_seen(p.s, u, key0 + 16, key0 + 32);
        bad_a = !see_a || a < 0 || a >= p.s.n_pages;
        bad_b = per == 2 ? !see_b || b < 0 || b >= p.s.n_pages : bad_a;
        if ((see_a && bad_a) || (see_b && bad_b)) record_error(p.err, FM_DEV_ERR_RANGE);
        src_a = ((int64_t)(bad_a ? 0 : a) * p.s.H_kv + walk.h) * P + (key0 - pg0 * P);
        src_b = per == 2 ? ((int64_t)(bad_b ? 0 : b) * p.s.H_kv + walk.h) * P : src_a + 16;
      }
      // keys that no row of the unit sees (past the sequence's end: anything may lie there) become zeros
      const bool edge = key0 + kTileKeys > u.hi || (p.s.window > 0 && key0 < u.lo) || bad_a || bad_b;
      const char* base = p.kv[which] + l_chunk * 16;
      const uint32_t dst = ring + slot * C::TILE + l_at;
      const char* from_a = base + (src_a + l_row) * C::RB;
      const char* from_b = base + (src_b + l_row) * C::RB;
      auto copies = [&](auto whole) {
#pragma unroll
        for (int i = 0; i < C::LOADS; ++i) {
          const int r0 = i * C::RPI;
          const char* from = r0 < 16 ? from_a + r0 * C::RB : from_b + (r0 - 16) * C::RB;
          const uint32_t x = C::ROW == 128 ? (uint32_t)((r0 & 7) << 4) : (uint32_t)(((r0 >> 1) & 3) << 4);
          if constexpr (whole.value) {
            copy16((dst ^ x) + r0 * C::ROW, from);
          } else {
            const int key = key0 + r0 + l_row;
            copy16((dst ^ x) + r0 * C::ROW, from,
                   key < u.hi && (key >= u.lo || key < p.s.sinks) && !(r0 < 16 ? bad_a : bad_b));
          }
        }
      };
      if (edge)
        copies(std::false_type{});
      else
        copies(std::true_type{});
      if (F8 && lane < 2)
        copy16(ring_exp + slot * C::EXP + 16 * lane, p.exps[which] + (lane ? src_b : src_a), !(lane ? bad_b : bad_a));
    }
    copy_commit();
  };
  if (walk.more()) {
    begin();
#pragma unroll 1
    for (int e = 0; e < C::AHEAD; ++e) issue(e, e);
  }

  while (walk.more()) {
    const PagedUnit& u = walk.u;
#pragma unroll 1
    for (int e = C::AHEAD; e < C::RING; ++e) issue(e, e);
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
            if (live && walk.n > 0) v = *reinterpret_cast<const uint4*>(src + 2 * (e0 + 8 * x4));
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
      // the top of fp16's range: values down to 2^-32 of it keep all their bits
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < C::KSTEPS; ++k)
          top = __vmaxu2(top, __vmaxu2(qf[k][i] & 0x7fff7fffu, qf[k][2 + i] & 0x7fff7fffu));
        top = __vmaxu2(top, __shfl_xor_sync(kAll, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(kAll, top, 2));
        const int E = (int)(max(top & 0xffffu, top >> 16) >> 7);
        // 2^(142 - E), kept finite; a row with infinities or NaN stays as it is
        const int up = E == 255 ? 0 : min(142 - E, 126);
        const float f = __uint_as_float((uint32_t)(127 + up) << 23);
        // 2^-up: on the sums (below 2^33) ahead of a key's scale, so that no score passes
        // fp32's range on the way to one inside it, what is above 2^80 after it. In
        // shared memory until the segment's end (d = 128 112 us, d = 256 271; in registers 116, 293).
        const int back = min(-up, 80);
        if (t == 0) ml[warp * kFewRows + g + 8 * i].x = __uint_as_float((uint32_t)(127 + back) << 23);
        sc[i] = fminf(sl2 * __uint_as_float((uint32_t)(127 - up - back) << 23), FLT_MAX);
#pragma unroll
        for (int k = 0; k < C::KSTEPS; ++k)
#pragma unroll
          for (int x = i; x < 4; x += 2)
            qf[k][x] = pack_f16x2(__uint_as_float(qf[k][x] << 16) * f, __uint_as_float(qf[k][x] & 0xffff0000u) * f);
      }
    }
    // Some thread has a second row (half the softmax otherwise: e4m3 steps of 4 rows a
    // unit 112 us instead of 119, d = 64 77 instead of 83; of 16 rows 124 instead of 122).
    const bool many = u.nrows > 8;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    // e4m3: the running maximum of score + exponent of the value's scale, less kTopBits
    float mo[2] = {-INFINITY, -INFINITY};
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    int slot = 0;  // of the next entry
    for (int j = 0; j < nt; ++j) {
      const int key0 = tile_of(u, walk.kt + j0 + j) * kTileKeys;
      const int sk = slot, sv = slot + 1 == C::RING ? 0 : slot + 1;
      slot = sv + 1 == C::RING ? 0 : sv + 1;
      copy_wait<C::RING - 1>();
      __syncwarp();
      float s[4][4];
      float ve[4][2];  // e4m3: the exponents of the values' scales
      {
        const uint32_t kb = ring + sk * C::TILE + k_at;
#pragma unroll
        for (int n = 0; n < 4; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
        for (int b = 0; b < C::BOXES; ++b)
#pragma unroll
          for (int c = 0; c < C::CHUNKS; ++c)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const uint4 v = lds128((kb ^ (16 * c)) + b * C::BOX + n * 8 * C::ROW);
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
        if constexpr (F8) {
          const float down[2] = {ml[warp * kFewRows + g].x, ml[warp * kFewRows + g + 8].x};
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const uint32_t ek = lds16(ring_exp + sk * C::EXP + 8 * n + 2 * t);
            const uint64_t f = f2_pack(scale_of(ek & 255u), scale_of(ek >> 8));
#pragma unroll
            for (int i = 0; i < 2; ++i)
              f2_unpack(f2_mul(f2_mul(f2_pack(s[n][2 * i], s[n][2 * i + 1]), f2_pack(down[i], down[i])), f), s[n][2 * i],
                        s[n][2 * i + 1]);
          }
        }
      }
      __syncwarp();
      issue(2 * j + C::RING, sk);
      copy_wait<C::RING - 1>();
      __syncwarp();
      {
        if constexpr (F8) {
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const uint32_t ev = lds16(ring_exp + sv * C::EXP + 8 * n + 2 * t);
            ve[n][0] = exponent_of(ev & 255u);
            ve[n][1] = exponent_of(ev >> 8);
          }
        }
        // masked scores: a tile whose keys all rows see is left as it is
        const bool part = key0 + kTileKeys > u.hi || (p.s.causal && key0 + kTileKeys - 1 > plo) ||
                          (p.s.window > 0 && key0 <= phi - p.s.window);
        if (part) {
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = key0 + 8 * n + 2 * t + (x & 1), ps = pos[x >> 1];
              const bool see = key <= ps && key < u.kv_len &&
                               (p.s.window == 0 || key > ps - p.s.window || key < p.s.sinks);
              s[n][x] = see ? s[n][x] : -INFINITY;
            }
          if constexpr (F8) {
            // a key that no row sees: whatever its exponent byte holds
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int key = key0 + 8 * n + 2 * t + x;
                if (!(key < u.hi && (key >= u.lo || key < p.s.sinks))) ve[n][x] = 0.f;
              }
          }
        }
        // a running maximum moves only when it is passed by more than 8 (weights stay below 2^8)
        float f[2] = {1.f, 1.f};
        bool moved = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1 && !many) break;
          float x = -INFINITY, z = -INFINITY;
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            x = max3f(x, s[n][2 * i], s[n][2 * i + 1]);
            if constexpr (F8)
              z = max3f(z, fmaf(s[n][2 * i], sc[i], ve[n][0]), fmaf(s[n][2 * i + 1], sc[i], ve[n][1]));
          }
          x = fmaxf(x, __shfl_xor_sync(kAll, x, 1));
          if constexpr (F8) z = fmaxf(z, __shfl_xor_sync(kAll, z, 1));
          x = fmaxf(x, __shfl_xor_sync(kAll, x, 2)) * sc[i];
          if constexpr (F8) z = fmaxf(z, __shfl_xor_sync(kAll, z, 2));
          if (x > m[i] + 8.f) {
            const float y = ex2_approx(m[i] - x);
            l[i] *= y;
            m[i] = x;
            if (!F8) {
              f[i] = y;
              moved = true;
            }
          }
          if (F8 && z > mo[i] + kTopBits + 8.f) {
            f[i] = ex2_approx(mo[i] + kTopBits - z);
            mo[i] = z - kTopBits;
            moved = true;
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
        uint32_t hi[2][4] = {}, lo[2][4] = {};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1 && !many) break;
          const float base = m[i] == -INFINITY ? 0.f : m[i], bo = mo[i] == -INFINITY ? 0.f : mo[i];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float a = ex2_approx(fmaf(s[n][2 * i], sc[i], -base));
            const float b = ex2_approx(fmaf(s[n][2 * i + 1], sc[i], -base));
            l[i] += a + b;
            if constexpr (F8) {
              const float x = ex2_approx(fmaf(s[n][2 * i], sc[i], ve[n][0] - bo));
              const float y = ex2_approx(fmaf(s[n][2 * i + 1], sc[i], ve[n][1] - bo));
              hi[n >> 1][2 * (n & 1) + i] = pack_f16x2(x, y);
            } else {
              const uint32_t h = pack_bf16x2(a, b);
              hi[n >> 1][2 * (n & 1) + i] = h;
              lo[n >> 1][2 * (n & 1) + i] =
                  pack_bf16x2(a - __uint_as_float(h << 16), b - __uint_as_float(h & 0xffff0000u));
            }
          }
        }
        const uint32_t vb0 = ring + sv * C::TILE + v_at0, vb1 = ring + sv * C::TILE + v_at1;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {  // 16 keys each
            const uint32_t at = 16 * kk * C::ROW;
            if constexpr (F8) {
#pragma unroll
              for (int cg = 0; cg < D / 64; ++cg) {
                // eight columns 64 cg + 8 g + i of keys 2t, 2t + 1, 2t + 8, 2t + 9
                const uint32_t box = (cg * 64 / C::ROW) * C::BOX + at, x64 = cg * 64 % C::ROW;
                const uint2 w0 = lds64((vb0 ^ x64) + box), w1 = lds64((vb1 ^ x64) + box);
                const uint2 w2 = lds64((vb0 ^ x64) + box + 8 * C::ROW), w3 = lds64((vb1 ^ x64) + box + 8 * C::ROW);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t a0 = h ? w0.y : w0.x, a1 = h ? w1.y : w1.x, a2 = h ? w2.y : w2.x, a3 = h ? w3.y : w3.x;
                  uint32_t b0[4], b1[4];
                  e4m3_to_f16(__byte_perm(a0, a1, 0x5140), b0[0], b0[1]);
                  e4m3_to_f16(__byte_perm(a0, a1, 0x7362), b0[2], b0[3]);
                  e4m3_to_f16(__byte_perm(a2, a3, 0x5140), b1[0], b1[1]);
                  e4m3_to_f16(__byte_perm(a2, a3, 0x7362), b1[2], b1[3]);
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    mma16816_f16(o[8 * cg + 4 * h + i], hi[kk], b0[i], b1[i]);
                }
              }
            } else {
#pragma unroll
              for (int c = 0; c < D / 8; c += 2) {
                uint32_t r[4];
                ldmatrix4_trans((vb0 ^ (16 * (c & 7))) + (c >> 3) * C::BOX + at, r);
                mma16816(o[c], hi[kk], r[0], r[1]);
                mma16816(o[c + 1], hi[kk], r[2], r[3]);
                mma16816(o[c], lo[kk], r[0], r[1]);
                mma16816(o[c + 1], lo[kk], r[2], r[3]);
              }
            }
        }
      }
      __syncwarp();
      issue(2 * j + 1 + C::RING, sv);
    }
    copy_wait<0>();

    // Join the warps' (m, l, O): each leaves its own in the last entries of its
    // ring, then every thread adds up four columns of a row at a time. Column c of
    // row r lies at c ^ 8 (r % 4): four rows start 8 banks apart.
    const int tok0 = u.tok, g0 = u.g0, nrows = u.nrows, h = walk.h, part_slot = walk.slot();
    const bool whole = walk.whole();
    walk.next();
    if (walk.more()) {
      begin();
#pragma unroll 1
      for (int e = 0; e < C::AHEAD; ++e) issue(e, e);
    }
    float* own = reinterpret_cast<float*>(smem + (warp * C::RING + C::AHEAD) * C::TILE);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(kAll, l[i], 1);
      l[i] += __shfl_xor_sync(kAll, l[i], 2);
      const int row = g + 8 * i;
      // O's unit is 2^m, e4m3: 2^mo
      if (t == 0) ml[warp * kFewRows + row] = make_float4(m[i], l[i], F8 ? mo[i] : m[i], 0.f);
      if constexpr (F8) {
        // columns 64 cg + 16 t + 8 y + (0 .. 7)
#pragma unroll
        for (int cg = 0; cg < D / 64; ++cg)
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int z = 0; z < 2; ++z)
              *reinterpret_cast<float4*>(own + row * D + ((64 * cg + 16 * t + 8 * y + 4 * z) ^ (8 * (row & 3)))) =
                  make_float4(o[8 * cg + 4 * z][2 * i + y], o[8 * cg + 4 * z + 1][2 * i + y],
                              o[8 * cg + 4 * z + 2][2 * i + y], o[8 * cg + 4 * z + 3][2 * i + y]);
      } else {
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<float2*>(own + row * D + ((8 * c + 2 * t) ^ (8 * (row & 3)))) =
              make_float2(o[c][2 * i], o[c][2 * i + 1]);
      }
    }
    __syncthreads();
    {
      constexpr int TPR = C::THREADS / kFewRows;  // threads a row
      const int row = threadIdx.x / TPR, c0 = threadIdx.x % TPR, x = g0 + row;
      if (row < nrows) {
        float top = -INFINITY, sum = 0.f, w[C::WARPS];
#pragma unroll
        for (int k = 0; k < C::WARPS; ++k) top = fmaxf(top, ml[k * kFewRows + row].x);
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int k = 0; k < C::WARPS; ++k) {
          const float4 v = ml[k * kFewRows + row];
          sum += ex2_approx(v.x - base) * v.y;
          w[k] = ex2_approx(v.z - base);
        }
        const float inv = !whole ? 1.f : sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        const int64_t tok = tok0 + x / G;
        const int head = h * G + x % G;
        char* dst = p.out.o + 2 * (tok * p.out.st + head * p.out.sh);
        float* part = p.w.part + p.w.part_floats * (2 * (size_t)blockIdx.x + part_slot);
#pragma unroll
        for (int c = 0; c < D / (4 * TPR); ++c) {
          const int col = 4 * (c0 + TPR * c);
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < C::WARPS; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(
                reinterpret_cast<const float*>(smem + (k * C::RING + C::AHEAD) * C::TILE) + row * D +
                (col ^ (8 * (row & 3))));
            a.x += w[k] * v.x;
            a.y += w[k] * v.y;
            a.z += w[k] * v.z;
            a.w += w[k] * v.w;
          }
          if (whole)
            *reinterpret_cast<uint2*>(dst + 2 * col) =
                make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
          else
            *reinterpret_cast<float4*>(part + (size_t)row * D + col) = a;
        }
        if (c0 == 0) {
          if (whole) {
            p.out.lse[tok * p.out.H_q + head] = sum == 0.f ? -INFINITY : top * kLn2F + logf(sum);
          } else {
            part[(size_t)kFewRows * D + 2 * row] = top;
            part[(size_t)kFewRows * D + 2 * row + 1] = sum;
          }
        }
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------- joining
struct JoinParams {
  PagedWork w;
  PagedOut out;
  int G, rows;  // rows of a slot
};

// Block (c, y): where CTA c's range is the second one inside a unit and head,
// their parts (CTA c - 1's last segment, then c .. last's first segments) are
// joined. Latency bounds it, so it goes by what there is more of. Many rows of a
// few parts each (chunk_kernel's slots of 256 rows): ROWS = 2 rows (d = 64: four) a
// warp, four parts of each in flight (256 tokens over 4096 keys 32.5 us; four rows, two
// parts 33.1; one row, eight parts 33.4). Few rows: one a warp, eight parts in flight, or,
// of many parts, a long cache's, one by WPR = 4 warps (one token over 32000 keys, 38
// parts: 32 us for the call, 35 with one warp a row; but where one warp is enough,
// three times the blocks cost about 2 us).
template <int D, int ROWS, int WPR>
__global__ void __launch_bounds__(256) join_kernel(const JoinParams p) {
  constexpr int LPR = D / 4 < 32 ? D / 4 : 32, RPW = 32 / LPR, V = D / (4 * LPR);  // lanes a row, rows a warp
  constexpr int PARTS = ROWS > 1 ? 4 : 8;
  __shared__ float4 other[WPR > 1 ? 8 * 32 * V : 1];
  __shared__ float2 other_ml[WPR > 1 ? 8 * RPW : 1];
  grid_dependency_wait();
  const int c = blockIdx.x + 1;
  const PagedStart& st = p.w.starts[c];
  if (st.count <= 0 || st.kt == 0 || st.first != c - 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = 4 * (lane % LPR);
  const int row0 = (blockIdx.y * (8 / WPR) + warp / WPR) * ROWS * RPW + lane / LPR;  // then every RPW-th
  const int nrows = st.unit.nrows;
  const int parts = st.last - c + 2;
  // part i: slot 1 of CTA c - 1 (i = 0), slot 0 of CTA c - 1 + i
  auto part = [&](int i) { return p.w.part + p.w.part_floats * (2 * (size_t)(c - 1 + i) + (i == 0 ? 1 : 0)); };
  float top[ROWS], sum[ROWS];
  float4 acc[ROWS][V];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    top[r] = -INFINITY;
    sum[r] = 0.f;
#pragma unroll
    for (int x = 0; x < V; ++x) acc[r][x] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // a row so far and one more part of it
  auto add = [&](float& t, float& s, float4 (&a)[V], float pt, float ps, const float4 (&pv)[V]) {
    const float m = fmaxf(t, pt), base = m == -INFINITY ? 0.f : m;
    const float f = ex2_approx(t - base), y = ex2_approx(pt - base);
    t = m;
    s = s * f + y * ps;
#pragma unroll
    for (int x = 0; x < V; ++x) {
      a[x].x = a[x].x * f + y * pv[x].x;
      a[x].y = a[x].y * f + y * pv[x].y;
      a[x].z = a[x].z * f + y * pv[x].z;
      a[x].w = a[x].w * f + y * pv[x].w;
    }
  };
  for (int i0 = PARTS * (warp % WPR); i0 < parts; i0 += PARTS * WPR) {
    float2 w[ROWS][PARTS];
    float4 v[ROWS][PARTS][V];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        const int row = row0 + r * RPW;
        w[r][k] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int x = 0; x < V; ++x) v[r][k][x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0 + k < parts && row < nrows) {
          const float* s = part(i0 + k);
          w[r][k] = *reinterpret_cast<const float2*>(s + (size_t)p.rows * D + 2 * row);
#pragma unroll
          for (int x = 0; x < V; ++x)
            v[r][k][x] = *reinterpret_cast<const float4*>(s + (size_t)row * D + 4 * LPR * x + col);
        }
      }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int k = 0; k < PARTS; ++k) add(top[r], sum[r], acc[r], w[r][k].x, w[r][k].y, v[r][k]);
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int x = 0; x < V; ++x) other[(warp * V + x) * 32 + lane] = acc[0][x];
    if (col == 0) other_ml[warp * RPW + lane / LPR] = make_float2(top[0], sum[0]);
    __syncthreads();
    if (warp % WPR) return;
#pragma unroll
    for (int k = 1; k < WPR; ++k) {
      float4 v[V];
#pragma unroll
      for (int x = 0; x < V; ++x) v[x] = other[((warp + k) * V + x) * 32 + lane];
      const float2 w = other_ml[(warp + k) * RPW + lane / LPR];
      add(top[0], sum[0], acc[0], w.x, w.y, v);
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int row = row0 + r * RPW;
    if (row >= nrows) continue;
    const float inv = sum[r] > 0.f ? 1.f / sum[r] : (sum[r] == 0.f ? 0.f : sum[r]);
    const int x0 = st.unit.g0 + row;
    const int64_t tok = st.unit.tok + x0 / p.G;
    const int head = st.h * p.G + x0 % p.G;
    char* dst = p.out.o + 2 * (tok * p.out.st + head * p.out.sh);
#pragma unroll
    for (int x = 0; x < V; ++x)
      *reinterpret_cast<uint2*>(dst + 2 * (4 * LPR * x + col)) = make_uint2(
          pack_bf16x2(acc[r][x].x * inv, acc[r][x].y * inv), pack_bf16x2(acc[r][x].z * inv, acc[r][x].w * inv));
    if (col == 0) p.out.lse[tok * p.out.H_q + head] = sum[r] == 0.f ? -INFINITY : top[r] * kLn2F + logf(sum[r]);
  }
}

template <int D>
cudaError_t launch_join(const PagedShape& s, const PagedWork& w, const PagedOut& out, int rows, cudaStream_t st) {
  if (s.ctas < 2) return cudaSuccess;
  const JoinParams j{w, out, s.G, rows};
  // units and heads, and the parts that each comes in, about
  const double units = (double)(s.max_units - s.R / 2) * s.H_kv;
  const double tiles = (double)s.width * s.page / s.tile;
  const double parts = std::min(s.ctas / units, tiles / s.least) + 1;
  auto go = [&](auto kernel, int per) {  // rows of a block
    const dim3 grid((unsigned)(s.ctas - 1), (unsigned)((rows + per - 1) / per));
    count_launches(1);
    return launch_dependent(kernel, grid, 256, 0, st, j);
  };
  constexpr int RPW = D == 64 ? 2 : 1;
  if (parts > 9) return go(join_kernel<D, 1, 4>, 2 * RPW);
  if (rows == kChunkRows) return go(join_kernel<D, 2, 1>, 16 * RPW);
  return go(join_kernel<D, 1, 1>, 8 * RPW);
}

template <int D, bool F8>
cudaError_t launch_few(const PagedShape& s, const PagedWork& w, const fm_kv_cache& c, const fm_paged_batch& b,
                       const fm_rows& q, const PagedOut& out, float scale, cudaStream_t st, int* err) {
  using C = FewCfg<D, F8>;
  static_assert(C::SMEM <= 232448 && C::PER_SM * (C::SMEM + 1024) <= 233472, "few_kernel: shared memory of an SM");
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(few_kernel<D, F8>), C::SMEM, ready);
  if (e != cudaSuccess) return e;
  FewParams p{s, w, static_cast<const char*>(q.ptr), q.st, q.sh, out,
              {static_cast<const char*>(c.k), static_cast<const char*>(c.v)}, {c.k_exp, c.v_exp}, b.q_off, b.kv_len,
              b.page_table, scale * 1.4426950408889634f, err};
  count_launches(1);
  return launch_dependent(few_kernel<D, F8>, dim3((unsigned)s.ctas), C::THREADS, C::SMEM, st, p);
}

// Whether units stay whole, one CTA each, or ranges of tiles may end inside them.
// Whole units leave CTAs idle in the last round, `most` tiles each at worst (and
// sequences are taken to be ragged: two fifths of it at least, where there are
// several); divided ones cost the parts' writing and joining, and a start and an end
// for every part. What the host knows decides: the units that T tokens make, the
// keys that the page table has room for. chunk_kernel (tiles of 128 keys, about 1.5
// us): 2048 tokens of 32 / 8 heads over themselves 33 us whole, 51 divided; 4096
// over themselves 100, 131; 2048 over 4096 keys 77, 92; 256 over 2048 keys 31, 27; 512
// over 4096 keys 53, 43; a full prompt's units grow from one tile to `most`, so less is
// left idle. few_kernel (tiles of 32 keys): 64 sequences of 500 keys 17 us whole, 23
// divided; one of 300 keys 9.1, 12.0; one of 1021 17.7, 10.0.
bool stay_whole(const PagedShape& s, const fm_paged_batch& b, long long most, bool chunk) {
  const double units = (double)s.H_kv * (chunk ? ((double)s.T * s.G / s.step + b.R / 2.0)
                                               : std::max((double)b.R, (double)s.T * s.G / s.step));
  const double rounds = units / s.ctas;
  double idle = most * std::max(std::ceil(rounds) - rounds, b.R > 1 ? 0.4 : 0.0);
  if (b.R == 1 && s.causal && s.window == 0 && 2ll * s.T >= (long long)b.width * s.page)
    idle /= 4 * std::max(1.0, rounds);
  if (!chunk || b.R > 1) idle /= std::max(1.0, rounds);  // ragged lengths even out over the rounds
  return idle <= (chunk ? 5 + 8 * std::min(1.0, rounds) : 12);
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
  s.page_log = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
  s.n_pages = c.n_pages;
  s.causal = causal;
  // positions stay below 2^30: larger windows and sinks hide nothing more
  s.window = std::min(window, 1 << 30);
  s.sinks = window > 0 ? std::min(sinks, 1 << 30) : 0;
  s.step = chunk ? 2 * (128 / s.G) * s.G : kFewRows;
  s.tile_log = chunk ? 7 : 5;
  s.tile = 1 << s.tile_log;
  static_assert(kTileKeys == 32, "tile_log");
  s.least = chunk ? 1 : few_warps(c.d, c.k_exp != nullptr);  // a tile for each computing warp, and fewer parts to join
  s.extra = chunk ? (c.k_exp ? 3 : 2) : (c.k_exp ? 10 : 4);
  s.ctas = sm_count() * (chunk ? 1 : few_ctas(c.d, c.k_exp != nullptr));
  s.max_units = ((long long)T * s.G + s.step - 1) / s.step + b.R;
  // Each CTA plans for itself where that is a few steps a warp; a plan kernel (one
  // CTA, about 4 us of the stream) for larger batches.
  const long long most = ((long long)b.width * s.page + s.tile - 1) / s.tile;  // tiles of a unit
  const bool few_seqs = b.R <= (chunk ? kLocalChunks : kLocalSeqs);
  s.whole = few_seqs && (b.R == 1 || s.max_units <= kWholeUnits) && stay_whole(s, b, most, chunk);
  s.local = s.whole || (few_seqs && s.max_units - b.R <= kLocalUnits &&
                        s.max_units * (most + s.extra) * s.H_kv * (s.ctas + 1) < (1ll << 31));
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
  cudaError_t e = cudaSuccess;
  if (!s.local) {
    const PlanParams pp{s, b.q_off, b.kv_len, w, err};
    count_launches(1);
    e = launch_dependent(plan_kernel, dim3(1), kPlanThreads, 0, st, pp);
    if (e != cudaSuccess) return e;
  }
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
  if (e != cudaSuccess || s.whole) return e;
  return c.d == 64    ? launch_join<64>(s, w, out, rows, st)
         : c.d == 128 ? launch_join<128>(s, w, out, rows, st)
                      : launch_join<256>(s, w, out, rows, st);
}

}  // namespace fm
