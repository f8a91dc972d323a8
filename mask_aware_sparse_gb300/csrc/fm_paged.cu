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
  PagedLists in;
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

template <bool SH>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  __shared__ long long sums[32];
  __shared__ long long carry;
  const PagedShape& s = p.s;
  const int tid = threadIdx.x;
  grid_dependency_wait();
  grid_launch_dependents();
  bool bad = false;
  // sequence r of the plan
  auto sequence = [&](int r, int4& q, int2& more) -> bool {
    if constexpr (SH) {
      const int vs = prefixes(s);
      int s0, s1, P;
      if (r < vs) return prefix_at(s, p.in, r, q, more, s0);
      const int g = last_at(p.in.seq_off, s.S, r - vs);
      const bool off = group_at(s, p.in, g, s0, s1, P);
      if (alone(p.in, r - vs, s0, s1)) P = 0;
      return rest_at(s, p.in, r - vs, P, p.in.prefix_len[g], q, more) || off;
    } else {
      const bool off = sequence_at(s, p.in.q_off, p.in.kv_len, r, q.x, q.y, q.z);
      q.w = (int)(((long long)q.y * s.G + s.step - 1) / s.step);
      return off;
    }
  };
  // units of each sequence
  if (tid == 0) {
    carry = 0;
    p.w.first[0] = 0;
  }
  __syncthreads();
  for (int r0 = 0; r0 < s.V; r0 += kPlanThreads) {
    const int r = r0 + tid;
    long long n = 0;
    if (r < s.V) {
      int4 q;
      int2 more;
      bad |= sequence(r, q, more);
      n = q.w;
    }
    const long long in = block_scan(n, sums) + carry;
    if (r < s.V) p.w.first[r + 1] = (int)min(in, s.max_units);
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
      const int r = last_at(p.w.first, s.V, u);
      int4 q;
      int2 more;
      sequence(r, q, more);
      PagedUnit unit;
      if constexpr (SH)
        unit = shared_unit_at(s, r, q, more, u - p.w.first[r]);
      else
        unit = unit_at(s, r, q.x, q.y, q.z, u - p.w.first[r]);
      p.w.units[u] = unit;
      work = (long long)max(unit.ntiles, 1) * s.H_kv;
    }
    const long long in = block_scan(work, sums) + carry;
    if (u < units) p.w.sum[u] = in - work;
    __syncthreads();
    if (tid == kPlanThreads - 1) carry = in;
    __syncthreads();
  }
  const PagedDivision<SH, long long> div(s, carry, units);
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
static_assert(kFewRows <= kMarkRows, "a mark's row");
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
  PagedLists in;
  SharedOut sh;
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

// How few_kernel shares its work out: kPlain, and, where sequences share prefixes, kBoth: as
// there, over the prefixes and what follows them, and kRest, over what follows them alone:
// each warp takes a range of its own, as a CTA of one warp. Its units are short, and no
// warp waits for others at their ends; merge_kernel joins parts in any case. (64 sequences
// of up to 1024 keys behind 16384 shared ones, e4m3: the whole call 73 us, with CTAs' ranges
// 76.5; 128 of them, bf16, 165, 173. Over the prefixes too, with four times the parts: 8
// sequences behind 2048 keys 20 us, with CTAs' ranges 15.9; 4 behind 32768 48, 37.6.)
enum Few { kPlain, kBoth, kRest };

template <int D, bool F8, Few MODE>
__global__ void __launch_bounds__(FewCfg<D, F8>::THREADS, FewCfg<D, F8>::PER_SM) few_kernel(const FewParams p) {
  using C = FewCfg<D, F8>;
  constexpr bool SH = MODE != kPlain, ALONE = MODE == kRest;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float4* ml = reinterpret_cast<float4*>(smem + C::ML_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int OWN = ALONE ? C::WARPS : 1, AHEAD = ALONE ? C::RING : C::AHEAD;
  const int worker = ALONE ? blockIdx.x * C::WARPS + warp : blockIdx.x;
  __shared__ PagedStart starts[OWN];
  __shared__ int4 seq[kLocalSeqs];
  __shared__ int2 more[SH ? kLocalSeqs : 1];
  __shared__ uint16_t first[SH ? 1 : kLocalSeqs + 1], order[SH ? 1 : kWholeUnits];
  grid_dependency_wait();
  grid_launch_dependents();
  if (!SH && p.s.whole) {
    plan_whole(p.s, p.in, seq, first, order, reinterpret_cast<uint16_t*>(smem), starts, p.err);
  } else if (p.s.local) {
    plan_locally<SH, OWN>(p.s, p.in, seq, more, reinterpret_cast<unsigned*>(smem), starts, p.err);
    if (!SH && threadIdx.x == 0) p.w.starts[blockIdx.x] = starts[0];  // for join_kernel
  } else {
    if (threadIdx.x < OWN) starts[threadIdx.x] = p.w.starts[blockIdx.x * OWN + threadIdx.x];
    __syncthreads();
  }
  const PagedStart& start = starts[ALONE ? warp : 0];
  const int G = p.s.G, P = p.s.page;
  PagedWalk<SH> walk(p.s, p.w.units, seq, more, first, order, start);
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
    j0 = ALONE ? 0 : walk.n * warp / C::WARPS;
    nt = ALONE ? walk.n : walk.n * (warp + 1) / C::WARPS - j0;
    pages.reset(p.table, walk.u.r, p.s.width);
  };
  auto issue = [&](int e, int slot) {
    const PagedUnit& u = walk.u;
    if (e < 2 * nt) {
      const int key0 = key_of<SH, kTileKeys>(u, walk.kt + j0 + (e >> 1));
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
  if (walk.going()) {
    begin();
#pragma unroll 1
    for (int e = 0; e < AHEAD; ++e) issue(e, e);
  }

  while (walk.going()) {
    const PagedUnit& u = walk.u;
#pragma unroll 1
    for (int e = AHEAD; e < C::RING; ++e) issue(e, e);
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
      const int key0 = key_of<SH, kTileKeys>(u, walk.kt + j0 + j);
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
    const uint32_t mark = SH ? shared_mark(whole, walk.kt, start, worker) : 0u;
    const int kind = u.ns;  // (SH)
    walk.next();
    if (walk.going()) {
      begin();
#pragma unroll 1
      for (int e = 0; e < AHEAD; ++e) issue(e, e);
    }
    if constexpr (ALONE) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(kAll, l[i], 1);
        l[i] += __shfl_xor_sync(kAll, l[i], 2);
        const int row = g + 8 * i, x = g0 + row;
        if (row >= nrows) continue;
        const long long at = kind * p.sh.rows + (long long)(tok0 + x / G) * p.out.H_q + h * G + x % G;
        float* part = p.w.part + p.w.part_floats * (2 * (size_t)worker + part_slot);
        float* to = whole ? p.sh.full + at * D : part + (size_t)row * D;
        // e4m3: O's unit is 2^mo, the part's 2^m (by two factors, as where warps are joined)
        const float apart = F8 ? mo[i] - (m[i] == -INFINITY ? 0.f : m[i]) : 0.f;
        const float f = F8 ? ex2_approx(apart < -64.f ? apart + 64.f : apart) : 1.f;
        const float down = F8 && apart < -64.f ? 0x1p-64f : 1.f;
        if constexpr (F8) {
          // columns 64 cg + 16 t + 8 y + (0 .. 7)
#pragma unroll
          for (int cg = 0; cg < D / 64; ++cg)
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const float(*a)[4] = o + 8 * cg + 4 * z;
                const int x = 2 * i + y;
                *reinterpret_cast<float4*>(to + 64 * cg + 16 * t + 8 * y + 4 * z) =
                    make_float4(f * a[0][x] * down, f * a[1][x] * down, f * a[2][x] * down, f * a[3][x] * down);
              }
        } else {
#pragma unroll
          for (int c = 0; c < D / 8; ++c)
            *reinterpret_cast<float2*>(to + 8 * c + 2 * t) = make_float2(o[c][2 * i], o[c][2 * i + 1]);
        }
        if (t == 0) {
          *(whole ? p.sh.full_ml + at : reinterpret_cast<float2*>(part + (size_t)kFewRows * D) + row) =
              make_float2(m[i], l[i]);
          if (mark) p.sh.where[at] = whole ? mark : mark | (uint32_t)row;
        }
      }
      __syncwarp();  // (ml is written again)
      continue;
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
        // e4m3: O's unit may be far below 2^m, by the values' scales (2^-126 and less): a factor
        // that exp2's smallest numbers do not hold, so it is taken as two
        float up = 0.f;
        if constexpr (F8) {
          float unit = -INFINITY;
#pragma unroll
          for (int k = 0; k < C::WARPS; ++k) unit = fmaxf(unit, ml[k * kFewRows + row].z);
          up = unit - base < -64.f ? 64.f : 0.f;
        }
        const float down = up > 0.f ? 0x1p-64f : 1.f;
#pragma unroll
        for (int k = 0; k < C::WARPS; ++k) {
          const float4 v = ml[k * kFewRows + row];
          sum += ex2_approx(v.x - base) * v.y;
          w[k] = ex2_approx(v.z - base + up);
        }
        const float inv = SH || !whole ? 1.f : sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        const int64_t tok = tok0 + x / G;
        const int head = h * G + x % G;
        char* dst = p.out.o + 2 * (tok * p.out.st + head * p.out.sh);
        float* part = p.w.part + p.w.part_floats * (2 * (size_t)blockIdx.x + part_slot);
        const long long at = SH ? kind * p.sh.rows + tok * p.out.H_q + head : 0;
        float* to = SH && whole ? p.sh.full + at * D : part + (size_t)row * D;
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
          a = make_float4(a.x * down, a.y * down, a.z * down, a.w * down);
          if (!SH && whole)
            *reinterpret_cast<uint2*>(dst + 2 * col) =
                make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
          else
            *reinterpret_cast<float4*>(to + col) = a;
        }
        if (c0 == 0) {
          if constexpr (SH) {
            *(whole ? p.sh.full_ml + at : reinterpret_cast<float2*>(part + (size_t)kFewRows * D) + row) =
                make_float2(top, sum);
            if (mark) p.sh.where[at] = whole ? mark : mark | (uint32_t)row;
          } else if (whole) {
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

// A row so far, and one more part of it.
template <int V>
__device__ __forceinline__ void add_part(float& t, float& s, float4 (&a)[V], const float2& ml, const float4 (&v)[V]) {
  const float m = fmaxf(t, ml.x), base = m == -INFINITY ? 0.f : m;
  const float f = ex2_approx(t - base), y = ex2_approx(ml.x - base);
  t = m;
  s = s * f + y * ml.y;
#pragma unroll
  for (int x = 0; x < V; ++x) {
    a[x].x = a[x].x * f + y * v[x].x;
    a[x].y = a[x].y * f + y * v[x].y;
    a[x].z = a[x].z * f + y * v[x].z;
    a[x].w = a[x].w * f + y * v[x].w;
  }
}

// A whole row, LPR lanes on it, four columns of V places each.
template <int LPR, int V>
__device__ __forceinline__ void store_row(const PagedOut& out, int64_t tok, int head, int col, float top, float sum,
                                          const float4 (&acc)[V]) {
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  char* dst = out.o + 2 * (tok * out.st + head * out.sh);
#pragma unroll
  for (int x = 0; x < V; ++x)
    *reinterpret_cast<uint2*>(dst + 2 * (4 * LPR * x + col)) =
        make_uint2(pack_bf16x2(acc[x].x * inv, acc[x].y * inv), pack_bf16x2(acc[x].z * inv, acc[x].w * inv));
  if (col == 0) out.lse[tok * out.H_q + head] = sum == 0.f ? -INFINITY : top * kLn2F + logf(sum);
}

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
      for (int k = 0; k < PARTS; ++k) add_part(top[r], sum[r], acc[r], w[r][k], v[r][k]);
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
      add_part(top[0], sum[0], acc[0], w, v);
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int row = row0 + r * RPW;
    if (row >= nrows) continue;
    const int x0 = st.unit.g0 + row;
    store_row<LPR>(p.out, st.unit.tok + x0 / p.G, st.h * p.G + x0 % p.G, col, top[r], sum[r], acc[r]);
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

// Rows of sequences that share a prefix: each row's parts over the prefix, then those over
// the rest. Latency bounds it (where the parts are, then the parts), so rows in flight
// count, and few registers for each: a row a warp, three parts at a time, the next row's
// places loaded meanwhile, five blocks an SM (41K rows of three parts 18.6 us; two rows a
// warp 20.4, four parts of each 25). Of many parts, four warps a row, five parts at a time
// each (64 sequences behind 16384 keys 71.3 us for the call; eight parts, three blocks 73.9).
struct MergeParams {
  PagedOut out;
  SharedOut sh;
  const float* part[2];  // of each kind: slots, floats of one, rows of one, CTAs
  size_t part_floats[2];
  int slot_rows[2], ctas[2];
  const int32_t* q_off;
  int R, T;
};

// Blocks an SM that registers are kept for.
constexpr int merge_blocks(int d, int wpr) { return d == 256 ? 2 : wpr > 1 ? 4 : 5; }

template <int D, int WPR>
__global__ void __launch_bounds__(256, merge_blocks(D, WPR)) merge_kernel(const MergeParams p) {
  constexpr int LPR = D / 4 < 32 ? D / 4 : 32, RPW = 32 / LPR, V = D / (4 * LPR);  // lanes a row, rows a warp
  constexpr int PARTS = WPR > 1 ? 5 : 3;
  constexpr int BLOCK = (8 / WPR) * RPW;  // rows of a block's step
  __shared__ float4 other[WPR > 1 ? 8 * 32 * V : 1];
  __shared__ float2 other_ml[WPR > 1 ? 8 * RPW : 1];
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = 4 * (lane % LPR);
  // (rows are below 2^30)
  const int all = (int)p.sh.rows, stride = gridDim.x * BLOCK;
  int i = blockIdx.x * BLOCK + (warp / WPR) * RPW + lane / LPR;  // this thread's row
  uint32_t next[2];
  auto look = [&](int r) {
#pragma unroll
    for (int k = 0; k < 2; ++k) next[k] = r < all ? p.sh.where[k * p.sh.rows + r] : 0u;
  };
  look(i);
  // tokens of no sequence keep their rows
  const int rows = min(all, min(max(p.q_off[p.R], 0), p.T) * p.out.H_q);
  for (int b = blockIdx.x * BLOCK; b < all; b += stride, i += stride) {
    uint32_t at[2];
    int n[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t w = at[k] = next[k];
      const int first = mark_first(w), parts = mark_parts(w), row = mark_row(w);
      n[k] = i >= rows ? 0 : w == kMarkWhole ? 1 : parts;
      // (what a batch that is none left there)
      if (w != kMarkWhole && (first + parts > p.ctas[k] || row >= p.slot_rows[k])) n[k] = 0;
    }
    look(i + stride);
    float top = -INFINITY, sum = 0.f;
    float4 acc[V];
#pragma unroll
    for (int x = 0; x < V; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int parts = n[0] + n[1];
    for (int j0 = PARTS * (warp % WPR); j0 < parts; j0 += PARTS * WPR) {
      float2 w[PARTS];
      float4 v[PARTS][V];
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        w[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int x = 0; x < V; ++x) v[k][x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j0 + k < parts) {
          const bool rest = j0 + k >= n[0];
          const int j = rest ? j0 + k - n[0] : j0 + k;
          const uint32_t where = rest ? at[1] : at[0];
          const float *from, *ml;
          if (where == kMarkWhole) {
            const size_t r = i + (rest ? p.sh.rows : 0);
            from = p.sh.full + r * D;
            ml = reinterpret_cast<const float*>(p.sh.full_ml + r);
          } else {  // slot 1 of the first CTA, slot 0 of the others
            const size_t slot = 2 * (size_t)(mark_first(where) + j) + (j == 0 ? 1 : 0);
            const float* s = (rest ? p.part[1] : p.part[0]) + (rest ? p.part_floats[1] : p.part_floats[0]) * slot;
            from = s + (size_t)mark_row(where) * D;
            ml = s + (size_t)(rest ? p.slot_rows[1] : p.slot_rows[0]) * D + 2 * mark_row(where);
          }
          w[k] = *reinterpret_cast<const float2*>(ml);
#pragma unroll
          for (int x = 0; x < V; ++x) v[k][x] = *reinterpret_cast<const float4*>(from + 4 * LPR * x + col);
        }
      }
#pragma unroll
      for (int k = 0; k < PARTS; ++k)
        if (j0 + k < parts) add_part(top, sum, acc, w[k], v[k]);
    }
    if constexpr (WPR > 1) {
#pragma unroll
      for (int x = 0; x < V; ++x) other[(warp * V + x) * 32 + lane] = acc[x];
      if (col == 0) other_ml[warp * RPW + lane / LPR] = make_float2(top, sum);
      __syncthreads();
      if (warp % WPR == 0) {
#pragma unroll
        for (int k = 1; k < WPR; ++k) {
          float4 v[V];
#pragma unroll
          for (int x = 0; x < V; ++x) v[x] = other[((warp + k) * V + x) * 32 + lane];
          add_part(top, sum, acc, other_ml[(warp + k) * RPW + lane / LPR], v);
        }
      }
      __syncthreads();
    }
    if (i < rows && warp % WPR == 0)
      store_row<LPR>(p.out, i / p.out.H_q, i % p.out.H_q, col, top, sum, acc);
  }
}

template <int D, bool F8, Few MODE>
cudaError_t launch_few(const PagedShape& s, const PagedWork& w, const fm_kv_cache& c, const PagedLists& in,
                       const int32_t* table, const fm_rows& q, const PagedOut& out, const SharedOut& sh, float scale,
                       cudaStream_t st, int* err) {
  using C = FewCfg<D, F8>;
  static_assert(C::SMEM <= 232448 && C::PER_SM * (C::SMEM + 1024) <= 233472, "few_kernel: shared memory of an SM");
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(few_kernel<D, F8, MODE>), C::SMEM, ready);
  if (e != cudaSuccess) return e;
  FewParams p{s, w, static_cast<const char*>(q.ptr), q.st, q.sh, out,
              {static_cast<const char*>(c.k), static_cast<const char*>(c.v)}, {c.k_exp, c.v_exp}, in, sh, table,
              scale * 1.4426950408889634f, err};
  count_launches(1);
  return launch_dependent(few_kernel<D, F8, MODE>, dim3((unsigned)(MODE == kRest ? s.ctas / C::WARPS : s.ctas)), C::THREADS, C::SMEM, st, p);
}

// The plan, where no CTA makes its own, and the attention kernel.
template <bool SH>
cudaError_t launch_attention(bool chunk, const PagedShape& s, const PagedWork& w, const fm_kv_cache& c,
                             const PagedLists& in, const int32_t* table, const fm_rows& q, const PagedOut& out,
                             const SharedOut& sh, float scale, cudaStream_t st, int* err) {
  if (!s.local) {
    const PlanParams pp{s, in, w, err};
    count_launches(1);
    const cudaError_t e = launch_dependent(plan_kernel<SH>, dim3(1), kPlanThreads, 0, st, pp);
    if (e != cudaSuccess) return e;
  }
  if (chunk) return launch_paged_chunk(s, w, c, in, table, q, out, SH ? &sh : nullptr, scale, st, err);
  auto go = [&](auto d, auto mode) {
    return c.k_exp ? launch_few<d.value, true, mode.value>(s, w, c, in, table, q, out, sh, scale, st, err)
                   : launch_few<d.value, false, mode.value>(s, w, c, in, table, q, out, sh, scale, st, err);
  };
  auto dims = [&](auto mode) {
    if constexpr (mode.value != kRest)  // (goes with chunk_kernel over the prefixes)
      if (c.d == 256) return go(std::integral_constant<int, 256>{}, mode);
    return c.d == 64 ? go(std::integral_constant<int, 64>{}, mode) : go(std::integral_constant<int, 128>{}, mode);
  };
  if constexpr (SH)
    return s.kinds == 3 ? dims(std::integral_constant<Few, kBoth>{}) : dims(std::integral_constant<Few, kRest>{});
  else
    return dims(std::integral_constant<Few, kPlain>{});
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
  s.V = b.R;
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
  const PagedLists in{b.q_off, b.kv_len, nullptr, nullptr};
  const cudaError_t e =
      launch_attention<false>(chunk, s, w, c, in, b.page_table, q, out, SharedOut{}, scale, st, err);
  if (e != cudaSuccess || s.whole) return e;
  return c.d == 64    ? launch_join<64>(s, w, out, rows, st)
         : c.d == 128 ? launch_join<128>(s, w, out, rows, st)
                      : launch_join<256>(s, w, out, rows, st);
}

// ------------------------------------------------------------ shared prefixes
namespace {

// How a call whose sequences share prefixes runs.
struct SharedPlan {
  bool apart;     // as if nothing were shared
  bool chunk[2];  // the kernel over the prefixes, and over the rest; one launch where it is the same one
};

// Lengths are on the device, so what the caller says that prefixes are at most decides, or
// the keys that the page table has room for. (Where a table has room for much more and no
// bound is given, to share is the smaller mistake: behind a table for 32768 keys, 64 sequences
// of up to 400 keys behind 100 36 us, apart 24, chunks of 250 tokens behind 1024 86, 59, but
// 64 single tokens behind 16384, d = 256, 246, apart 628.)
//
// The kernel over the prefixes: few_kernel reads them again for every 16 rows, chunk_kernel
// is a launch of its own. 16 sequences of 32 / 8 heads behind 8192 keys (64 rows): 29.5 us,
// with chunk_kernel 32.4, e4m3 26.7, 34.8; 32 behind 32768 (128 rows) 142, 60; e4m3 107, 66.
//
// Whether to share at all, by what it spares at most against what it costs. Few rows a
// sequence: the prefixes' bytes, against parts and their joining (2 us, where units that share
// nothing stay whole) or a second kernel too (30 us): 8 sequences behind 128 keys 11.1 us,
// apart 9.0, 2 behind 1021 10.7, 12.3, 8 behind 8192 20.8, 41; 64 of 400 keys behind 100 37.6, 20.9.
// (Units that are divided anyway cost nothing more: 2 sequences of up to 12000 keys behind 512
// 20.9 us, apart 19.7, 8 of 4000 behind 512 22.2, 22.8, 16 of 1000 behind 2048 19.9, 26.7.)
// Chunks: products are not spared, but a group's rows fill the tiles of 256 rows, where each
// sequence's last one is half empty on average, or emptier; that against the joining of all
// rows, and short units (4 tiles' time each). 32 chunks of 160 rows behind 8192 keys 146 us,
// apart 190, of 256 221, 291; of 160 behind 2048 73, 53; 8 of 1000 behind 4096 153, 112,
// behind 16384 409, 415, behind 30000 713, 775.
//
// Chunks where chunk_kernel has no form (d = 256): few_kernel's units of 16 rows are full either
// way, and ranges that start anywhere in a prefix read it from L2 at two thirds of the rate of
// units that start together (32 sequences of 30 tokens of 16 / 4 heads behind 8192 keys 2006 us,
// apart 1299, e4m3 1303, 779; of 5 tokens 319, 272, e4m3 225, 171). What sharing brings there is
// that units are divided where whole ones, about 0.5 us a tile, would leave most CTAs idle: 4
// sequences of 9 tokens of 8 / 4 heads behind 655 keys, e4m3, 18.0, apart 23.2. Long ones are
// divided either way; sharing still gains with very few units (3 of 8 tokens of 4 / 1 heads
// behind 4187 19.0, 24.6), not with more (4 of 18 of 16 / 4 behind 8192 164, 113).
SharedPlan shared_plan(const fm_kv_cache& c, const fm_paged_batch& b, const fm_shared_prefix& x, int T, int H_q,
                       const fm_rows* q) {
  SharedPlan p = {};
  const int S = x.S, room = b.width * c.page_size;
  const double rows = (double)T * (H_q / c.H_kv);
  const double keys = (x.max_prefix > 0 ? std::min(x.max_prefix, room) : room) & -c.page_size;  // whole pages
  p.chunk[1] = use_chunk(c, b, T, H_q, q);
  fm_paged_batch groups = b;
  groups.R = S;
  p.chunk[0] = p.chunk[1] || (use_chunk(c, groups, T, H_q, q) && rows > 64.0 * S);
  double spared, cost;  // microseconds
  if (rows <= 16.0 * b.R) {
    const double row = c.k_exp ? c.d + 1.0 : 2.0 * c.d;
    spared = std::max(0, b.R - S) * keys * 2 * c.H_kv * row / 6.5e6;
    cost = p.chunk[0] != p.chunk[1] ? 30 : shape_of(c, b, T, H_q, 1, 0, 0, false).whole ? 2 : 0;
  } else if (p.chunk[1]) {
    const double tile = 1.5 / sm_count(), fill = rows / b.R / 256;
    spared = std::max(0, b.R - S) * std::max(0.5, 1 - fill) * c.H_kv * keys / 128 * tile;
    cost = 12 + 0.0005 * T * H_q + b.R * std::ceil(fill) * c.H_kv * 4 * tile;
  } else {
    const double units = b.R * std::ceil(rows / b.R / kFewRows) * c.H_kv;
    const double busy = units / (sm_count() * few_ctas(c.d, c.k_exp != nullptr));
    const double whole = keys / kTileKeys * 0.5 * c.d / 256;  // a unit's time
    spared = whole > 32 && busy > 0.125 ? 0 : std::max(0, b.R - S) / (double)b.R * (1 - 1.5 * busy) * whole;
    cost = 3;
  }
  p.apart = spared <= cost;
  return p;
}

PagedShape shared_shape(const fm_kv_cache& c, const fm_paged_batch& b, int S, int T, int H_q, int causal, bool chunk,
                        int kinds) {
  PagedShape s = shape_of(c, b, T, H_q, causal, 0, 0, chunk);
  const long long units = ((long long)T * s.G + s.step - 1) / s.step;  // of each kind, and one a sequence
  const long long most = ((long long)b.width * s.page + s.tile - 1) / s.tile;
  s.S = S;
  s.kinds = kinds;
  // what starting on a unit costs, in tiles (chunks of 20 to 60 tokens behind 8192 keys 157 us, with 2
  // 196: short units of many rows; 6 and 8 as 4)
  if (chunk) s.extra = 4;
  const bool rest = !chunk && kinds == 2;  // (kRest)
  s.ctas = marked_workers(s.ctas, rest ? few_warps(c.d, c.k_exp != nullptr) : 1);
  if (rest) {
    s.least = 1;
    s.extra = 4;
  }
  s.V = (kinds & 1 ? S : 0) + (kinds & 2 ? b.R : 0);
  s.max_units = (kinds == 3 ? 2 : 1) * units + s.V;
  s.whole = 0;
  s.local = std::max(s.V, S) <= (chunk ? kSharedChunks : kLocalSeqs) && s.max_units - s.V <= kLocalUnits &&
            s.max_units * (most + s.extra) * s.H_kv * (s.ctas + 1) < (1ll << 31);
  return s;
}

// The workspace: full results and where the others are, then each launch's own.
struct SharedWork {
  SharedOut sh;
  PagedShape s[2];
  PagedWork w[2];
  int launches;
  size_t bytes;
};

SharedWork shared_work(const SharedPlan& p, const fm_kv_cache& c, const fm_paged_batch& b, int S, int T, int H_q,
                       int causal, void* ws) {
  SharedWork k = {};
  char* at = reinterpret_cast<char*>(round256(reinterpret_cast<uintptr_t>(ws)));
  size_t o = 0;
  auto take = [&](size_t bytes) {
    char* x = at ? at + o : nullptr;
    o += round256(bytes);
    return x;
  };
  const size_t rows = (size_t)T * H_q;
  k.sh.rows = (long long)rows;
  k.sh.full = reinterpret_cast<float*>(take(2 * rows * c.d * sizeof(float)));
  k.sh.full_ml = reinterpret_cast<float2*>(take(2 * rows * sizeof(float2)));
  k.sh.where = reinterpret_cast<uint32_t*>(take(2 * rows * sizeof(uint32_t)));
  k.launches = p.chunk[0] == p.chunk[1] ? 1 : 2;
  for (int i = 0; i < k.launches; ++i) {
    k.s[i] = shared_shape(c, b, S, T, H_q, causal, p.chunk[i], k.launches == 1 ? 3 : i + 1);
    const int slot = p.chunk[i] ? kChunkRows : kFewRows;
    const size_t bytes = paged_work(k.s[i], slot, nullptr).bytes;
    char* x = take(bytes);
    k.w[i] = paged_work(k.s[i], slot, x);
  }
  k.bytes = o + 255;
  return k;
}

template <int D>
cudaError_t launch_merge(const MergeParams& m, double parts, cudaStream_t st) {
  auto go = [&](auto kernel, int rows, int per_sm) {  // rows of a block's step
    const long long blocks = (m.sh.rows + rows - 1) / rows, most = (long long)sm_count() * per_sm;
    count_launches(1);
    return launch_dependent(kernel, dim3((unsigned)std::min(blocks, most)), 256, 0, st, m);
  };
  constexpr int RPW = D == 64 ? 2 : 1;
  return parts > 9 ? go(merge_kernel<D, 4>, 2 * RPW, merge_blocks(D, 4))
                   : go(merge_kernel<D, 1>, 8 * RPW, merge_blocks(D, 1));
}

}  // namespace

size_t shared_ws_bytes(const fm_kv_cache& c, const fm_paged_batch& b, const fm_shared_prefix& x, int T, int H_q) {
  // of every way a call of these sizes may run: it goes by the queries' strides too
  const fm_rows broadcast{nullptr, 0, 0};
  size_t bytes = paged_ws_bytes(c, b, T, H_q);
  for (const fm_rows* q : {(const fm_rows*)nullptr, &broadcast}) {
    const SharedPlan p = shared_plan(c, b, x, T, H_q, q);
    if (!p.apart) bytes = std::max(bytes, shared_work(p, c, b, x.S, T, H_q, 1, nullptr).bytes);
  }
  return bytes;
}

cudaError_t launch_shared(const fm_kv_cache& c, const fm_paged_batch& b, const fm_shared_prefix& x, int T, int H_q,
                          const fm_rows& q, const fm_rows& o, float* lse, float scale, int causal, void* ws,
                          cudaStream_t st, int* err) {
  const SharedPlan p = shared_plan(c, b, x, T, H_q, &q);
  if (p.apart) return launch_paged(c, b, T, H_q, q, o, lse, scale, causal, 0, 0, ws, st, err);
  const SharedWork k = shared_work(p, c, b, x.S, T, H_q, causal, ws);
  const PagedOut out{static_cast<char*>(o.ptr), o.st, o.sh, lse, H_q};
  const PagedLists in{b.q_off, b.kv_len, x.seq_off, x.prefix_len};
  MergeParams m = {};
  m.out = out;
  m.sh = k.sh;
  m.q_off = b.q_off;
  m.R = b.R;
  m.T = T;
  double parts = 0;
  for (int i = 0; i < k.launches; ++i) {
    const cudaError_t e =
        launch_attention<true>(p.chunk[i], k.s[i], k.w[i], c, in, b.page_table, q, out, k.sh, scale, st, err);
    if (e != cudaSuccess) return e;
  }
  for (int kind = 0; kind < 2; ++kind) {
    const int i = k.launches == 1 ? 0 : kind;
    const PagedShape& s = k.s[i];
    m.part[kind] = k.w[i].part;
    m.part_floats[kind] = k.w[i].part_floats;
    m.slot_rows[kind] = p.chunk[i] ? kChunkRows : kFewRows;
    m.ctas[kind] = s.ctas;
    // CTAs that a unit and head is divided among, about
    const double units = std::max((double)(kind ? b.R : x.S), (double)T * s.G / s.step) * s.H_kv;
    parts += std::min(s.ctas / units, (double)b.width * s.page / s.tile / s.least) + 1;
  }
  return c.d == 64    ? launch_merge<64>(m, parts, st)
         : c.d == 128 ? launch_merge<128>(m, parts, st)
                      : launch_merge<256>(m, parts, st);
}

}  // namespace fm
