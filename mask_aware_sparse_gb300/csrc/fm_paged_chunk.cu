// fm_paged_chunk.cu — attention of new tokens over the paged cache with many
// query rows a KV head (chunks of prompts, wide groups): tcgen05 + TMEM + TMA.
//
// A unit is up to two tiles of 128 query rows of one sequence and KV head. A
// tile's rows are whole tokens, each with its G query heads of the group (one
// 4-D TMA box: d, head of the group, KV head, token), so all heads that share a
// key tile's load share its products too, and a short chunk fills a tile with
// heads. Keys come in tiles of 128, page by page, into a two-stage ring (d = 64:
// four) shared by both query tiles. Bound by the tensor core and the softmax,
// as the dense forward; with a single tile's few rows by memory.
//
//   warps 0-3, 4-7  softmax of query tile 0, 1: a thread a row
//   warp 8          producer (TMA); warp 9: MMA issue and TMEM
//   warps 12-15, 16-19  e4m3 caches: the bytes of a tile's keys, and of its values,
//                   to bf16, times the row's scale, exact (a thread a row), from a
//                   staging ring to the bf16 ring the tensor core reads
//
// TMEM: S_0, S_1 (128 columns each; P overwrites S as bf16), O_0, O_1. With two
// query tiles the tensor core works on one while the softmax works on the
// other. A unit with one tile uses both S buffers for it, alternating, with the
// next tile's S issued ahead of this one's P V. Products are issued by one
// thread and run in order: what reads a buffer is issued before what
// overwrites it. The running maximum moves only when passed by more than 8
// (log2 units). Masks are intervals of keys per row, four 32-bit words a tile,
// built only for tiles that some row of the warp sees in part. Warps whose rows
// are all past the unit's end only keep the barriers going.
//
// Values of keys that no row of the unit sees (the end of the last page may hold
// anything) are overwritten with zeros in shared memory before the product that
// would read them: 0 * NaN is NaN.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cuda.h>
#include <cuda_bf16.h>
#include "fm_internal.h"
#include "paged.cuh"
#include "sm100.cuh"

namespace fm {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kLn2C = 0.69314718055994530942f;

template <int D, bool F8>
struct ChunkCfg {
  // e4m3: warpgroups that widen tiles, and the registers that the launch's are
  // redistributed into: d = 128: 20 warps at 96, 8 softmax warps at 168, 12 others
  // at 48 (one group, 16 warps: a 2048-token chunk over 32768 keys 1031 us instead
  // of 936); d = 64, half as much to widen for each product: 16 warps at 128, 184 and
  // 72 (two groups: ragged chunks of 1111 tokens 31.8 us instead of 30.2, 20 of 4000 tokens
  // over up to 8000 keys 137 instead of 132, 2048 tokens over 32768 keys 681 instead of 685)
  static constexpr int WIDEN = !F8 ? 0 : D == 128 ? 2 : 1;
  static constexpr int SOFTMAX_REGS = WIDEN == 2 ? 168 : 184, OTHER_REGS = WIDEN == 2 ? 48 : 72;
  static constexpr int THREADS = F8 ? 384 + 128 * WIDEN : 320;
  static constexpr int TILE = 128 * D * 2;
  static constexpr int BOXES = D / 64;
  static constexpr int STAGES = D == 64 ? 4 : 2;
  static constexpr int RAW = 128 * D, RAWS = F8 ? (D == 64 ? 4 : 2) : 0;
  static constexpr int K_OFF = 2 * TILE;
  static constexpr int V_OFF = K_OFF + STAGES * TILE;
  static constexpr int RAW_OFF = V_OFF + STAGES * TILE;
  static constexpr int EXP_OFF = RAW_OFF + RAWS * RAW;
  static constexpr int BAR_OFF = EXP_OFF + RAWS * 128;
  static constexpr int QFULL = 0, QFREE = 1, SFULL = 2, PREADY = 4;  // two tiles: [tile]
  static constexpr int SSFULL = 6, SPREADY = 8;                      // one tile: [S buffer]
  static constexpr int ODONE = 10, OEND = 12;                        // [tile]
  static constexpr int KFULL = 14, KEMPTY = KFULL + STAGES, VFULL = KEMPTY + STAGES, VEMPTY = VFULL + STAGES;
  static constexpr int RFULL = VEMPTY + STAGES, REMPTY = RFULL + RAWS;
  static constexpr int MEND = REMPTY + RAWS;  // all products done
  static constexpr int NBAR = MEND + 1;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int SMEM = MISC_OFF + 16 + 1024;
};

struct ChunkParams {
  PagedShape s;
  PagedWork w;
  PagedOut out;
  const uint8_t* k_exp;
  const uint8_t* v_exp;
  const int32_t* q_off;
  const int32_t* kv_len;
  const int32_t* table;
  int tile_rows;  // rows of a query tile: whole tokens, at most 128
  int wide;       // output rows start on 32-byte boundaries
  float scale_log2;
  int* err;
};

__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, uint64_t* bar, int32_t x, int32_t y, int32_t z,
                                            int32_t w) {
  if (!FM_DBG(smem_range(smem_u32(dst), 16, 128) && smem_range(smem_u32(bar), 8, 8) && (x & 7) == 0)) return;
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// The low n bits (n clamped to [0, 32]).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

template <int D, bool F8>
__global__ void __launch_bounds__(ChunkCfg<D, F8>::THREADS, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                 const __grid_constant__ CUtensorMap tv, const ChunkParams p) {
  using C = ChunkCfg<D, F8>;
  constexpr int S = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  FM_DEBUG_BEGIN();
  if (threadIdx.x == 0) {
    mbar_init(&bars[C::QFULL], 1);
    mbar_init(&bars[C::QFREE], 1);
    mbar_init(&bars[C::MEND], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[C::SFULL + i], 1);
      mbar_init(&bars[C::PREADY + i], 128);
      mbar_init(&bars[C::SSFULL + i], 1);
      mbar_init(&bars[C::SPREADY + i], 128);
      mbar_init(&bars[C::ODONE + i], 1);
      mbar_init(&bars[C::OEND + i], 1);
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(&bars[C::KFULL + i], F8 ? 4 : 1);
      mbar_init(&bars[C::KEMPTY + i], 1);
      mbar_init(&bars[C::VFULL + i], F8 ? 4 : 1);
      mbar_init(&bars[C::VEMPTY + i], 1);
    }
    for (int i = 0; i < C::RAWS; ++i) {
      mbar_init(&bars[C::RFULL + i], 1);
      mbar_init(&bars[C::REMPTY + i], 4);
    }
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc<512>(tmem_slot);
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  __shared__ PagedStart start;
  __shared__ int4 seq[kLocalChunks];
  __shared__ uint16_t first[kLocalChunks + 1], order[kWholeUnits];
  grid_dependency_wait();
  grid_launch_dependents();
  if (threadIdx.x == 0) *abort_flag = timeout_pending(p.err) ? 1 : 0;  // (the kernel before may have set it)
  // (the plans' scratch lies where the first keys will)
  if (p.s.whole) {
    plan_whole(p.s, p.q_off, p.kv_len, seq, first, order, reinterpret_cast<uint16_t*>(smem + C::K_OFF), &start, p.err);
  } else if (p.s.local) {
    plan_locally(p.s, p.q_off, p.kv_len, seq, reinterpret_cast<unsigned*>(smem + C::K_OFF), &start, p.err);
    if (threadIdx.x == 0) p.w.starts[blockIdx.x] = start;  // for join_kernel
  } else {
    if (threadIdx.x == 0) start = p.w.starts[blockIdx.x];
  }
  fence_proxy_async_smem();
  __syncthreads();
  const int G = p.s.G, TR = p.tile_rows;
  bool ok = *abort_flag == 0;
  PagedWalk walk(p.s, p.w.units, seq, first, order, start);

  if (!ok) {
    // an unread timeout of an earlier launch: nothing is computed
  } else if (warp < 8) {
    if constexpr (F8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX_REGS));
    // ------------------------------------------------------------- softmax
    const int t = warp >> 2;
    const int row = ((warp & 3) << 5) + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tbase + lane_off + 256u + (uint32_t)(t * D);
    const float sl2 = p.scale_log2;
    uint32_t jt = 0, jh = 0, ends = 0;  // key tiles of the CTA, of this query tile, ended segments of this tile
    uint32_t nf = 0, nsf0 = 0, nsf1 = 0;  // waits done on SFULL[t], SSFULL[0, 1]
    for (; walk.more() && ok; walk.next()) {
      const PagedUnit& u = walk.u;
      const int n = walk.n, T = u.nrows > TR ? 2 : 1;
      const int rr = t * TR + row;  // row of the unit
      const bool live = row < TR && rr < u.nrows;
      const bool warp_live = ((warp & 3) << 5) < TR && t * TR + ((warp & 3) << 5) < u.nrows;
      const int ps = u.pos + rr / G;
      const int64_t tok = u.tok + rr / G;
      const int head = walk.h * G + rr % G;
      // this row sees keys [0, hi) that are at lo or above, or sinks
      // (rows past the unit: all of them, so that they ask for no masks; nothing of them is kept)
      const int hi = !live ? 1 << 30 : p.s.causal ? min(max(ps + 1, 0), u.kv_len) : u.kv_len;
      const int lo = live && p.s.window > 0 ? ps - p.s.window + 1 : 0;
      float m_run = -INFINITY, l_run = 0.f;
      if (n > 0 && t >= T) {
        jt += n;
        continue;
      }
      for (int j = 0; j < n; ++j, ++jt, ++jh) {
        const int key0 = tile_of(u, walk.kt + j) * 128;
        uint32_t buf, ph;
        uint64_t* full;
        if (T == 2) {
          buf = t;
          full = &bars[C::SFULL + t];
          ph = nf++;
        } else {
          buf = j & 1;
          full = &bars[C::SSFULL + buf];
          ph = buf ? nsf1++ : nsf0++;
        }
        ok = __all_sync(kAll, mbar_wait(full, ph & 1u, abort_flag, p.err));
        if (!ok) break;
        tc_fence_after();
        if (!F8 && t == 0) {
          // values of keys that no row of the unit sees
          const bool edge = key0 + 128 > u.hi || (p.s.window > 0 && key0 < u.lo && key0 + 128 > p.s.sinks);
          if (edge) {
            const int slot = jt % S, key = key0 + row;
            ok = __all_sync(kAll, mbar_wait(&bars[C::VFULL + slot], (jt / S) & 1u, abort_flag, p.err));
            if (!ok) break;
            if (!(key < u.hi && (key >= u.lo || key < p.s.sinks))) {
              const uint32_t at = smem_u32(smem + C::V_OFF + slot * C::TILE) + row * 128;
#pragma unroll
              for (int b = 0; b < C::BOXES; ++b)
#pragma unroll
                for (int c = 0; c < 8; ++c) sts_b32x4(at + b * 16384 + 16 * c, 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
        }
        if (warp_live) {
          const uint32_t tS = tbase + lane_off + (buf << 7);
          uint32_t sr[128];
#pragma unroll
          for (int c = 0; c < 128; c += 32) tmem_ld32(tS + c, *reinterpret_cast<uint32_t(*)[32]>(&sr[c]));
          tmem_ld_wait();
          const int h_c = hi - key0, l_c = lo - key0, s_c = p.s.sinks - key0;
          if (__any_sync(kAll, h_c < 128 || l_c > 0)) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t vis = low_bits(h_c - 32 * q) & (~low_bits(l_c - 32 * q) | low_bits(s_c - 32 * q));
#pragma unroll
              for (int c = 0; c < 32; ++c)
                sr[32 * q + c] = ((vis >> c) & 1u) ? sr[32 * q + c] : __float_as_uint(-INFINITY);
            }
          }
          float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
          for (int c = 0; c < 128; c += 8) {
            mx0 = max3f(mx0, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
            mx1 = max3f(mx1, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
            mx2 = max3f(mx2, __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
            mx3 = max3f(mx3, __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
          }
          const float m_new = fmaxf(m_run, max3f(mx0, mx1, fmaxf(mx2, mx3)) * sl2);
          const bool resc = m_new > m_run + 8.0f;
          float factor = 1.f;
          if (resc) {
            factor = ex2_approx(m_run - m_new);
            m_run = m_new;
          }
          const float base = (m_run == -INFINITY) ? 0.f : m_run;
          const uint64_t sl2x2 = f2_pack(sl2, sl2), nm2 = f2_pack(-base, -base);
          uint64_t rs0 = f2_pack(0.f, 0.f), rs1 = rs0;
          uint32_t pk[64];
#pragma unroll
          for (int c = 0; c < 64; ++c) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), sl2x2, nm2), x0, x1);
            const float a = ex2_approx(x0), b = ex2_approx(x1);
            if (c & 1)
              rs1 = f2_add(rs1, f2_pack(a, b));
            else
              rs0 = f2_add(rs0, f2_pack(a, b));
            pk[c] = pack_bf16x2(a, b);
          }
          float r0a, r0b, r1a, r1b;
          f2_unpack(rs0, r0a, r0b);
          f2_unpack(rs1, r1a, r1b);
          l_run = l_run * factor + ((r0a + r0b) + (r1a + r1b));
#pragma unroll
          for (int c = 0; c < 64; c += 16) tmem_st16(tS + c, *reinterpret_cast<uint32_t(*)[16]>(&pk[c]));
          tmem_st_wait();
          if (j > 0 && __any_sync(kAll, resc)) {
            // O holds the products of the tiles before: wait for the last of them
            ok = __all_sync(kAll, mbar_wait(&bars[C::ODONE + t], (jh - 1) & 1u, abort_flag, p.err));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t r[32];
              tmem_ld32(tO + c0, r);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 32; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * factor);
              tmem_st32(tO + c0, r);
            }
            tmem_st_wait();
          }
        }
        tc_fence_before();
        mbar_arrive(&bars[(T == 2 ? C::PREADY + t : C::SPREADY + buf)]);
      }
      if (!ok) break;
      if (n > 0) {
        ok = __all_sync(kAll, mbar_wait(&bars[C::OEND + t], ends & 1u, abort_flag, p.err));
        ++ends;
        if (!ok) break;
        tc_fence_after();
      }
      if (!warp_live) continue;
      // The row's result, 32 columns at a time: O / l, or the partial sums. A lane's
      // row is its own, so a store of 16 bytes a lane would touch every sector twice:
      // whole sectors (32 bytes) where the output allows.
      const bool whole = walk.whole();
      const float inv = l_run > 0.f ? 1.f / l_run : (l_run == 0.f ? 0.f : l_run);
      char* dst = p.out.o + 2 * (tok * p.out.st + head * p.out.sh);
      float* part = p.w.part + p.w.part_floats * (2 * (size_t)blockIdx.x + walk.slot());
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t r[32];
        if (n > 0) {
          tmem_ld32(tO + c0, r);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) r[c] = 0u;
        }
        if (!live) continue;
        const float* f = reinterpret_cast<const float*>(r);
        if (whole) {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) w[c] = pack_bf16x2(f[2 * c] * inv, f[2 * c + 1] * inv);
          if (p.wide) {
#pragma unroll
            for (int c = 0; c < 16; c += 8)
              stg_b32x8(dst + 2 * c0 + 4 * c, w[c], w[c + 1], w[c + 2], w[c + 3], w[c + 4], w[c + 5], w[c + 6],
                        w[c + 7]);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              reinterpret_cast<uint4*>(dst + 2 * c0)[c] =
                  make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
          }
        } else {
          float* at = part + (size_t)rr * D + c0;
#pragma unroll
          for (int c = 0; c < 32; c += 8)
            stg_b32x8(at + c, r[c], r[c + 1], r[c + 2], r[c + 3], r[c + 4], r[c + 5], r[c + 6], r[c + 7]);
        }
      }
      if (live) {
        if (whole) {
          p.out.lse[tok * p.out.H_q + head] = l_run == 0.f ? -INFINITY : m_run * kLn2C + logf(l_run);
        } else {
          float* ml = part + (size_t)(2 * 128) * D + 2 * rr;
          ml[0] = m_run;
          ml[1] = l_run;
        }
      }
    }
  } else if (warp < 12) {
    if constexpr (F8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    if (warp == 8) {
      // ------------------------------------------------------------- producer
      const int P = p.s.page, rows = P, per = 128 >> p.s.page_log;  // P <= 128
      const int zmax = p.s.n_pages * p.s.H_kv;
      uint32_t jt = 0, seg = 0;  // key tiles, segments with keys so far
      uint32_t asked = 0, asked_q = 0;  // tiles of keys and of values, and of queries, whose copies were started
      PageWindow pages;
      for (; walk.more() && ok; walk.next()) {
        if (walk.n == 0) continue;
        const PagedUnit& u = walk.u;
        const int T = u.nrows > TR ? 2 : 1;
        pages.reset(p.table, u.r, p.s.width);
        if (lane == 0) {
          // the unit's queries, once the last S of the segment before is done
          if (seg > 0) ok = mbar_wait(&bars[C::QFREE], (seg - 1) & 1u, abort_flag, p.err);
          if (ok) {
            mbar_arrive_expect_tx(&bars[C::QFULL], T * TR * D * 2);
            for (int t = 0; t < T; ++t)
              for (int x = 0; x < C::BOXES; ++x)
                tma_load_4d(smem + t * C::TILE + x * 16384, &tq, &bars[C::QFULL], x * 64, 0, walk.h,
                            u.tok + t * (TR / G));
            ++asked_q;
          }
        }
        ok = __shfl_sync(kAll, ok, 0);
        ++seg;
        for (int j = 0; j < walk.n && ok; ++j, ++jt) {
          const int key0 = tile_of(u, walk.kt + j) * 128;
          const int pg0 = key0 >> p.s.page_log;
          pages.hold(pg0, per, lane);
          const int boxes = min(per, (u.kv_len - key0 + rows - 1) >> p.s.page_log);
          // lane i copies the i-th box of the tile's keys (x fastest), then of its values
          constexpr int XS = F8 ? 1 : C::BOXES;
          const int b = min(lane / XS, boxes - 1), x = lane % XS;
          const int pg = __shfl_sync(kAll, pages.held, pg0 + b - pages.base);
          const bool mine = lane < boxes * XS;
          const bool good = pg >= 0 && pg < p.s.n_pages;
          if (mine && !good && any_seen(p.s, u, key0 + b * rows, key0 + (b + 1) * rows))
            record_error(p.err, FM_DEV_ERR_RANGE);
          const int z = good ? pg * p.s.H_kv + walk.h : zmax;  // zmax: out of range, reads as zero
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            uint64_t *fb, *eb;
            uint32_t ph;
            uint8_t* at;
            if constexpr (F8) {
              const uint32_t ri = 2 * jt + v;
              fb = &bars[C::RFULL + ri % C::RAWS];
              eb = &bars[C::REMPTY + ri % C::RAWS];
              ph = (ri / C::RAWS) & 1u;
              at = smem + C::RAW_OFF + (ri % C::RAWS) * C::RAW;
            } else {
              fb = &bars[(v ? C::VFULL : C::KFULL) + jt % S];
              eb = &bars[(v ? C::VEMPTY : C::KEMPTY) + jt % S];
              ph = (jt / S) & 1u;
              at = smem + (v ? C::V_OFF : C::K_OFF) + (jt % S) * C::TILE;
            }
            ok = __all_sync(kAll, mbar_wait(eb, ph ^ 1u, abort_flag, p.err));
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(fb, boxes * rows * (F8 ? D + 1 : 2 * D));
            __syncwarp();
            ++asked;
            if (mine) {
              if constexpr (F8) {
                tma_load_3d(at + b * rows * D, v ? &tv : &tk, fb, 0, key0 - pg0 * P, z);
                bulk_load(smem + C::EXP_OFF + ((2 * jt + v) % C::RAWS) * 128 + b * rows,
                          (v ? p.v_exp : p.k_exp) + (int64_t)(good ? z : walk.h) * P + (key0 - pg0 * P), rows, fb);
              } else {
                tma_load_3d(at + x * 16384 + b * rows * 128, v ? &tv : &tk, fb, x * 64, key0 - pg0 * P, z);
              }
            }
          }
        }
      }
      if (lane == 0) {
        // The CTA ends with no copy in flight, however its other warps end: the last ones
        // have landed, or a second bound passed.
        volatile int none = 0;
        constexpr uint32_t kRing = F8 ? C::RAWS : 2 * S;
        if (asked_q > 0) mbar_wait(&bars[C::QFULL], (asked_q - 1) & 1u, &none, p.err);
        for (uint32_t r = asked > kRing ? asked - kRing : 0; r < asked; ++r) {
          uint64_t* full = F8 ? &bars[C::RFULL + r % kRing] : &bars[(r & 1 ? C::VFULL : C::KFULL) + (r >> 1) % S];
          mbar_wait(full, (r / kRing) & 1u, &none, p.err);
        }
      }
    } else if (warp == 9) {
      // --------------------------------------------------------- MMA issue
      // (elected, not lane 0: the compiler then knows that one thread runs and keeps what
      // the products take in uniform registers: 2048 tokens over 32768 keys, ten calls in a
      // graph, 653 us instead of 764; called for a second on end, at the power cap, 760)
      if (elect_one()) {
        const uint32_t id_s = idesc_bf16_f32(128, 128, 0, 0), id_o = idesc_bf16_f32(128, D, 0, 1);
        const uint64_t dQ = sdesc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t dK = sdesc_sw128(smem_u32(smem + C::K_OFF), 16, 1024);
        const uint64_t dV = sdesc_sw128(smem_u32(smem + C::V_OFF), 16384, 1024);
        constexpr uint64_t kStep = C::TILE >> 4;
        uint32_t jt = 0, seg = 0, np0 = 0, np1 = 0, ns0 = 0, ns1 = 0;  // waits done on PREADY[0, 1], SPREADY[0, 1]
        auto issue_s = [&](int t, int slot, int buf, uint64_t* full) {
          const uint64_t qd = dQ + kStep * (uint64_t)t, kd = dK + kStep * (uint64_t)slot;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t off = (uint64_t)((k >> 2) * 1024 + (k & 3) * 2);
            mma_ss(tbase + (uint32_t)(buf * 128), qd + off, kd + off, id_s, k > 0 ? 1u : 0u);
          }
          mma_commit(full);
        };
        auto issue_pv = [&](int t, int slot, int buf, bool first, uint64_t* ready, uint32_t& count) -> bool {
          if (!mbar_wait(ready, count & 1u, abort_flag, p.err)) return false;
          ++count;
          tc_fence_after();
          const uint64_t vd = dV + kStep * (uint64_t)slot;
          const uint32_t tO = tbase + 256u + (uint32_t)(t * D);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ts(tO, tbase + (uint32_t)(buf * 128 + k * 8), vd + (uint64_t)(k * 128), id_o,
                   (!first || k > 0) ? 1u : 0u);
          mma_commit(&bars[C::ODONE + t]);
          return true;
        };
        for (; walk.more() && ok; walk.next()) {
          const int n = walk.n;
          if (n == 0) continue;
          const bool two = walk.u.nrows > TR;
          ok = mbar_wait(&bars[C::QFULL], seg & 1u, abort_flag, p.err);
          ++seg;
          tc_fence_after();
          if (two) {
            for (int j = 0; j < n && ok; ++j, ++jt) {
              const int slot = jt % S, prev = (jt - 1) % S;
              ok = mbar_wait(&bars[C::KFULL + slot], (jt / S) & 1u, abort_flag, p.err);
              if (ok && j > 0) ok = mbar_wait(&bars[C::VFULL + prev], ((jt - 1) / S) & 1u, abort_flag, p.err);
              tc_fence_after();
              if (!ok) break;
              if (j > 0 && !(ok = issue_pv(0, prev, 0, j == 1, &bars[C::PREADY], np0))) break;
              issue_s(0, slot, 0, &bars[C::SFULL]);
              if (j > 0 && !(ok = issue_pv(1, prev, 1, j == 1, &bars[C::PREADY + 1], np1))) break;
              issue_s(1, slot, 1, &bars[C::SFULL + 1]);
              if (j > 0) mma_commit(&bars[C::VEMPTY + prev]);
              mma_commit(&bars[C::KEMPTY + slot]);
              if (j == n - 1) mma_commit(&bars[C::QFREE]);
            }
          } else {
            for (int j = 0; j < n && ok; ++j, ++jt) {
              const int slot = jt % S, prev = (jt - 1) % S, buf = j & 1;
              ok = mbar_wait(&bars[C::KFULL + slot], (jt / S) & 1u, abort_flag, p.err);
              tc_fence_after();
              if (!ok) break;
              issue_s(0, slot, buf, &bars[C::SSFULL + buf]);
              mma_commit(&bars[C::KEMPTY + slot]);
              if (j == n - 1) mma_commit(&bars[C::QFREE]);
              if (j > 0) {
                ok = mbar_wait(&bars[C::VFULL + prev], ((jt - 1) / S) & 1u, abort_flag, p.err);
                tc_fence_after();
                if (ok) ok = issue_pv(0, prev, buf ^ 1, j == 1, &bars[C::SPREADY + (buf ^ 1)], buf ? ns0 : ns1);
                if (ok) mma_commit(&bars[C::VEMPTY + prev]);
              }
            }
          }
          if (!ok) break;
          // the segment's last P V; the softmax warps wait for exactly this one (OEND)
          const int last = (jt - 1) % S;
          ok = mbar_wait(&bars[C::VFULL + last], ((jt - 1) / S) & 1u, abort_flag, p.err);
          tc_fence_after();
          if (!ok) break;
          if (two) {
            if (!(ok = issue_pv(0, last, 0, n == 1, &bars[C::PREADY], np0))) break;
            mma_commit(&bars[C::OEND]);
            if (!(ok = issue_pv(1, last, 1, n == 1, &bars[C::PREADY + 1], np1))) break;
            mma_commit(&bars[C::OEND + 1]);
          } else {
            const int buf = (n - 1) & 1;
            if (!(ok = issue_pv(0, last, buf, n == 1, &bars[C::SPREADY + buf], buf ? ns1 : ns0))) break;
            mma_commit(&bars[C::OEND]);
          }
          mma_commit(&bars[C::VEMPTY + last]);
        }
        // nor with a product in flight, which would use its memory after it
        volatile int none = 0;
        mma_commit(&bars[C::MEND]);
        mbar_wait(&bars[C::MEND], 0u, &none, p.err);
      }
    }
  } else if constexpr (F8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    // -------------------------------------------------- e4m3 tiles to bf16
    constexpr int ROW = D;  // bytes of a staged row: 128 or 64, swizzled as wide
    const int row = threadIdx.x & 127;
    uint32_t jt = 0;
    for (; walk.more() && ok; walk.next()) {
      const PagedUnit& u = walk.u;
      for (int j = 0; j < walk.n && ok; ++j, ++jt) {
        const int key = tile_of(u, walk.kt + j) * 128 + row;
        // rows that no query of the unit sees become zeros, whatever they hold
        const bool dead = !(key < u.hi && (key >= u.lo || key < p.s.sinks));
        // keys and values in turn, or, with two groups, keys the first and values the second
#pragma unroll 1
        for (int v = (warp - 12) >> 2; v < 2 && ok; v += C::WIDEN) {
          const uint32_t ri = 2 * jt + v, rs = ri % C::RAWS;
          ok = __all_sync(kAll, mbar_wait(&bars[C::RFULL + rs], (ri / C::RAWS) & 1u, abort_flag, p.err));
          if (ok)
            ok = __all_sync(
                kAll, mbar_wait(&bars[(v ? C::VEMPTY : C::KEMPTY) + jt % S], ((jt / S) & 1u) ^ 1u, abort_flag, p.err));
          if (!ok) break;
          const uint32_t src = smem_u32(smem + C::RAW_OFF + rs * C::RAW);
          const uint32_t dst = smem_u32(smem + (v ? C::V_OFF : C::K_OFF) + (jt % S) * C::TILE) + row * 128;
          const uint32_t e = lds8(smem_u32(smem + C::EXP_OFF) + rs * 128 + row);
          const uint32_t fl = dead ? 0u : factor_lo(e) * 0x10001u;  // (the bits it multiplies are finite)
          const bool wide = __any_sync(kAll, !dead && e > 134u && e < 255u);
          // 64 bytes of the row at a time: the staged tile is free for the next one as soon as
          // the last of them are in registers (its load is otherwise waited for: 2048 tokens
          // over 32768 keys, d = 128, 1016 us instead of 936, d = 64 715 instead of 685)
          constexpr int kPart = 4;
          uint32_t top = 0;  // the row's largest magnitudes, before its scale
#pragma unroll
          for (int part = 0; part < D / 64; ++part) {
            uint4 rr[kPart];
#pragma unroll
            for (int c = 0; c < kPart; ++c) rr[c] = lds128(src + in_box<ROW>(row, part * kPart + c));
            if (part == D / 64 - 1) {
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars[C::REMPTY + rs]);
            }
#pragma unroll
            for (int cc = 0; cc < kPart; ++cc) {
              const int c = part * kPart + cc;
              const uint32_t w[4] = {rr[cc].x, rr[cc].y, rr[cc].z, rr[cc].w};
              uint32_t o[8];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t a = __byte_perm(w[x], 0, 0x1404), b = __byte_perm(w[x], 0, 0x3424);
                const uint32_t ma = (a >> 4) & kE4m3Mag, mb = (b >> 4) & kE4m3Mag;
                top = __vimax3_u16x2(top, ma, mb);
                o[2 * x] = mul_bf2(ma | (a & kE4m3Sign), fl);
                o[2 * x + 1] = mul_bf2(mb | (b & kE4m3Sign), fl);
              }
              if (wide) {
                const uint32_t fh = factor_hi(e) * 0x10001u;
#pragma unroll
                for (int x = 0; x < 8; ++x) o[x] = mul_bf2(o[x], fh);
              }
              const uint32_t at = dst + (c >> 2) * 16384;
              const int ch = 2 * (c & 3);
              sts_b32x4(at + (((ch) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
              sts_b32x4(at + (((ch + 1) ^ (row & 7)) << 4), o[4], o[5], o[6], o[7]);
            }
          }
          // The row holds NaN, which was widened like a number, 480, that e4m3 does not have:
          // back to NaN (with it, at scales of 2^120 and more, what bf16 has no number for)
          if (max(top & 0xffffu, top >> 16) == (kE4m3Mag & 0xffffu) && !dead) {
            const uint32_t lo = mul_bf2(kE4m3Mag, fl);
            const uint32_t n480 = (wide ? mul_bf2(lo, factor_hi(e) * 0x10001u) : lo) & 0x7fffu;
#pragma unroll 1
            for (int i = 0; i < D; ++i) {
              const uint32_t at = dst + (i >> 6) * 16384 + ((((i >> 3) & 7) ^ (row & 7)) << 4) + 2 * (i & 7);
              if (((lds8(at) | lds8(at + 1) << 8) & 0x7fffu) == n480) sts_b16(at, 0x7fffu);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[(v ? C::VFULL : C::KFULL) + jt % S]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  FM_DEBUG_END(p.err);
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<512>(tbase);
  }
}

template <int D, bool F8>
cudaError_t launch(const PagedShape& s, const PagedWork& w, const fm_kv_cache& c, const fm_paged_batch& b,
                   const fm_rows& q, const PagedOut& out, float scale, cudaStream_t st, int* err) {
  using C = ChunkCfg<D, F8>;
  static_assert(C::SMEM <= 232448, "chunk_kernel: shared memory of an SM");
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(chunk_kernel<D, F8>), C::SMEM, ready);
  if (e != cudaSuccess) return e;
  const int rows = std::min(s.page, 128), tokens = 128 / s.G;
  CUtensorMap tq, tk, tv;
  if (!make_tmap_tokens(&tq, q, s.T, s.H_kv, s.G, D, tokens) ||
      !make_tmap_pages(&tk, c.k, c, rows, F8 ? D : 128) || !make_tmap_pages(&tv, c.v, c, rows, F8 ? D : 128))
    return cudaErrorInvalidValue;
  const int wide = reinterpret_cast<uintptr_t>(out.o) % 32 == 0 && out.st % 16 == 0 && out.sh % 16 == 0;
  ChunkParams p{s,        w,            out,           c.k_exp, c.v_exp,
                b.q_off,  b.kv_len,     b.page_table,  tokens * s.G,
                wide,     scale * 1.4426950408889634f, err};
  count_launches(1);
  return launch_dependent(chunk_kernel<D, F8>, dim3((unsigned)s.ctas), C::THREADS, C::SMEM, st, tq, tk, tv, p);
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedShape& s, const PagedWork& w, const fm_kv_cache& c, const fm_paged_batch& b,
                               const fm_rows& q, const PagedOut& out, float scale, cudaStream_t st, int* err) {
  const bool f8 = c.k_exp != nullptr;
  if (s.d == 64)
    return f8 ? launch<64, true>(s, w, c, b, q, out, scale, st, err)
              : launch<64, false>(s, w, c, b, q, out, scale, st, err);
  return f8 ? launch<128, true>(s, w, c, b, q, out, scale, st, err)
            : launch<128, false>(s, w, c, b, q, out, scale, st, err);
}

}  // namespace fm
