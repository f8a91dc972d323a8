// paged.cuh — what the kernels of attention over the paged cache share: the
// work units, how a persistent grid divides them, and the partial results of
// units that several CTAs computed.
//
// A unit is a tile of query rows of one sequence (rows = tokens x the query
// heads of a KV head's group, tokens outermost); its work, for each KV head, is
// its list of key tiles. All tiles of all units and heads form one sequence,
// cut into equal ranges, one per CTA: a CTA's range may end inside a unit, so
// ragged batches, one long sequence or many short ones all fill the GPU. A
// range that covers a unit only in part leaves (m, l, O) in a partial slot, and
// the combining kernel joins the slots of such units in CTA order.
#pragma once
#include <atomic>
#include <climits>
#include <cstdint>
#include "dependent.cuh"
#include "fm_internal.h"
#include "sm100.cuh"

namespace fm {

// One tile of query rows. Row i is query head h * G + (g0 + i) % G of token
// tok + (g0 + i) / G, at position pos + (g0 + i) / G.
struct __align__(16) PagedUnit {
  int tok, g0, nrows, pos;
  int r, hi, ns, w0;  // sequence; keys [0, hi) may be visible; tiles [0, ns) hold sinks, then from w0 on
  int ntiles, kv_len, lo, pad;  // lo: keys below it are visible as sinks only
};

// A CTA's range: `count` tiles from tile kt of head h of a unit on. The unit is
// number u of the plan kernel's list, or, where each CTA plans for itself, unit i
// of sequence u.
struct __align__(16) PagedStart {
  int u, i, h, kt, count;
  int first, last;  // where kt > 0: the first and the last CTA with tiles of that unit and head
  int extra;        // places that a unit and head takes besides its tiles'
  PagedUnit unit;
};

struct PagedShape {
  int T, R, H_q, H_kv, G, d, width, page, n_pages;
  int causal, window, sinks;  // window 0: none
  int step, tile;  // query rows of a unit, keys of a tile
  int tile_log, page_log;  // tile = 2^tile_log, page = 2^page_log
  int ctas, least;  // CTAs launched; tiles a CTA gets before another one does
  int extra;  // tiles that a segment's start and end are counted as
  int local;  // every CTA plans for itself: no plan kernel
  int whole;  // no unit and head is divided (every CTA plans for itself): nothing to join
  long long max_units;
};

// Tile number kt of a unit's list.
__device__ __forceinline__ int tile_of(const PagedUnit& u, int kt) { return kt < u.ns ? kt : kt - u.ns + u.w0; }

// The new tokens of sequence r, [a, a + n), kept inside [0, T] whatever q_off
// holds, and its keys, kept inside the page table; true where either was not, or the
// first sequence's tokens do not start at 0.
__device__ __forceinline__ bool sequence_at(const PagedShape& s, const int32_t* q_off, const int32_t* kv_len, int r,
                                            int& a, int& n, int& L) {
  const int b0 = q_off[r], e0 = q_off[r + 1], L0 = kv_len[r];
  a = min(max(b0, 0), s.T);
  const int e = min(max(e0, a), s.T);
  n = e - a;
  L = min(max(L0, 0), s.width * s.page);
  return a != b0 || e != e0 || L != L0 || (r == 0 && b0 != 0);
}

// Unit i of a sequence.
__device__ __forceinline__ PagedUnit unit_at(const PagedShape& s, int r, int a, int n, int L, int i) {
  const int row0 = i * s.step, tok = row0 / s.G;  // T * H_q stays below 2^30
  PagedUnit q;
  q.r = r;
  q.tok = a + tok;
  q.g0 = row0 - tok * s.G;
  q.nrows = min(s.step, n * s.G - row0);
  q.pos = L - n + tok;
  q.kv_len = L;
  const int last = q.pos + (q.g0 + q.nrows - 1) / s.G;
  q.hi = s.causal ? min(max(last + 1, 0), L) : L;
  q.lo = s.window > 0 ? max(0, q.pos - s.window + 1) : 0;
  const int all = (q.hi + s.tile - 1) >> s.tile_log;
  q.ns = s.window > 0 ? min((s.sinks + s.tile - 1) >> s.tile_log, all) : 0;
  q.w0 = max(q.ns, min(q.lo >> s.tile_log, all));
  q.ntiles = q.ns + max(0, all - q.w0);
  q.pad = 0;
  return q;
}

// Some row of the unit sees some of the keys [a, b): only then does it matter which page holds them.
__device__ __forceinline__ bool any_seen(const PagedShape& s, const PagedUnit& u, int a, int b) {
  return a < u.hi && (b > u.lo || a < s.sinks);
}

// Units are divided on a line: each unit and head takes `extra` places, for what
// starting on it costs, then one a tile (one in all where it has none). CTA c of
// `used` gets the tiles that lie on its places, [c total / used, (c + 1) total / used)
// of all of them. Used are all CTAs, or as many as get s.least tiles each; extra is
// then 0, for equal parts (one token over 1021 keys 10.1 us, with 4 11.9). Where all
// have work, CTAs that took up a second or third segment were up to 10 us later than
// the others (a segment's end, the next one's first loads), and the grid waits for them: 32 ragged sequences of up to
// 4096 keys, e4m3: 46.6 us with extra = 0, 43.3 with 10; bf16 62.9, with 4 61.6;
// chunks of 1111 tokens over 3000 keys, e4m3, 38.3, with 3 34.4. Long ranges gain
// less: up to 16384 keys, e4m3, 119.6, 117.5; bf16 199, 202.
// (I: unsigned where 32 bits hold ctas * total.)
template <typename I>
struct PagedDivision {
  I total, used, extra;
  __device__ PagedDivision(const PagedShape& s, I tiles, I units) {
    used = max((I)1, min((I)s.ctas, tiles / (I)s.least));
    extra = used == (I)s.ctas ? (I)s.extra : (I)0;
    total = tiles + units * (I)s.H_kv * extra;
  }
  __device__ I begin(I c) const { return total * c / used; }
  // The range of CTA c, from the unit and head whose places [f0, f0 + extra + nt) hold
  // its first one on, and the CTAs that share its tiles: those with places f0 + extra
  // on. (The CTA of place x is the last c with begin(c) <= x.)
  __device__ void set(PagedStart& st, I c, I f0, I nt) const {
    const I f = begin(c), g = begin(c + 1), tile0 = f0 + extra;
    st.extra = (int)extra;
    st.kt = f > tile0 ? (int)(f - tile0) : 0;
    st.count = f < tile0 ? (g > tile0 ? (int)(g - tile0) : 0) : (int)(g - f);
    if (st.kt) {
      st.first = (int)(((tile0 + 1) * used - 1) / total);
      st.last = (int)(((tile0 + nt) * used - 1) / total);
    }
  }
};

// The plan as one CTA makes it for itself, for a few hundred units at most and a
// total work that 32 bits hold (offsets that descend, whose spans may overlap and add
// up to more, plan nothing): every sequence into seq (first token, tokens,
// keys, units), its work into work (both shared memory, R entries), the CTA's
// range into *out (shared memory).
__device__ __forceinline__ void plan_locally(const PagedShape& s, const int32_t* q_off, const int32_t* kv_len,
                                             int4* seq, unsigned* work, PagedStart* out, int* err) {
  bool bad = false, descends = false;
  const int lane = threadIdx.x & 31;
  constexpr int kAlone = 4;  // units that a thread counts by itself
  for (int r = threadIdx.x; r < s.R; r += blockDim.x) {
    int a, n, L;
    bad |= sequence_at(s, q_off, kv_len, r, a, n, L);
    descends |= q_off[r + 1] < q_off[r];
    const int units = (n * s.G + s.step - 1) / s.step;
    unsigned w = 0;
    for (int i = 0; i < units && units <= kAlone; ++i) w += max(unit_at(s, r, a, n, L, i).ntiles, 1);
    seq[r] = make_int4(a, n, L, units);
    work[r] = w * s.H_kv;
  }
  if (bad && blockIdx.x == 0) record_error(err, FM_DEV_ERR_RANGE);
  const bool none = __syncthreads_or(descends);
  for (int r = threadIdx.x >> 5; r < s.R; r += blockDim.x >> 5) {  // longer ones: a lane a unit
    const int4 q = seq[r];
    if (q.w <= kAlone) continue;
    unsigned w = 0;
    for (int i = lane; i < q.w; i += 32) w += max(unit_at(s, r, q.x, q.y, q.z, i).ntiles, 1);
    w = __reduce_add_sync(0xffffffffu, w);
    if (lane == 0) work[r] = w * s.H_kv;
  }
  if (threadIdx.x == 0) *out = PagedStart{};
  __syncthreads();
  if (threadIdx.x < 32) {
    const int per = (s.R + 31) / 32, r0 = lane * per, r1 = min(s.R, r0 + per);
    unsigned tiles = 0, units = 0;
    for (int r = r0; r < r1; ++r) {
      tiles += work[r];
      units += seq[r].w;
    }
    const PagedDivision<unsigned> div(s, __reduce_add_sync(0xffffffffu, tiles), __reduce_add_sync(0xffffffffu, units));
    const unsigned ex = div.extra * s.H_kv, mine = tiles + units * ex, c = blockIdx.x;
    unsigned upto = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, upto, m);
      if (lane >= m) upto += x;
    }
    if (c < div.used && div.total > 0 && !none) {  // (the same for every lane)
      const unsigned f = div.begin(c);
      // place f: its sequence, in the range of the one lane whose sequences hold it
      int r = r0;
      unsigned at = upto - mine;
      const bool holds = at <= f && f < upto;
      if (holds)
        while (r < r1 - 1 && at + work[r] + seq[r].w * ex <= f) {
          at += work[r] + seq[r].w * ex;
          ++r;
        }
      const int owner = __ffs(__ballot_sync(0xffffffffu, holds)) - 1;
      r = __shfl_sync(0xffffffffu, r, owner);
      at = __shfl_sync(0xffffffffu, at, owner);
      // its unit, 32 at a time
      const int4 q = seq[r];
      for (int i0 = 0; i0 < q.w; i0 += 32) {
        const int i = i0 + lane;
        PagedStart st = {};
        unsigned nt = 0;
        if (i < q.w) {
          st.unit = unit_at(s, r, q.x, q.y, q.z, i);
          nt = max(st.unit.ntiles, 1);
        }
        const unsigned places = i < q.w ? nt + div.extra : 0;
        unsigned end = places * s.H_kv;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const unsigned x = __shfl_up_sync(0xffffffffu, end, m);
          if (lane >= m) end += x;
        }
        const unsigned from = at + end - places * s.H_kv;  // this lane's unit: places [from, at + end)
        if (i < q.w && from <= f && f < at + end) {
          st.u = r;
          st.i = i;
          st.h = (f - from) / places;
          div.set(st, c, from + st.h * places, nt);
          *out = st;
        }
        at += __shfl_sync(0xffffffffu, end, 31);
        if (at > f) break;
      }
    }
  }
  __syncthreads();
}

// The same where no unit and head is divided (s.whole): they are dealt to the CTAs
// largest first, forth and back, so that each CTA's tiles add up to about the same.
// For several sequences (one's units are in order as they are): first: R + 1 running
// sums of the sequences' units; order: the units from the largest on; sizes: their
// tiles (scratch); all shared memory.
__device__ __forceinline__ void plan_whole(const PagedShape& s, const int32_t* q_off, const int32_t* kv_len,
                                           int4* seq, uint16_t* first, uint16_t* order, uint16_t* sizes,
                                           PagedStart* out, int* err) {
  bool bad = false;
  for (int r = threadIdx.x; r < s.R; r += blockDim.x) {
    int a, n, L;
    bad |= sequence_at(s, q_off, kv_len, r, a, n, L);
    seq[r] = make_int4(a, n, L, (n * s.G + s.step - 1) / s.step);
  }
  if (bad && blockIdx.x == 0) record_error(err, FM_DEV_ERR_RANGE);
  __syncthreads();
  int units = seq[0].w;
  if (s.R > 1) {
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x, per = (s.R + 31) / 32, r0 = lane * per, r1 = min(s.R, r0 + per);
      const int cap = (int)s.max_units;  // spans that overlap may hold more
      int mine = 0;
      for (int r = r0; r < r1; ++r) mine = min(mine + seq[r].w, cap);
      int upto = mine;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, m);
        if (lane >= m) upto = min(upto + x, cap);
      }
      int sum = __shfl_up_sync(0xffffffffu, upto, 1);
      if (lane == 0) sum = 0;
      for (int r = r0; r < r1; ++r) {
        first[r] = (uint16_t)sum;
        sum = min(sum + seq[r].w, cap);
      }
      if (r0 < s.R && r1 == s.R) first[s.R] = (uint16_t)sum;
    }
    __syncthreads();
    units = first[s.R];
    for (int u = threadIdx.x; u < units; u += blockDim.x) {
      int r = 0;
      for (int hi = s.R - 1; r < hi;) {
        const int mid = (r + hi) >> 1;
        if (first[mid + 1] <= u)
          r = mid + 1;
        else
          hi = mid;
      }
      sizes[u] = (uint16_t)unit_at(s, r, seq[r].x, seq[r].y, seq[r].z, u - first[r]).ntiles;
    }
    __syncthreads();
    for (int u = threadIdx.x; u < units; u += blockDim.x) {
      int rank = 0;
      for (int v = 0; v < units; ++v) rank += (sizes[v] > sizes[u] || (sizes[v] == sizes[u] && v < u)) ? 1 : 0;
      order[rank] = (uint16_t)u;
    }
  }
  if (threadIdx.x == 0) {
    // this CTA's items: number c of every even row of ctas items, ctas - 1 - c of every odd one
    const int items = units * s.H_kv, rows = items / s.ctas, rest = items - rows * s.ctas, c = blockIdx.x;
    PagedStart st = {};
    st.count = rows + ((rows & 1 ? s.ctas - 1 - c : c) < rest ? 1 : 0);
    *out = st;
  }
  __syncthreads();
}

// A CTA's walk over its range of tiles, or its units: one (unit, head) at a time.
struct PagedWalk {
  const PagedShape& s;
  const PagedUnit* units;  // the plan kernel's list
  const int4* seq;         // or this CTA's own sequences
  const uint16_t* first;   // (whole) their first units
  const uint16_t* order;   // (whole) the units, largest first
  int left, at, i, h, kt, n;  // current segment: tiles [kt, kt + n) of head h (n 0: a unit without keys)
  int extra;
  PagedUnit u;

  __device__ PagedWalk(const PagedShape& s_, const PagedUnit* units_, const int4* seq_, const uint16_t* first_,
                       const uint16_t* order_, const PagedStart& st)
      : s(s_), units(units_), seq(seq_), first(first_), order(order_), left(st.count), at(st.u), i(st.i), h(st.h),
        kt(st.kt), extra(st.extra), u(st.unit) {
    if (s.whole && left > 0) deal();
    n = s.whole ? u.ntiles : min(u.ntiles - kt, left);
  }
  __device__ bool more() const { return left > 0; }
  // the segment covers its unit wholly
  __device__ bool whole() const { return s.whole || (kt == 0 && n == u.ntiles); }
  __device__ int slot() const { return kt == 0 ? 1 : 0; }
  // (whole) row number `at` of the items
  __device__ void deal() {
    const int k = at * s.ctas + (at & 1 ? s.ctas - 1 - (int)blockIdx.x : (int)blockIdx.x);
    h = k % s.H_kv;
    int v = k / s.H_kv, r = 0;
    if (s.R == 1) {
      v = seq[0].w - 1 - v;  // one sequence: its last units are its largest
    } else {
      v = order[v];
      for (int hi = s.R - 1; r < hi;) {  // the sequence of unit v
        const int mid = (r + hi) >> 1;
        if (first[mid + 1] <= v)
          r = mid + 1;
        else
          hi = mid;
      }
    }
    u = unit_at(s, r, seq[r].x, seq[r].y, seq[r].z, s.R == 1 ? v : v - first[r]);
  }
  __device__ void next() {
    left -= s.whole ? 1 : max(n, 1) + extra;
    if (left <= 0) return;
    if (s.whole) {
      ++at;
      deal();
      n = u.ntiles;
      return;
    }
    kt = 0;
    if (++h == s.H_kv) {
      h = 0;
      if (s.local) {
        int4 q = seq[at];
        if (++i >= q.w) {
          i = 0;
          do q = seq[++at];
          while (q.w == 0 && at + 1 < s.R);
        }
        u = unit_at(s, at, q.x, q.y, q.z, i);
      } else {
        u = units[++at];
      }
    }
    n = min(u.ntiles, left);
  }
};

// Limits of a CTA's own plan: sequences (kLocalChunks: chunk_kernel, whose shared
// memory is nearly full), units more than one a sequence, all units where those of
// several sequences are dealt whole (each is ranked against all others).
constexpr int kLocalSeqs = 256, kLocalChunks = 32;
constexpr int kLocalUnits = 512;
constexpr int kWholeUnits = 320;

// Workspace of one call: units, the running sum of their work, CTA starts, the
// partial slots (two a CTA: rows x d sums, then rows x (m, l)).
struct PagedWork {
  int32_t* first;      // (R + 1) first unit of each sequence
  PagedUnit* units;    // max_units
  long long* sum;      // max_units + 1
  PagedStart* starts;  // ctas
  float* part;
  size_t part_floats;  // floats of one slot
  size_t bytes;
};

inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// (wherever the workspace starts: its parts start on 256-byte boundaries, for which the
// size has room; the parts' rows are stored 32 bytes at a time)
inline PagedWork paged_work(const PagedShape& s, int rows, void* ws) {
  PagedWork w = {};
  char* p = reinterpret_cast<char*>(round256(reinterpret_cast<uintptr_t>(ws)));
  size_t o = 0;
  auto take = [&](size_t bytes) {
    char* at = p ? p + o : nullptr;
    o += round256(bytes);
    return at;
  };
  w.first = reinterpret_cast<int32_t*>(take(sizeof(int32_t) * ((size_t)s.R + 1)));
  w.units = reinterpret_cast<PagedUnit*>(take(sizeof(PagedUnit) * (size_t)s.max_units));
  w.sum = reinterpret_cast<long long*>(take(sizeof(long long) * ((size_t)s.max_units + 1)));
  w.starts = reinterpret_cast<PagedStart*>(take(sizeof(PagedStart) * (size_t)s.ctas));
  w.part_floats = (size_t)rows * (s.d + 2);
  w.part = reinterpret_cast<float*>(take(sizeof(float) * w.part_floats * 2 * (size_t)s.ctas));
  w.bytes = o + 255;
  return w;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
// Byte address of 16-byte chunk `chunk` of row `row` inside a swizzled box.
template <int ROW>
__device__ __forceinline__ uint32_t in_box(int row, int chunk) {
  if constexpr (ROW == 128)
    return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
  else
    return (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}

__device__ __forceinline__ void sts_b16(uint32_t addr, uint32_t v) {
  if (!FM_DBG(smem_range(addr, 2, 2))) return;
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"((uint16_t)v) : "memory");
}

// e4m3 in the high byte of a 16-bit lane, t: (t >> 4) & kE4m3Mag | t & kE4m3Sign is the
// value as bf16, times 2^-120, and NaN (all magnitude bits) becomes 480 times that
constexpr uint32_t kE4m3Mag = 0x07f007f0u, kE4m3Sign = 0x80008000u;
__device__ __forceinline__ uint32_t mul_bf2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The bf16 bits of 2^(e - 7) = 2^(e - 127) 2^120, up to e = 134; and of what is
// left above that, 2^(e - 134). e = 255: NaN.
__device__ __forceinline__ uint32_t factor_lo(uint32_t e) { return e == 255u ? 0x7fc0u : (min(e, 134u) + 120u) << 7; }
__device__ __forceinline__ uint32_t factor_hi(uint32_t e) {
  return (127u + (e > 134u && e < 255u ? e - 134u : 0u)) << 7;
}

// What the producer keeps of a page table: 32 entries from `base` on, one a lane.
struct PageWindow {
  const int32_t* row;
  int base, held, width;
  __device__ void reset(const int32_t* table, int r, int w) {
    row = table + (int64_t)r * w;
    width = w;
    base = INT_MIN / 2;
    held = -1;
  }
  // entries [i, i + n), n <= 32, may be asked next
  __device__ void hold(int i, int n, int lane) {
    if (i < base || i + n > base + 32) {
      base = i;
      held = (i + lane < width) ? row[i + lane] : -1;
    }
  }
};

// Where a row's output goes.
struct PagedOut {
  char* o;
  int64_t st, sh;  // element strides of token and head
  float* lse;      // (T, H_q)
  int H_q;
};

// A kernel's dynamic shared memory limit belongs to the device: raised once on
// each (one bit of `done` a device).
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

constexpr int kChunkRows = 256;  // rows of a chunk_kernel partial slot: two tiles
cudaError_t launch_paged_chunk(const PagedShape& s, const PagedWork& w, const fm_kv_cache& c, const fm_paged_batch& b,
                               const fm_rows& q, const PagedOut& out, float scale, cudaStream_t st, int* err);

}  // namespace fm
