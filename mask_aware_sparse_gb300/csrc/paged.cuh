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

struct __align__(16) PagedStart {
  int u, h, kt, count;  // a CTA's first unit, head and tile, and its number of tiles
  int first, last;      // where kt > 0: the first and the last CTA with tiles of that unit and head
  int pad[2];
};

struct PagedShape {
  int T, R, H_q, H_kv, G, d, width, page, n_pages;
  int causal, window, sinks;  // window 0: none
  int step, tile;  // query rows of a unit, keys of a tile
  int ctas, least;  // CTAs launched; tiles a CTA gets before another one does
  long long max_units;
};

// Tile number kt of a unit's list.
__device__ __forceinline__ int tile_of(const PagedUnit& u, int kt) { return kt < u.ns ? kt : kt - u.ns + u.w0; }

// A CTA's walk over its range of tiles: one (unit, head) at a time.
struct PagedWalk {
  const PagedUnit* units;
  int H_kv, left;
  int ui, h, kt, n;  // current segment: tiles [kt, kt + n) of unit ui, head h (n 0: a unit without keys)
  PagedUnit u;

  __device__ PagedWalk(const PagedUnit* units_, const PagedStart& s, int H_kv_)
      : units(units_), H_kv(H_kv_), left(s.count), ui(s.u), h(s.h), kt(s.kt), n(0) {
    if (left > 0) load();
  }
  __device__ void load() {
    u = units[ui];
    n = min(u.ntiles - kt, left);
  }
  __device__ bool more() const { return left > 0; }
  // the segment covers its unit wholly
  __device__ bool whole() const { return kt == 0 && n == u.ntiles; }
  __device__ int slot() const { return kt == 0 ? 1 : 0; }
  __device__ void next() {
    left -= max(n, 1);
    if (left <= 0) return;
    kt = 0;
    if (++h == H_kv) {
      h = 0;
      ++ui;
      load();
    } else {
      n = min(u.ntiles, left);
    }
  }
};

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

inline PagedWork paged_work(const PagedShape& s, int rows, void* ws) {
  PagedWork w = {};
  char* p = static_cast<char*>(ws);
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
  w.bytes = o;
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

// e4m3 in the high bytes of two 16-bit lanes -> bf16 pair, times 2^-120
__device__ __forceinline__ uint32_t e4m3_bits(uint32_t t) {
  return ((t >> 4) & 0x07f007f0u) | (t & 0x80008000u);
}
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

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" :::); }

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

// Launch with the programmatic dependency on the kernel before it: the new
// grid's prologue runs while that kernel ends, and its grid_dependency_wait
// returns once it has.
template <typename... Args, typename... Given>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, unsigned block, size_t smem, cudaStream_t s,
                             Given&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Args(args)...);
}

}  // namespace fm
