// fm_cache.cu — writing new keys and values into the paged cache, quantising
// them on the way where the cache is e4m3, and reading it back.
//
// A quantised row (one slot of one head, d values) has one scale, a power of
// two kept as its biased exponent byte e (value 2^(e - 127)): the smallest with
// max |x| <= 448 * 2^(e - 127), e >= 1. Stored x * 2^(127 - e) is exact before
// the one rounding to e4m3 (half a step, 2^-4 of the value, in its normal
// range), no result depends on how a division rounds, and what is read back,
// stored * 2^(e - 127), is exact in bf16. A scale that is no power of two would
// reach one binade further below the row's largest value, where e4m3's steps
// are absolute; it would keep no more digits elsewhere. A row that holds a NaN
// or an infinity gets e = 255 and reads as NaN throughout.
//
// What bounds both kernels: memory, each row read once and written once, 16
// bytes a load; a block looks its tokens' pages up once for all heads.
//
// Pages are copied to pages as they are (copy_kernel): a sequence that forks takes
// copies of the pages it will write, on free pages.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include "dependent.cuh"
#include "fm_internal.h"
#include "sm100.cuh"

namespace fm {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kAll = 0xffffffffu;

struct CacheParams {
  char* c[2];         // k, v pages
  uint8_t* e[2];      // their exponents, or null: a bf16 cache
  const char* in[2];  // write: new rows; read: unused
  int64_t st[2], sh[2];
  char* out[2];  // read: (H_kv, n_rows, d)
  const int32_t* off;     // first token (write) or output row (read) of each sequence, R + 1
  const int32_t* kv_len;  // write: keys of each sequence, the new ones among them
  const int32_t* table;
  int R, width, n_pages, H_kv, page, T;
  int wide;  // read: the output rows start on 32-byte boundaries
  int* err;
};

// The sequence whose rows [off[r], off[r + 1]) hold t = t0 + lane, or -1; called
// by a whole warp, for its lanes below n. 32 of the offsets, one a lane, are
// compared with each t at once, so that up to 32 sequences cost one load's latency
// (a bisection's is what a block of a few tokens would mostly wait for), then a
// bisection between two of them.
__device__ __forceinline__ int sequence_of(const int32_t* off, int R, int t0, int n) {
  const int lane = threadIdx.x & 31, t = t0 + lane, S = (R + 31) / 32;
  const int ends = off[min((lane + 1) * S, R)];
  int k = 0;  // parts of S sequences that end at or before t
  for (int i = 0; i < n; ++i) {
    const int x = __popc(__ballot_sync(kAll, lane * S < R && ends <= t0 + i));
    if (i == lane) k = x;
  }
  int lo = min(k * S, R), hi = min(lo + S - 1, R);  // first r with off[r + 1] > t lies in [lo, hi]
  while (lo < hi && lo < R) {
    const int mid = (lo + hi) >> 1;
    if (off[min(mid + 1, R)] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return (lane < n && lo < R && off[lo] <= t && t < off[lo + 1]) ? lo : -1;
}

// Cache row (head 0) of this lane's token, or -1: a token of no sequence, or (flagged) one
// whose place has no page.
template <bool READ>
__device__ __forceinline__ int64_t slot_of(const CacheParams& p, int t0, int n) {
  const int r = sequence_of(p.off, p.R, t0, n), t = t0 + (threadIdx.x & 31);
  if (r < 0) return -1;
  const int a = t - p.off[r];
  const int64_t pos = READ ? a : (int64_t)p.kv_len[r] - (p.off[r + 1] - p.off[r]) + a;
  if (pos >= 0 && pos < (int64_t)p.width * p.page) {
    const int pg = p.table[(int64_t)r * p.width + pos / p.page];
    if (pg >= 0 && pg < p.n_pages) return ((int64_t)pg * p.H_kv) * p.page + pos % p.page;
  }
  record_error(p.err, FM_DEV_ERR_RANGE);
  return -1;
}

__device__ __forceinline__ float scale_of(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7fc00000u : e == 0u ? 0x00400000u : e << 23);
}

// 8 e4m3 values times a power of two, as 8 bf16
__device__ __forceinline__ uint4 dequant8(uint32_t w0, uint32_t w1, float s) {
  const uint32_t w[2] = {w0, w1};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3));
    const float2 f = __half22float2(h);
    o[i] = pack_bf16x2(f.x * s, f.y * s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The block's tokens' places, by its first warp, and by the others whether the batch is
// one at all: offsets that do not ascend from 0 or pass T, lengths outside the table.
// False (flagged once): nothing is written, as tokens would be taken for those of other
// places. Every block reads all of them, which a few thousand sequences hardly notice
// (8192 tokens of 4 sequences 8.5 -> 8.6 us, of 4096 10.4 -> 11.9; 65536 tokens of as
// many sequences 91 -> 257).
template <bool READ>
__device__ __forceinline__ bool look_up(const CacheParams& p, int64_t* slot, int t0, int TB) {
  grid_dependency_wait();
  bool bad = false;
  if (threadIdx.x < 32) {  // TB <= 32
    const int64_t s = slot_of<READ>(p, t0, min(TB, p.T - t0));
    if (threadIdx.x < TB) slot[threadIdx.x] = s;
  } else {
    const int most = p.width * p.page;
    for (int r = (int)threadIdx.x - 32; r <= p.R; r += kThreads - 32) {
      const int o = p.off[r];
      bad |= r == 0 ? o != 0 : o < p.off[r - 1];
      if (r == p.R)
        bad |= o > p.T;
      else if (!READ)
        bad |= p.kv_len[r] < 0 || p.kv_len[r] > most;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && blockIdx.x == 0 && threadIdx.x == 0) record_error(p.err, FM_DEV_ERR_RANGE);
  return !bad;
}

// A block: TB = 2^log tokens, keys of every head, then values. Its rows go by token
// first, and a step's rows are a multiple of TB, so that each thread stays with one
// token: what belongs to the token is worked out once, a head costs a multiplication
// and an addition (with places and addresses from each row's number, the write of
// 8192 tokens took 12.4 us, and more with more loads ahead: its instructions bound it).
template <int TR>
struct Rows {
  static constexpr int STEP = kThreads / TR;  // rows
  int c, t, h, heads;                         // this thread's part of a row, token, first head; heads of a step
  __device__ Rows(int log) {
    const int r = threadIdx.x / TR;
    c = threadIdx.x % TR;
    t = r & ((1 << log) - 1);
    h = r >> log;
    heads = STEP >> log;
  }
};
constexpr int most_log(int tr) { return kThreads / tr >= 32 ? 5 : kThreads / tr >= 16 ? 4 : 3; }

// Rows whose loads a thread has in flight (reading, one: the 16K-key read of four
// sequences took 66 us).
constexpr int kWriteAhead = 2, kReadAhead = 4;

// D / 16 threads a row, 32 bytes of bf16 each: neighbouring ones where they become 16
// bytes of e4m3, else two pieces half a row apart, so that each load and store of a
// row's threads covers whole lines (side by side: 8192 tokens 13.2 us instead of 9.3).
template <int D, bool F8>
__global__ void __launch_bounds__(kThreads) write_kernel(const CacheParams p, const int log) {
  constexpr int TR = D / 16, kAhead = kWriteAhead, PIECE = F8 ? 32 : 16, NEXT = F8 ? 1 : TR;
  __shared__ int64_t slot[32];
  const int t0 = blockIdx.x << log;
  if (!look_up<false>(p, slot, t0, 1 << log)) return;
  const Rows<TR> own(log);
  const int64_t s = slot[own.t];
  const char* in[2];
  char* out[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    in[i] = p.in[i] + 2 * ((int64_t)(t0 + own.t) * p.st[i]) + PIECE * own.c;
    out[i] = p.c[i] + s * D * (F8 ? 1 : 2) + 16 * own.c;
  }
  // every thread of a warp takes the same number of turns: the rows' maxima are exchanged
  for (int g = 0; g < 2 * p.H_kv; g += kAhead * own.heads) {
    uint4 x[kAhead][2];
    int h[kAhead], which[kAhead];
    bool live[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      h[k] = g + k * own.heads + own.h;
      live[k] = s >= 0 && h[k] < 2 * p.H_kv;
      which[k] = h[k] >= p.H_kv ? 1 : 0;
      h[k] -= which[k] * p.H_kv;
      x[k][0] = x[k][1] = make_uint4(0, 0, 0, 0);
      if (live[k]) {
        const uint4* from = reinterpret_cast<const uint4*>((which[k] ? in[1] : in[0]) + 2 * (h[k] * p.sh[which[k]]));
        x[k][0] = from[0];
        x[k][1] = from[NEXT];
      }
    }
    if constexpr (!F8) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (live[k]) {
          uint4* to = reinterpret_cast<uint4*>((which[k] ? out[1] : out[0]) + (int64_t)h[k] * p.page * D * 2);
          to[0] = x[k][0];
          to[NEXT] = x[k][1];
        }
    } else {
      // each row's largest magnitude as bits: infinities and NaN are the largest of all
      uint32_t m[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        m[k] = 0;
#pragma unroll
        for (int y = 0; y < 2; ++y)
          m[k] = __vmaxu2(m[k], __vmaxu2(__vmaxu2(x[k][y].x & 0x7fff7fffu, x[k][y].y & 0x7fff7fffu),
                                         __vmaxu2(x[k][y].z & 0x7fff7fffu, x[k][y].w & 0x7fff7fffu)));
      }
#pragma unroll
      for (int y = TR / 2; y > 0; y >>= 1)
#pragma unroll
        for (int k = 0; k < kAhead; ++k) m[k] = __vmaxu2(m[k], __shfl_xor_sync(kAll, m[k], y));
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const uint32_t top = max(m[k] & 0xffffu, m[k] >> 16);
        const int E = (int)(top >> 7);  // 448 = 1.75 * 2^8
        const int e = max(1, E - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0));
        const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
        uint32_t q[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint4& v = x[k][y >> 1];
          const uint32_t a = y & 1 ? v.z : v.x, b = y & 1 ? v.w : v.y;
          q[y] = pack_e4m3x4(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xffff0000u) * inv,
                             __uint_as_float(b << 16) * inv, __uint_as_float(b & 0xffff0000u) * inv);
          if (E == 255) q[y] = 0x7f7f7f7fu;
        }
        if (live[k]) {
          *reinterpret_cast<uint4*>((which[k] ? out[1] : out[0]) + (int64_t)h[k] * p.page * D) =
              make_uint4(q[0], q[1], q[2], q[3]);
          if (own.c == 0) p.e[which[k]][s + (int64_t)h[k] * p.page] = (uint8_t)(E == 255 ? 255 : e);
        }
      }
    }
  }
}

// 16 bytes of the cache a thread.
template <int D, bool F8>
__global__ void __launch_bounds__(kThreads) read_kernel(const CacheParams p, const int log) {
  constexpr int TR = D * (F8 ? 1 : 2) / 16, kAhead = kReadAhead;
  __shared__ int64_t slot[32];
  const int t0 = blockIdx.x << log;
  if (!look_up<true>(p, slot, t0, 1 << log)) return;
  const Rows<TR> own(log);
  const int64_t s = slot[own.t];
  if (s < 0) return;
  const char* in[2] = {p.c[0] + s * D * (F8 ? 1 : 2) + 16 * own.c, p.c[1] + s * D * (F8 ? 1 : 2) + 16 * own.c};
  for (int g = own.h; g < 2 * p.H_kv; g += kAhead * own.heads) {
    uint4 x[kAhead];
    uint32_t e[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int h = g + k * own.heads, which = h >= p.H_kv ? 1 : 0;
      if (h >= 2 * p.H_kv) continue;
      const int64_t row = (int64_t)(h - which * p.H_kv) * p.page;
      x[k] = *reinterpret_cast<const uint4*>((which ? in[1] : in[0]) + row * D * (F8 ? 1 : 2));
      if constexpr (F8) e[k] = p.e[which][s + row];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int h = g + k * own.heads, which = h >= p.H_kv ? 1 : 0;
      if (h >= 2 * p.H_kv) continue;
      uint4* to = reinterpret_cast<uint4*>(p.out[which] +
                                           ((int64_t)(h - which * p.H_kv) * p.T + t0 + own.t) * D * 2);
      if constexpr (F8) {
        const float f = scale_of(e[k]);
        const uint4 lo = dequant8(x[k].x, x[k].y, f), hi = dequant8(x[k].z, x[k].w, f);
        if (p.wide) {
          // one whole 32-byte sector a thread (two stores of 16 bytes: 62 us for the read of four 16K sequences)
          stg_b32x8(to + 2 * own.c, lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w);
        } else {
          to[2 * own.c] = lo;
          to[2 * own.c + 1] = hi;
        }
      } else {
        to[own.c] = x[k];
      }
    }
  }
}

// A page's keys lie together, so do its values and its exponents: pieces of 16 KB, and
// both exponents as one, dealt to blocks in turn. Memory bounds it: 4096 pages of 64
// e4m3 rows of 8 heads, d = 128, 168 us (6.4 TB/s, 95% of the copy rate). A pair outside the
// cache is flagged and left out. Blocks wait for none: a page that is both copied to and in
// another pair would be undefined.
struct CopyParams {
  char* c[2];
  uint8_t* e[2];
  const int32_t* src;
  const int32_t* dst;
  int n, n_pages;
  int64_t bytes, exps;  // of a page's keys, of their exponents (0: a bf16 cache)
  int* err;
};

constexpr int kPiece = kThreads * 16 * 4;

__global__ void __launch_bounds__(kThreads) copy_kernel(const CopyParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int each = (int)((p.bytes + kPiece - 1) / kPiece), all = 2 * each + (p.exps ? 1 : 0);  // pieces of a page
  for (int64_t i = blockIdx.x; i < (int64_t)p.n * all; i += gridDim.x) {
    const int64_t pair = i / all;
    const int piece = (int)(i - pair * all), which = piece >= each ? 1 : 0;
    const int from = p.src[pair], to = p.dst[pair];
    if (from == -1 && to == -1) continue;
    if (from < 0 || to < 0 || from >= p.n_pages || to >= p.n_pages) {
      if (piece == 0 && threadIdx.x == 0) record_error(p.err, FM_DEV_ERR_RANGE);
      continue;
    }
    if (piece == 2 * each) {
      for (int64_t x = 16 * threadIdx.x; x < 2 * p.exps; x += 16 * kThreads) {
        uint8_t* e = x < p.exps ? p.e[0] : p.e[1];
        const int64_t at = x < p.exps ? x : x - p.exps;
        *reinterpret_cast<uint4*>(e + to * p.exps + at) = *reinterpret_cast<const uint4*>(e + from * p.exps + at);
      }
      continue;
    }
    char* c = which ? p.c[1] : p.c[0];
    const int64_t x0 = (int64_t)(piece - which * each) * kPiece + 16 * threadIdx.x;
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t x = x0 + k * 16 * kThreads;
      if (x < p.bytes) v[k] = *reinterpret_cast<const uint4*>(c + from * p.bytes + x);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t x = x0 + k * 16 * kThreads;
      if (x < p.bytes) *reinterpret_cast<uint4*>(c + to * p.bytes + x) = v[k];
    }
  }
}

template <bool READ>
cudaError_t launch(const CacheParams& p, int d, bool f8, cudaStream_t s) {
  // Tokens of a block: as many as fill its threads' loads once, if that leaves two
  // blocks an SM; then more of them (fewer look-ups) while that leaves more than fill
  // an SM. Writing 1000 / 8192 / 12000 tokens of 8 heads, d = 128: 3.2 / 8.5 / 11.2 us
  // (before the batch was looked at, 0.1 us); with one step less 3.4 / 8.7 / 13.8 (fewer,
  // larger blocks) or 4.6 / 8.9 / 11.3 us.
  const int tr = READ ? d * (f8 ? 1 : 2) / 16 : d / 16, full = kThreads / tr * (READ ? kReadAhead : kWriteAhead);
  int log = 0;
  while (log < most_log(tr) && p.T >= (((2ll * p.H_kv << log) < full ? 2ll : READ ? 4 : 8) << log) * sm_count()) ++log;
  const unsigned grid = (unsigned)((p.T + (1 << log) - 1) >> log);
  auto pick = [&](auto write, auto read) {
    if constexpr (READ)
      return launch_dependent(read, dim3(grid), kThreads, 0, s, p, log);
    else
      return launch_dependent(write, dim3(grid), kThreads, 0, s, p, log);
  };
  count_launches(1);
  if (d == 64)
    return f8 ? pick(write_kernel<64, true>, read_kernel<64, true>)
              : pick(write_kernel<64, false>, read_kernel<64, false>);
  if (d == 128)
    return f8 ? pick(write_kernel<128, true>, read_kernel<128, true>)
              : pick(write_kernel<128, false>, read_kernel<128, false>);
  return f8 ? pick(write_kernel<256, true>, read_kernel<256, true>)
            : pick(write_kernel<256, false>, read_kernel<256, false>);
}

CacheParams params_of(const fm_kv_cache& c, int* err) {
  CacheParams p = {};
  p.c[0] = static_cast<char*>(c.k);
  p.c[1] = static_cast<char*>(c.v);
  p.e[0] = c.k_exp;
  p.e[1] = c.v_exp;
  p.n_pages = c.n_pages;
  p.H_kv = c.H_kv;
  p.page = c.page_size;
  p.err = err;
  return p;
}

}  // namespace

cudaError_t launch_cache_write(const fm_kv_cache& c, const fm_paged_batch& b, int T, const fm_rows& k,
                               const fm_rows& v, cudaStream_t s, int* err) {
  CacheParams p = params_of(c, err);
  p.in[0] = static_cast<const char*>(k.ptr);
  p.in[1] = static_cast<const char*>(v.ptr);
  p.st[0] = k.st;
  p.sh[0] = k.sh;
  p.st[1] = v.st;
  p.sh[1] = v.sh;
  p.off = b.q_off;
  p.kv_len = b.kv_len;
  p.table = b.page_table;
  p.R = b.R;
  p.width = b.width;
  p.T = T;
  return launch<false>(p, c.d, c.k_exp != nullptr, s);
}

cudaError_t launch_cache_copy(const fm_kv_cache& c, const int32_t* src, const int32_t* dst, int n, cudaStream_t s,
                              int* err) {
  CopyParams p = {};
  p.c[0] = static_cast<char*>(c.k);
  p.c[1] = static_cast<char*>(c.v);
  p.e[0] = c.k_exp;
  p.e[1] = c.v_exp;
  p.src = src;
  p.dst = dst;
  p.n = n;
  p.n_pages = c.n_pages;
  const int64_t rows = (int64_t)c.H_kv * c.page_size;
  p.bytes = rows * c.d * (c.k_exp ? 1 : 2);
  p.exps = c.k_exp ? rows : 0;
  p.err = err;
  const int64_t pieces = (int64_t)n * (2 * ((p.bytes + kPiece - 1) / kPiece) + (p.exps ? 1 : 0));
  const int64_t most = 8ll * sm_count();
  count_launches(1);
  return launch_dependent(copy_kernel, dim3((unsigned)(pieces < most ? pieces : most)), kThreads, 0, s, p);
}

cudaError_t launch_cache_read(const fm_kv_cache& c, const int32_t* kv_off, const int32_t* table, int R, int width,
                              int n_rows, void* k, void* v, cudaStream_t s, int* err) {
  CacheParams p = params_of(c, err);
  p.out[0] = static_cast<char*>(k);
  p.out[1] = static_cast<char*>(v);
  p.off = kv_off;
  p.table = table;
  p.R = R;
  p.width = width;
  p.T = n_rows;
  p.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31) == 0;
  return launch<true>(p, c.d, c.k_exp != nullptr, s);
}

}  // namespace fm
