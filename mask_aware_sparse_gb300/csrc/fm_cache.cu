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
// bytes of bf16 a thread; a block looks its tokens' pages up once for all heads.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
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
  int* err;
};

// The sequence whose rows [off[r], off[r + 1]) hold t, or -1.
__device__ __forceinline__ int sequence_of(const int32_t* off, int R, int t) {
  int lo = 0, hi = R;  // first r with off[r + 1] > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (off[mid + 1] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return (lo < R && off[lo] <= t) ? lo : -1;
}

// Cache row (head 0) of token t, or -1: a token of no sequence, or (flagged) one
// whose place has no page.
template <bool READ>
__device__ __forceinline__ int64_t slot_of(const CacheParams& p, int t) {
  const int r = sequence_of(p.off, p.R, t);
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
__device__ __forceinline__ uint4 dequant8(uint2 raw, float s) {
  const uint32_t w[2] = {raw.x, raw.y};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3));
    const float2 f = __half22float2(h);
    o[i] = pack_bf16x2(f.x * s, f.y * s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// One block: TB tokens, every head, keys then values; d / 8 threads a row.
template <int D, bool F8, bool READ>
__global__ void __launch_bounds__(kThreads) cache_kernel(const CacheParams p, const int TB) {
  constexpr int TR = D / 8, ES = F8 ? 1 : 2;
  __shared__ int64_t slot[kThreads];
  const int t0 = blockIdx.x * TB;
  if (threadIdx.x < TB) slot[threadIdx.x] = (t0 + (int)threadIdx.x < p.T) ? slot_of<READ>(p, t0 + threadIdx.x) : -1;
  __syncthreads();
  const int c = threadIdx.x % TR;
  const int rows = TB * p.H_kv * 2;
  // every thread of a warp takes the same number of turns: the rows' maxima are exchanged
  for (int i0 = 0; i0 < rows; i0 += kThreads / TR) {
    const int i = i0 + threadIdx.x / TR;
    const int which = i >= rows / 2 ? 1 : 0;
    const int j = i - which * (rows / 2);
    // write: neighbouring rows are heads of a token; read: tokens of a head
    const int h = READ ? j / TB : j % p.H_kv;
    const int t = READ ? j - h * TB : j / p.H_kv;
    const int64_t s = i < rows ? slot[t] : -1;
    const bool live = s >= 0;
    const int64_t row = s + (int64_t)h * p.page;
    if constexpr (READ) {
      if (!live) continue;
      uint4 r;
      if constexpr (F8)
        r = dequant8(reinterpret_cast<const uint2*>(p.c[which] + row * D)[c], scale_of(p.e[which][row]));
      else
        r = reinterpret_cast<const uint4*>(p.c[which] + row * D * 2)[c];
      reinterpret_cast<uint4*>(p.out[which] + ((int64_t)h * p.T + t0 + t) * D * 2)[c] = r;
    } else {
      uint4 r = make_uint4(0, 0, 0, 0);
      if (live) r = *reinterpret_cast<const uint4*>(p.in[which] + 2 * ((int64_t)(t0 + t) * p.st[which] + h * p.sh[which] + 8 * c));
      if constexpr (!F8) {
        if (live) reinterpret_cast<uint4*>(p.c[which] + row * D * ES)[c] = r;
      } else {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        // the largest magnitude as bits: infinities and NaN are the largest of all
        uint32_t m = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) m = __vmaxu2(m, w[x] & 0x7fff7fffu);
#pragma unroll
        for (int x = TR / 2; x > 0; x >>= 1) m = __vmaxu2(m, __shfl_xor_sync(kAll, m, x));
        const uint32_t top = max(m & 0xffffu, m >> 16);
        const int E = (int)(top >> 7);  // 448 = 1.75 * 2^8
        int e = max(1, E - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0));
        uint2 q = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
        if (E == 255) {
          e = 255;
        } else {
          const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
          float f[8];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            f[2 * x] = __uint_as_float(w[x] << 16) * inv;
            f[2 * x + 1] = __uint_as_float(w[x] & 0xffff0000u) * inv;
          }
          q.x = pack_e4m3x4(f[0], f[1], f[2], f[3]);
          q.y = pack_e4m3x4(f[4], f[5], f[6], f[7]);
        }
        if (live) {
          reinterpret_cast<uint2*>(p.c[which] + row * D)[c] = q;
          if (c == 0) p.e[which][row] = (uint8_t)e;
        }
      }
    }
  }
}

template <bool READ>
cudaError_t launch(const CacheParams& p, int d, bool f8, cudaStream_t s) {
  // few tokens: one a block, so that the heads' rows spread over the SMs; many:
  // enough tokens a block that looking a page up is a small part of its work
  int tb = 1;
  while (tb < 32 && p.T >= 2ll * tb * 8 * sm_count()) tb *= 2;
  const unsigned grid = (unsigned)((p.T + tb - 1) / tb);
  auto go = [&](auto kernel) { kernel<<<grid, kThreads, 0, s>>>(p, tb); };
  if (d == 64)
    f8 ? go(cache_kernel<64, true, READ>) : go(cache_kernel<64, false, READ>);
  else if (d == 128)
    f8 ? go(cache_kernel<128, true, READ>) : go(cache_kernel<128, false, READ>);
  else
    f8 ? go(cache_kernel<256, true, READ>) : go(cache_kernel<256, false, READ>);
  count_launches(1);
  return cudaGetLastError();
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
  return launch<true>(p, c.d, c.k_exp != nullptr, s);
}

}  // namespace fm
