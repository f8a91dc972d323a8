// fm_append.cu — new tokens into the paged cache, one pass from the projection's
// output: queries and keys normed per head and rotated by their positions, queries
// out, keys and values into their places (quantised where the cache is e4m3).
//
// Mathematics: the norm and rotation are fm_rope.cu's, with the same arithmetic, so
// that queries and the keys of a bf16 cache have the same bits; places and scales are
// fm_cache.cu's. A key of an e4m3 cache is rounded once, from 32 bits (by way of a
// bf16 tensor it would be rounded twice): with top its row's largest magnitude, the
// scale is 2^(e - 127), e the smallest >= 1 with top <= 448 * 2^(e - 127).
//
// What bounds it: memory at large sizes, each element read once and written once, and
// latency at small ones: offsets, then a table entry, then the rows. The rows' loads
// need none of that and are in flight first; offsets and lengths are read once a block,
// into shared memory, where each token looks its sequence up; a step's table entries are
// loaded while the step before it is computed.
// Between both no one resource is full (8192 tokens of 32 / 8 heads into an e4m3 cache:
// issue slots 67%, memory 45%, the last of 1.7 rounds of steps part empty; the largest stall
// is a step's barriers, of which there are three), and what counts is warps that have work
// meanwhile: four blocks an SM with one row ahead a thread and nothing spilled take 213 us
// for 32768 tokens of 64 / 8 heads, d = 128 (6.3 TB/s, 93% of the copy rate), and 40.7 us
// for 8192 tokens of 32 / 8 into an e4m3 cache; with three blocks 231 and 44.9, two rows ahead in as many registers (spilled)
// 257 and 48.8, rows by asynchronous copies three ahead 294 and 43.2, teams of warps that
// wait for one another alone 237 and 45.1. 64 tokens of 64 sequences: 4.8 us.
#include <type_traits>
#include <cuda_bf16.h>
#include "dependent.cuh"
#include "fm_internal.h"
#include "rope.cuh"
#include "sm100.cuh"

namespace fm {
namespace {

constexpr int kThreads = kRopeThreads, kWarps = kRopeWarps;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kPerSm = 4;   // blocks that an SM holds; of each side as many at most, queries' before keys'
constexpr int kHeld = 256;  // sequences whose offsets and lengths a block keeps

struct Rows3 {
  const char* p;
  int64_t st, sh;
};

struct AppendParams {
  int T, H_q, H_kv, rot, w_f32;
  float eps, rot_scale;
  const int32_t* pos;  // null: the places in the sequences
  const float* inv_freq;
  const void* wq;
  const void* wk;
  Rows3 q, k, v;
  char* qo;
  int64_t qo_st, qo_sh;
  char* c[2];     // k, v pages
  uint8_t* e[2];  // their exponents, or null: a bf16 cache
  const int32_t* off;
  const int32_t* kv_len;
  const int32_t* table;
  int R, width, n_pages, page;
  int* err;
};

// Sixteen values of a row (its D / 16 threads together) as e4m3 with one scale: 8 bytes
// each of a and b, and the exponent byte.
template <int TG>
__device__ __forceinline__ uint32_t quantise(const F2 (&a)[4], const F2 (&b)[4], uint2& qa, uint2& qb) {
  float f[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f2_unpack(a[i], f[2 * i], f[2 * i + 1]);
    f2_unpack(b[i], f[8 + 2 * i], f[8 + 2 * i + 1]);
  }
  // largest magnitude as bits: infinities and NaN are the largest of all
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
#pragma unroll
  for (int m = TG / 2; m > 0; m >>= 1) top = max(top, __shfl_xor_sync(kAll, top, m));
  const int E = (int)(top >> 23);  // 448 = 1.75 * 2^8
  const int e = max(1, E - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0));
  const float inv = __uint_as_float((uint32_t)(254 - min(e, 253)) << 23);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = pack_e4m3x4(f[4 * i] * inv, f[4 * i + 1] * inv, f[4 * i + 2] * inv, f[4 * i + 3] * inv);
    if (E == 255) q[i] = 0x7f7f7f7fu;
  }
  qa = make_uint2(q[0], q[1]);
  qb = make_uint2(q[2], q[3]);
  return E == 255 ? 255u : (uint32_t)e;
}

template <int D>
struct AppendShared {
  static constexpr int kMost = kWarps * 512 / D;  // tokens of a step
  float4 cs[kMost * D / 4];
  float4 ws[D / 4];
  unsigned long long frac[D / 2];
  int64_t slot[kMost];  // keys: head 0's row of the cache; below 0: a token that is left out
  int32_t held[2 * kHeld + 1];
  int32_t pos[kMost];
};

// A block's steps over its tokens' queries, or their keys and then values as one list of
// heads. Warps, rows and steps are divided as in the norm and rotation by itself.
template <int D, bool INTER, bool F8, bool keys>
__device__ __forceinline__ void append_rows(const AppendParams& p, const int TB, AppendShared<D>& sm) {
  using C = Chunks<D, INTER>;
  constexpr int TG = C::TG, HPW = 32 / TG;  // threads per row, rows per warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = lane % TG, hl = lane / TG;
  const C ch(c, p.rot);
  const int RT = p.rot / 16;
  const int H = keys ? 2 * p.H_kv : p.H_q;
  const void* wp = keys ? p.wk : p.wq;
  const int TPW = tokens_per_warp(H, D), HS = HPW / TPW;  // tokens a warp, heads of each at a time
  const int wpt = kWarps / side_groups(H, D, TB);
  const int tw = warp / wpt, w0 = warp - tw * wpt;  // this warp's tokens of the step, its place among their warps
  const int ti = tw * TPW + hl / HS, h0 = hl % HS;  // this thread's token of the step, its first head
  const int tokens = kWarps / wpt * TPW;
  const int stride = gridDim.x * tokens;  // (no more than 2^30 tokens)
  int tok0 = blockIdx.x * tokens;
  // A row's loads are in flight while the one before is computed, and the next step's first
  // ones while its angles are.
  uint4 ra = make_uint4(0, 0, 0, 0), rb = ra;
  auto fetch = [&](int h) {  // of the token at tok0 + ti
    const int64_t t = (int64_t)tok0 + ti;
    if (h < H && t < p.T) {
      const bool val = keys && h >= p.H_kv;
      const Rows3& in = val ? p.v : keys ? p.k : p.q;
      const char* r = in.p + 2 * (t * in.st + (val ? h - p.H_kv : h) * in.sh);
      ra = *reinterpret_cast<const uint4*>(r + 2 * (val ? 16 * c : ch.oa));
      rb = *reinterpret_cast<const uint4*>(r + 2 * (val ? 16 * c + 8 : ch.ob));
    }
  };
  const int first = w0 * HS + h0, step = wpt * HS;  // this thread's heads
  fetch(first);
  // Offsets that do not ascend from 0 or pass T, lengths outside the table: nothing is
  // written (flagged once), as tokens would be taken for those of other places.
  bool bad = false;
  const bool hold = p.R <= kHeld;
  for (int r = threadIdx.x; r <= p.R; r += kThreads) {
    const int o = p.off[r];
    bad |= r == 0 ? o != 0 : o < p.off[r - 1];
    if (hold) sm.held[r] = o;
    if (r == p.R) {
      bad |= o > p.T;
    } else {
      const int L = p.kv_len[r];
      bad |= L < 0 || L > p.width * p.page;
      if (hold) sm.held[kHeld + 1 + r] = L;
    }
  }
  for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) sm.frac[i] = turn_fraction(p.inv_freq[i]);
  if (wp && threadIdx.x < TG) {
    // slot j * TG + c: a quarter of thread c's sixteen weights
    const C mine(threadIdx.x, p.rot);
    for (int j = 0; j < 4; ++j) {
      const int o = (j < 2 ? mine.oa : mine.ob) + 4 * (j & 1);
      sm.ws[j * TG + threadIdx.x] = make_float4(weight_at(wp, p.w_f32, o), weight_at(wp, p.w_f32, o + 1),
                                                weight_at(wp, p.w_f32, o + 2), weight_at(wp, p.w_f32, o + 3));
    }
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (blockIdx.x == 0 && keys && threadIdx.x == 0) record_error(p.err, FM_DEV_ERR_RANGE);
    return;
  }
  // A step's tokens, one a thread: sequence, place, position, page. (Keys: looked up while the
  // step before is computed, as the page is a load that waits for another.)
  int look_pos = 0, look_page = 0, look_at = -1;  // look_at below 0: a token of no sequence, or without a place
  auto look = [&] {
    const int32_t *off = hold ? sm.held : p.off, *len = hold ? sm.held + kHeld + 1 : p.kv_len;
    const int t = tok0 + (int)threadIdx.x;
    look_at = -1;
    if ((int)threadIdx.x >= tokens || t >= p.T || t >= off[p.R]) return;
    int lo = 0, hi = p.R - 1;  // the first r with off[r + 1] > t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (off[mid + 1] > t)
        hi = mid;
      else
        lo = mid + 1;
    }
    const int place = len[lo] - (off[lo + 1] - t);
    look_pos = p.pos ? p.pos[t] : place;
    look_at = 0;
    if (keys) {
      look_page = place >= 0 ? p.table[(int64_t)lo * p.width + place / p.page] : -1;
      look_at = place >= 0 ? place % p.page : 0;
    }
  };
  if (keys) look();
  while (tok0 < p.T) {
    if (!keys) look();
    if ((int)threadIdx.x < tokens) {
      int64_t s = look_at;
      if (keys && look_at >= 0) {
        const bool there = look_page >= 0 && look_page < p.n_pages;
        if (!there) record_error(p.err, FM_DEV_ERR_RANGE);
        s = there ? (int64_t)look_page * p.H_kv * p.page + look_at : -1;
      }
      sm.pos[threadIdx.x] = look_pos;
      sm.slot[threadIdx.x] = s;
    }
    __syncthreads();
    {
      const int half = p.rot / 2;
      for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int t = i / half, f = i - t * half;
        if (sm.slot[t] < 0) continue;
        float s, co;
        angle_of(sm.pos[t], sm.frac[f], s, co);
        store_angle(reinterpret_cast<float*>(sm.cs + t * (p.rot / 4)), RT, f, co * p.rot_scale, s * p.rot_scale);
      }
    }
    __syncthreads();
    const int64_t slot = sm.slot[ti];
    char* out = keys ? nullptr : p.qo + 2 * (((int64_t)tok0 + ti) * p.qo_st);
    F2 co[4], si[4];
    if (ch.turned) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 t = slot >= 0 ? sm.cs[ti * (p.rot / 4) + j * RT + c] : make_float4(0.f, 0.f, 0.f, 0.f);
        co[j] = f2_pack(t.x, t.y);
        si[j] = f2_pack(t.z, t.w);
      }
    }
    if (keys) {
      tok0 += stride;
      look();
      tok0 -= stride;
    }
    // (every lane of a warp takes the same number of turns: sums and maxima are exchanged)
    for (int g = w0 * HS; g < H; g += step) {
      const int h = g + h0;
      const bool val = keys && h >= p.H_kv, live = slot >= 0 && h < H;
      F2 fa[4], fb[4];
      unpack8(ra, fa);
      unpack8(rb, fb);
      int64_t row = 0;
      char* page = nullptr;
      if constexpr (keys) {
        row = slot + (int64_t)(val ? h - p.H_kv : h) * p.page;
        page = val ? p.c[1] : p.c[0];
        if (!F8 && val && live) {  // as they are
          *reinterpret_cast<uint4*>(page + 2 * (row * D + 16 * c)) = ra;
          *reinterpret_cast<uint4*>(page + 2 * (row * D + 16 * c + 8)) = rb;
        }
      }
      if (g + step < H) {
        fetch(h + step);
      } else {
        tok0 += stride;
        fetch(first);
        tok0 -= stride;
      }
      if (wp) {
        F2 sa = f2_mul(fa[0], fa[0]), sb = f2_mul(fb[0], fb[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) {
          sa = f2_fma(fa[i], fa[i], sa);
          sb = f2_fma(fb[i], fb[i], sb);
        }
        const F2 r = f2_both(rsqrtf(row_sum<D>(f2_sum(f2_add(sa, sb))) * (1.f / D) + p.eps));
        if (!val) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            F2* f = j < 2 ? fa + 2 * j : fb + 2 * j - 4;
            const float4 w = sm.ws[j * TG + c];
            f[0] = f2_mul(f[0], f2_mul(r, f2_pack(w.x, w.y)));
            f[1] = f2_mul(f[1], f2_mul(r, f2_pack(w.z, w.w)));
          }
        }
      }
      if (ch.turned && !val) turn<INTER, 1>(fa, fb, co, si);
      if constexpr (!keys) {
        if (live) {
          char* to = out + 2 * (h * p.qo_sh);
          *reinterpret_cast<uint4*>(to + 2 * ch.oa) = pack8(fa);
          *reinterpret_cast<uint4*>(to + 2 * ch.ob) = pack8(fb);
        }
      } else if constexpr (F8) {
        uint2 qa, qb;
        const uint32_t e = quantise<TG>(fa, fb, qa, qb);
        if (live) {
          *reinterpret_cast<uint2*>(page + row * D + (val ? 16 * c : ch.oa)) = qa;
          *reinterpret_cast<uint2*>(page + row * D + (val ? 16 * c + 8 : ch.ob)) = qb;
          if (c == 0) (val ? p.e[1] : p.e[0])[row] = (uint8_t)e;
        }
      } else if (live && !val) {
        *reinterpret_cast<uint4*>(page + 2 * (row * D + ch.oa)) = pack8(fa);
        *reinterpret_cast<uint4*>(page + 2 * (row * D + ch.ob)) = pack8(fb);
      }
    }
    tok0 += stride;
    __syncthreads();
  }
}

// blockIdx.y 0: queries, 1: keys and values.
template <int D, bool INTER, bool F8>
__global__ void __launch_bounds__(kThreads, kPerSm) append_kernel(const AppendParams p, const int TB) {
  __shared__ __align__(16) AppendShared<D> sm;
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.y == 0)
    append_rows<D, INTER, F8, false>(p, TB, sm);
  else
    append_rows<D, INTER, F8, true>(p, TB, sm);
}

Rows3 rows_of(const fm_rows& r) { return Rows3{static_cast<const char*>(r.ptr), r.st, r.sh}; }

// Steps of a side of H heads.
int64_t steps_of(int T, int H, int d, int tb) {
  const int tokens = side_groups(H, d, tb) * tokens_per_warp(H, d);
  return ((int64_t)T + tokens - 1) / tokens;
}

}  // namespace

cudaError_t launch_cache_append(const fm_kv_cache& c, const fm_paged_batch& b, const fm_qk_problem& P, const fm_rows& q,
                                const fm_rows& k, const fm_rows& v, const fm_rows& qo, cudaStream_t s, int* err) {
  AppendParams p = {};
  p.T = P.N;
  p.H_q = P.H_q;
  p.H_kv = P.H_kv;
  p.rot = P.rot;
  p.w_f32 = P.w_f32;
  p.eps = P.eps;
  p.rot_scale = P.rot_scale;
  p.pos = P.pos;
  p.inv_freq = P.inv_freq;
  p.wq = P.q_weight;
  p.wk = P.k_weight;
  p.q = rows_of(q);
  p.k = rows_of(k);
  p.v = rows_of(v);
  p.qo = static_cast<char*>(qo.ptr);
  p.qo_st = qo.st;
  p.qo_sh = qo.sh;
  p.c[0] = static_cast<char*>(c.k);
  p.c[1] = static_cast<char*>(c.v);
  p.e[0] = c.k_exp;
  p.e[1] = c.v_exp;
  p.off = b.q_off;
  p.kv_len = b.kv_len;
  p.table = b.page_table;
  p.R = b.R;
  p.width = b.width;
  p.n_pages = c.n_pages;
  p.page = c.page_size;
  p.err = err;
  // As for the norm and rotation by itself: a warp a group of tokens once that leaves a block
  // for every other SM, more warps on each before that; two columns of blocks, at most what
  // the SMs hold at once of each.
  const int64_t groups = (int64_t)p.T / tokens_per_warp(p.H_q, c.d);
  int tb = 1;
  while (tb < kWarps && groups >= (long long)tb * sm_count()) tb *= 2;
  int64_t grid = steps_of(p.T, p.H_q, c.d, tb);
  if (steps_of(p.T, 2 * p.H_kv, c.d, tb) > grid) grid = steps_of(p.T, 2 * p.H_kv, c.d, tb);
  if (grid > (int64_t)kPerSm * sm_count()) grid = (int64_t)kPerSm * sm_count();
  count_launches(1);
  auto go = [&](auto kernel) { return launch_dependent(kernel, dim3((unsigned)grid, 2), kThreads, 0, s, p, tb); };
  auto pick = [&](auto d, auto inter) {
    return c.k_exp ? go(append_kernel<d.value, inter.value, true>) : go(append_kernel<d.value, inter.value, false>);
  };
  auto dims = [&](auto inter) {
    return c.d == 64    ? pick(std::integral_constant<int, 64>{}, inter)
           : c.d == 128 ? pick(std::integral_constant<int, 128>{}, inter)
                        : pick(std::integral_constant<int, 256>{}, inter);
  };
  return P.interleaved ? dims(std::true_type{}) : dims(std::false_type{});
}

}  // namespace fm
