// fm_rope.cu — per-head norm and position rotation of queries and keys, one
// pass from a projection's output to the attention kernels' inputs, and its
// backward pass.
//
// Mathematics, per token and head (x: d elements, w: the norm's weights):
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r w          (n = x without weights)
//   theta_i = pos f_i,  c_i = s cos theta_i,  s_i = s sin theta_i
//   (a, b) -> (a c_i - b s_i, a s_i + b c_i)            for pair i < rot / 2
// with pairs (i, i + rot/2) (half layout) or (2i, 2i + 1) (interleaved); the
// elements from rot on pass through. Backward, with g the rotation's transpose
// applied to dy and z = x r:  dw = sum g z,  dx = r (g w - z / d sum(g w z)); r^3, which
// that spares, would leave fp32's range for rows far from 1.
// Sums, norms and the rotation are fp32; each output is rounded to bf16 once.
//
// What bounds it: memory, one read and one write of every element (backward:
// dy and x read, dx written). The layout therefore needs no exchange between
// threads but the norm's sum: d / 16 threads own a head's row, each holding the
// two 8-element chunks whose elements pair up, so one 16-byte load per chunk,
// the rotation in registers, one 16-byte store per chunk.
//
// Angles: f_i / 2 pi is turned once per block into a 64-bit fraction of a turn;
// pos times it, modulo 2^64, is the fraction of theta (error below |pos| 2^-64
// turns for |f_i| < 2^32, against |pos| f_i 2^-25 for an fp32 product), which
// sincospif takes. A block computes the angles of its tokens once, in shared
// memory, for all heads.
#include <cmath>
#include <cuda_bf16.h>
#include "dependent.cuh"
#include "fm_internal.h"
#include "sm100.cuh"

namespace fm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
static_assert(kWarps == 8, "side_groups");
constexpr unsigned kAll = 0xffffffffu;

struct View {
  char* p;
  int64_t sb, sh, sn;  // element strides
};

struct QkParams {
  int B, N, H_q, H_kv, rot;
  int w_f32;
  float eps, rot_scale;
  const int32_t* pos;
  int64_t pos_sb;
  const float* inv_freq;
  const void* wq;
  const void* wk;
  View q, k, v;     // forward: inputs; backward: gradients of the outputs
  View xq, xk;      // backward: the forward's inputs (read where normed)
  View qo, ko, vo;  // forward: outputs; backward: gradients of the inputs
  int has_v;
  float* part;  // backward: per-block partial weight gradients, (grid, 2, d)
};

// Two fp32 numbers as one operand: half the instructions (8192 tokens of 48 heads,
// both ways: 110 us, 2 us more one by one).
using F2 = uint64_t;
__device__ __forceinline__ F2 f2_both(float x) { return f2_pack(x, x); }
__device__ __forceinline__ float f2_sum(F2 a) {
  float x, y;
  f2_unpack(a, x, y);
  return x + y;
}
__device__ __forceinline__ void unpack8(const uint4& r, F2 (&f)[4]) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2_pack(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack8(const F2 (&f)[4]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x, y;
    f2_unpack(f[i], x, y);
    u[i] = pack_bf16x2(x, y);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Where thread c of a row finds its two chunks. Rotated threads of the half
// layout hold [8c, 8c + 8) and the same of the second half; all others 16
// consecutive elements. Either way a rotated thread's eight pairs have the
// frequencies 8c .. 8c + 7.
template <int D, bool INTER>
struct Chunks {
  static constexpr int TG = D / 16;  // threads per row
  int oa, ob;
  bool turned;
  __device__ Chunks(int c, int rot) {
    turned = 16 * c < rot;
    oa = (!INTER && turned) ? 8 * c : 16 * c;
    ob = (!INTER && turned) ? rot / 2 + 8 * c : 16 * c + 8;
  }
};

// (a, b) of the eight pairs rotated by +theta (DIR = 1) or -theta (DIR = -1); co and
// si hold two frequencies each
template <bool INTER, int DIR>
__device__ __forceinline__ void turn(F2 (&a)[4], F2 (&b)[4], const F2 (&co)[4], const F2 (&si)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTER) {
      F2* f = i < 2 ? a + 2 * i : b + 2 * i - 4;  // pairs 2 i and 2 i + 1
      float c[2], s[2];
      f2_unpack(co[i], c[0], c[1]);
      f2_unpack(si[i], s[0], s[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x, y;
        f2_unpack(f[k], x, y);
        const float t = DIR > 0 ? s[k] : -s[k];
        f[k] = f2_pack(x * c[k] - y * t, x * t + y * c[k]);
      }
    } else {
      const F2 x = a[i], y = b[i];
      a[i] = DIR > 0 ? f2_sub(f2_mul(x, co[i]), f2_mul(y, si[i])) : f2_fma(x, co[i], f2_mul(y, si[i]));
      b[i] = DIR > 0 ? f2_fma(x, si[i], f2_mul(y, co[i])) : f2_sub(f2_mul(y, co[i]), f2_mul(x, si[i]));
    }
  }
}

// Tokens that a warp takes at a time, each with all of its H heads.
__host__ __device__ __forceinline__ int tokens_per_warp(int H, int d) {
  int t = 512 / d;  // rows a warp holds
  while (t > 1 && t * H > 512 / d) t /= 2;
  return t;
}

// Groups of such tokens per step of a side with H heads: TB, or as many as leave
// each of a group's warps some of the heads.
__host__ __device__ __forceinline__ int side_groups(int H, int d, int TB) {
  const int rows = 512 / d, hs = rows / tokens_per_warp(H, d);
  int wpt = 8 / TB;
  while (wpt > 1 && (wpt / 2) * hs >= H) wpt /= 2;
  return 8 / wpt;
}

template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = D / 32; m > 0; m >>= 1) v += __shfl_xor_sync(kAll, v, m);
  return v;
}

__device__ __forceinline__ float weight_at(const void* w, int f32, int i) {
  return f32 ? static_cast<const float*>(w)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// x / (2 pi) modulo 1, in units of 2^-64: x = m 2^k times 1 / (2 pi) to 128 bits, for
// |x| < 2^32 within one unit (below 2^24 half of one).
__device__ __forceinline__ unsigned long long turn_fraction(float x) {
  constexpr unsigned long long hi = 0x28be60db9391054aull, lo = 0x7f09d5f47d4d3770ull;  // 1 / (2 pi)
  const uint32_t u = __float_as_uint(x);
  const int e = (int)(u >> 23) & 255, k = (e ? e : 1) - 150;
  const unsigned long long m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);
  const unsigned __int128 p = (unsigned __int128)m * hi + __umul64hi(m, lo);  // m / (2 pi)
  unsigned long long t = 0;
  if (k > 0)
    t = k < 64 ? (unsigned long long)p << k | m * lo >> (64 - k) : 0;
  else if (k > -128)
    t = (unsigned long long)(k ? (p + ((unsigned __int128)1 << (-k - 1))) >> -k : p);
  return u >> 31 ? 0 - t : t;
}

// The block's frequencies as fractions of a turn.
__device__ __forceinline__ void load_fractions(const QkParams& p, unsigned long long* frac) {
  for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) frac[i] = turn_fraction(p.inv_freq[i]);
}

// cos and sin (times rot_scale) of the block's TB tokens from tok0 on. Slot
// (pair of frequencies j of thread c): cs[t][j * rot/16 + c] = {cos, cos, sin,
// sin}, so that the 16-byte reads of neighbouring threads are neighbours.
__device__ __forceinline__ void load_angles(const QkParams& p, const unsigned long long* frac, float4* cs, int TB,
                                            int64_t tok0, int64_t total) {
  const int half = p.rot / 2, RT = p.rot / 16;
  float* out = reinterpret_cast<float*>(cs);
  for (int i = threadIdx.x; i < TB * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    const int64_t tok = tok0 + t;
    if (tok >= total) break;
    const int64_t b = tok / p.N;
    const int pos = p.pos[b * p.pos_sb + (tok - b * p.N)];
    const unsigned long long turns = (unsigned long long)(long long)pos * frac[f];
    float s, c;
    sincospif((float)(long long)turns * 1.0842021724855044e-19f /* 2^-63 */, &s, &c);
    const int thr = f >> 3, k = f & 7;
    float* to = out + 2 * t * half + ((k >> 1) * RT + thr) * 4 + (k & 1);
    to[0] = c * p.rot_scale;
    to[2] = s * p.rot_scale;
  }
}

__device__ __forceinline__ uint4* at(const View& v, int64_t b, int h, int64_t n, int off) {
  return reinterpret_cast<uint4*>(v.p + 2 * (b * v.sb + h * v.sh + n * v.sn + off));
}

// blockIdx.y 0: queries, 1: keys and values. BWD: the backward. A warp holds HPW
// rows at a time: heads of one token, or, with fewer heads than that, those of
// several tokens (two heads at d = 64 would leave three quarters of a warp idle).
// A block and step: TB groups of such tokens, kWarps / TB warps on each.
//
// Loads in flight bound it: two rows' groups ahead of the one computed (kAhead),
// three blocks an SM (backward: two, with twice as much to load), weights in
// shared memory to leave registers for that. One group ahead at 118 registers
// (two blocks an SM) moved 4.8 TB/s at 65536 tokens of 80 heads, d = 128.
template <int D, bool INTER, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD ? 2 : 3) qk_kernel(const QkParams p, const int TB) {
  using C = Chunks<D, INTER>;
  constexpr int TG = C::TG, HPW = 32 / TG;  // threads per row, rows per warp
  constexpr int kAhead = 2;
  __shared__ __align__(16) float4 cs[kWarps * HPW * D / 4];  // at most kWarps * HPW tokens, rot <= D
  __shared__ unsigned long long frac[D / 2];
  __shared__ float4 ws[D / 4];
  __shared__ float red[BWD ? kWarps * D : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = lane % TG, hl = lane / TG;
  const C ch(c, p.rot);
  const int total = p.B * p.N;
  const int RT = p.rot / 16;
  const bool keys = blockIdx.y != 0;
  const View in = keys ? p.k : p.q, out = keys ? p.ko : p.qo, src = keys ? p.xk : p.xq;
  const int H = keys ? p.H_kv : p.H_q;
  const void* wp = keys ? p.wk : p.wq;
  const int TPW = tokens_per_warp(H, D), HS = HPW / TPW;  // tokens a warp, heads of each at a time
  const int wpt = kWarps / side_groups(H, D, TB);
  const int tw = warp / wpt, w0 = warp - tw * wpt;  // this warp's tokens of the step, its place among their warps
  const int ti = tw * TPW + hl / HS, h0 = hl % HS;  // this thread's token of the step, its first head
  const int tokens = kWarps / wpt * TPW;
  F2 acc[BWD ? 8 : 1];  // weight gradients of this thread's 16 columns
  if constexpr (BWD) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = f2_both(0.f);
  }
  grid_dependency_wait();
  grid_launch_dependents();
  load_fractions(p, frac);
  if (wp && threadIdx.x < TG) {
    // slot j * TG + c: a quarter of thread c's sixteen weights
    const C mine(threadIdx.x, p.rot);
    for (int j = 0; j < 4; ++j) {
      const int o = (j < 2 ? mine.oa : mine.ob) + 4 * (j & 1);
      ws[j * TG + threadIdx.x] = make_float4(weight_at(wp, p.w_f32, o), weight_at(wp, p.w_f32, o + 1),
                                             weight_at(wp, p.w_f32, o + 2), weight_at(wp, p.w_f32, o + 3));
    }
  }
  __syncthreads();
  const int groups = (H + HS - 1) / HS;
  const int stride = gridDim.x * tokens;  // (no more than 2^30 tokens)
  int tok0 = blockIdx.x * tokens, b = 0, n = 0;
  bool there = false;
  // The next rows' loads are in flight while these are computed, and the next step's
  // first ones while its angles are (a row is read and written by the same threads, so
  // in and out may be one tensor).
  uint4 ra[kAhead], rb[kAhead], xa[BWD ? kAhead : 1], xb[BWD ? kAhead : 1];
  auto fetch = [&](int k, int g) {
    const int h = g * HS + h0;
    if (there && h < H) {
      ra[k] = *at(in, b, h, n, ch.oa);
      rb[k] = *at(in, b, h, n, ch.ob);
      if constexpr (BWD) {
        if (wp) {
          xa[k] = *at(src, b, h, n, ch.oa);
          xb[k] = *at(src, b, h, n, ch.ob);
        }
      }
    }
  };
  auto begin = [&] {
    there = tok0 + ti < total;
    b = (tok0 + ti) / p.N;
    n = tok0 + ti - b * p.N;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(k, w0 + k * wpt);
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    ra[k] = rb[k] = make_uint4(0, 0, 0, 0);
    if constexpr (BWD) xa[k] = xb[k] = make_uint4(0, 0, 0, 0);
  }
  begin();
  while (tok0 < total) {
    load_angles(p, frac, cs, tokens, tok0, total);
    __syncthreads();
    {
      F2 co[4], si[4];
      if (ch.turned) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 t = there ? cs[ti * (p.rot / 4) + j * RT + c] : make_float4(0.f, 0.f, 0.f, 0.f);
          co[j] = f2_pack(t.x, t.y);
          si[j] = f2_pack(t.z, t.w);
        }
      }
      for (int g0 = w0; g0 < groups; g0 += kAhead * wpt) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int g = g0 + k * wpt;
          if (g >= groups) break;
          const int h = g * HS + h0;
          const bool live = there && h < H;
          F2 fa[4], fb[4];
          unpack8(ra[k], fa);
          unpack8(rb[k], fb);
          // 1 / sqrt(mean(x^2) + eps) of the row in a and b
          auto factor = [&](const F2 (&a)[4], const F2 (&b)[4]) {
            F2 sa = f2_mul(a[0], a[0]), sb = f2_mul(b[0], b[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) {
              sa = f2_fma(a[i], a[i], sa);
              sb = f2_fma(b[i], b[i], sb);
            }
            return rsqrtf(row_sum<D>(f2_sum(f2_add(sa, sb))) * (1.f / D) + p.eps);
          };
          // weights of pairs 2 j and 2 j + 1 of a (j < 2) or b
          auto weight = [&](int j, F2& w0, F2& w1) {
            const float4 w = ws[j * TG + c];
            w0 = f2_pack(w.x, w.y);
            w1 = f2_pack(w.z, w.w);
          };
          if constexpr (!BWD) {
            fetch(k, g + kAhead * wpt);
            if (wp) {
              const F2 r = f2_both(factor(fa, fb));
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                F2* f = j < 2 ? fa + 2 * j : fb + 2 * j - 4;
                F2 w0, w1;
                weight(j, w0, w1);
                f[0] = f2_mul(f[0], f2_mul(r, w0));
                f[1] = f2_mul(f[1], f2_mul(r, w1));
              }
            }
            if (ch.turned) turn<INTER, 1>(fa, fb, co, si);
          } else {
            F2 va[4], vb[4];
            if (wp) {
              unpack8(xa[k], va);
              unpack8(xb[k], vb);
            }
            fetch(k, g + kAhead * wpt);
            if (ch.turned) turn<INTER, -1>(fa, fb, co, si);
            if (wp) {
              const F2 r = f2_both(factor(va, vb));
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                va[i] = f2_mul(va[i], r);
                vb[i] = f2_mul(vb[i], r);
              }
              if (live) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  acc[i] = f2_fma(fa[i], va[i], acc[i]);
                  acc[4 + i] = f2_fma(fb[i], vb[i], acc[4 + i]);
                }
              }
              F2 s0 = f2_both(0.f), s1 = s0;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                F2* f = j < 2 ? fa + 2 * j : fb + 2 * j - 4;
                const F2* v = j < 2 ? va + 2 * j : vb + 2 * j - 4;
                F2 w0, w1;
                weight(j, w0, w1);
                f[0] = f2_mul(f[0], w0);
                f[1] = f2_mul(f[1], w1);
                s0 = f2_fma(f[0], v[0], s0);
                s1 = f2_fma(f[1], v[1], s1);
              }
              const F2 t = f2_both(row_sum<D>(f2_sum(f2_add(s0, s1))) * (-1.f / D));
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                fa[i] = f2_mul(r, f2_fma(va[i], t, fa[i]));
                fb[i] = f2_mul(r, f2_fma(vb[i], t, fb[i]));
              }
            }
          }
          if (live) {
            *at(out, b, h, n, ch.oa) = pack8(fa);
            *at(out, b, h, n, ch.ob) = pack8(fb);
          }
        }
      }
      const int64_t vb = b, vn = n;
      const bool v_there = there;
      tok0 += stride;
      begin();
      if (keys && p.has_v) {
        for (int g = w0; g < groups; g += wpt) {
          const int h = g * HS + h0;
          if (v_there && h < H) {
            const uint4 x = *at(p.v, vb, h, vn, 16 * c), y = *at(p.v, vb, h, vn, 16 * c + 8);
            *at(p.vo, vb, h, vn, 16 * c) = x;
            *at(p.vo, vb, h, vn, 16 * c + 8) = y;
          }
        }
      }
    }
    __syncthreads();
  }
  if constexpr (BWD) {
    // one fixed order: lanes of a warp, then warps, then (next kernel) blocks
    if (wp) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float two[2];
        f2_unpack(acc[i / 2], two[0], two[1]);
        float v = two[i & 1];
#pragma unroll
        for (int m = TG; m < 32; m <<= 1) v += __shfl_xor_sync(kAll, v, m);
        if (hl == 0) red[warp * D + (i < 8 ? ch.oa + i : ch.ob + i - 8)] = v;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < D; i += kThreads) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += red[w * D + i];
        p.part[((int64_t)blockIdx.x * 2 + (keys ? 1 : 0)) * D + i] = v;
      }
    }
  }
}

// Weight gradients: the blocks' partial sums, 32 columns a block, in one order.
__global__ void __launch_bounds__(1024) qk_weights_kernel(const float* part, int blocks, int D, void* dwq, void* dwk,
                                                          int f32) {
  __shared__ float red[32][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
  const int kind = col / D, i = col - kind * D;
  void* dst = kind ? dwk : dwq;
  float v = 0.f;
  if (dst)
    for (int r = y; r < blocks; r += 32) v += part[((int64_t)r * 2 + kind) * D + i];
  red[y][threadIdx.x & 31] = v;
  __syncthreads();
  if (y == 0 && dst) {
    v = 0.f;
    for (int r = 0; r < 32; ++r) v += red[r][threadIdx.x];
    if (f32)
      static_cast<float*>(dst)[i] = v;
    else
      static_cast<__nv_bfloat16*>(dst)[i] = __float2bfloat16_rn(v);
  }
}

View view_of(const fm_view* v) {
  if (!v) return View{nullptr, 0, 0, 0};
  return View{static_cast<char*>(v->ptr), v->sb, v->sh, v->sn};
}

// Groups of tokens per block and step: one warp on each (the angles are then read once
// per token) once that leaves a block for every other SM, more warps on each before
// that. 512 / 1000 tokens of 48 heads, d = 128, both ways: 14.0 / 20.8 us; only when
// four blocks an SM are left 2 us more, eight 6 us more.
int groups_per_step(const fm_qk_problem& P) {
  const int64_t groups = (int64_t)P.B * P.N / tokens_per_warp(P.H_q, P.d);
  int tb = 1;
  while (tb < kWarps && groups >= (long long)tb * sm_count()) tb *= 2;
  return tb;
}
// Two columns of blocks, queries and keys (with values), at most what the SMs hold
// at once of each (forward, 8192 tokens of 48 heads: 43.3 us, with 8 blocks an SM 2 us more); the
// backward has a partial row per block besides.
int grid_blocks(const fm_qk_problem& P, int tb, int per_sm) {
  const int H = P.H_q > P.H_kv ? P.H_q : P.H_kv;  // the side that needs more steps
  const int tokens = side_groups(H, P.d, tb) * tokens_per_warp(H, P.d);
  const int64_t steps = ((int64_t)P.B * P.N + tokens - 1) / tokens;
  const int64_t most = (int64_t)sm_count() * per_sm;
  return (int)(steps < most ? steps : most);
}
constexpr int kFwdPerSm = 3, kBwdPerSm = 2;

template <bool BWD>
cudaError_t launch_qk(const fm_qk_problem& P, const QkParams& p, int grid, int tb, cudaStream_t s) {
  auto go = [&](auto kernel) { return launch_dependent(kernel, dim3((unsigned)grid, 2), kThreads, 0, s, p, tb); };
  count_launches(1);
  if (P.d == 64)
    return P.interleaved ? go(qk_kernel<64, true, BWD>) : go(qk_kernel<64, false, BWD>);
  if (P.d == 128)
    return P.interleaved ? go(qk_kernel<128, true, BWD>) : go(qk_kernel<128, false, BWD>);
  return P.interleaved ? go(qk_kernel<256, true, BWD>) : go(qk_kernel<256, false, BWD>);
}

QkParams params_of(const fm_qk_problem& P) {
  QkParams p = {};
  p.B = P.B;
  p.N = P.N;
  p.H_q = P.H_q;
  p.H_kv = P.H_kv;
  p.rot = P.rot;
  p.w_f32 = P.w_f32;
  p.eps = P.eps;
  p.rot_scale = P.rot_scale;
  p.pos = P.pos;
  p.pos_sb = P.pos_sb;
  p.inv_freq = P.inv_freq;
  p.wq = P.q_weight;
  p.wk = P.k_weight;
  return p;
}

}  // namespace

cudaError_t launch_qk_fwd(const fm_qk_problem& P, const fm_view* q, const fm_view* k, const fm_view* v,
                          const fm_view* qo, const fm_view* ko, const fm_view* vo, cudaStream_t s) {
  QkParams p = params_of(P);
  p.q = view_of(q);
  p.k = view_of(k);
  p.v = view_of(v);
  p.qo = view_of(qo);
  p.ko = view_of(ko);
  p.vo = view_of(vo);
  p.has_v = v != nullptr;
  const int tb = groups_per_step(P);
  return launch_qk<false>(P, p, grid_blocks(P, tb, kFwdPerSm), tb, s);
}

size_t qk_bwd_ws_bytes(const fm_qk_problem& P) { return (size_t)sm_count() * kBwdPerSm * 2 * P.d * sizeof(float); }

cudaError_t launch_qk_bwd(const fm_qk_problem& P, const fm_view* dqo, const fm_view* dko, const fm_view* dvo,
                          const fm_view* q, const fm_view* k, const fm_view* dq, const fm_view* dk, const fm_view* dv,
                          void* dwq, void* dwk, void* ws, cudaStream_t s) {
  QkParams p = params_of(P);
  p.q = view_of(dqo);
  p.k = view_of(dko);
  p.v = view_of(dvo);
  p.xq = view_of(q);
  p.xk = view_of(k);
  p.qo = view_of(dq);
  p.ko = view_of(dk);
  p.vo = view_of(dv);
  p.has_v = dvo != nullptr;
  p.part = static_cast<float*>(ws);
  const int tb = groups_per_step(P);
  const int grid = grid_blocks(P, tb, kBwdPerSm);
  cudaError_t e = launch_qk<true>(P, p, grid, tb, s);
  if (e != cudaSuccess || (!P.q_weight && !P.k_weight)) return e;
  count_launches(1);
  return launch_dependent(qk_weights_kernel, dim3(2 * P.d / 32), 1024, 0, s, p.part, grid, P.d,
                          P.q_weight ? dwq : nullptr, P.k_weight ? dwk : nullptr, P.w_f32);
}

}  // namespace fm
