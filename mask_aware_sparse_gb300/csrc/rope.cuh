// rope.cuh — what the kernels that norm and rotate rows of heads share: a row's
// layout over its threads, the rotation, the norm's sum, angles as fractions of a turn.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include "sm100.cuh"

namespace fm {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
static_assert(kRopeWarps == 8, "side_groups");

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
  for (int m = D / 32; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
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

// Angle f of a token: slot (pair of frequencies j of thread c)
// cs[j * rot/16 + c] = {cos, cos, sin, sin}, so that the 16-byte reads of neighbouring
// threads are neighbours. `out`: the token's rot / 4 slots as floats.
__device__ __forceinline__ void store_angle(float* out, int RT, int f, float c, float s) {
  const int thr = f >> 3, k = f & 7;
  float* to = out + ((k >> 1) * RT + thr) * 4 + (k & 1);
  to[0] = c;
  to[2] = s;
}

// cos and sin of pos times a frequency that is `frac` of a turn.
__device__ __forceinline__ void angle_of(int pos, unsigned long long frac, float& s, float& c) {
  const unsigned long long turns = (unsigned long long)(long long)pos * frac;
  sincospif((float)(long long)turns * 1.0842021724855044e-19f /* 2^-63 */, &s, &c);
}

}  // namespace fm
