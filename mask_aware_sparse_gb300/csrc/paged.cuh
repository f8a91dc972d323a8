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
//
// Sequences that share a prefix (SH = true): a group's new tokens lie side by side,
// so over the shared keys they are the rows of one long sequence, and each sequence
// has rows of its own over the rest of its keys. Both kinds are virtual sequences of
// one list, prefixes first; a row's results of both are joined by merge_kernel.
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
  int r, hi, ns, w0;  // row of the page table; keys [0, hi) may be visible; tiles [0, ns) hold sinks, then from w0 on
  int ntiles, kv_len, lo, base;  // lo: keys below it are visible as sinks only; base (SH): key of the first tile
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
  int V;       // sequences of the plan: R, or (SH) groups' prefixes, then sequences, as `kinds` has them
  int S;       // groups
  int kinds;   // 1: prefixes, 2: what follows them, 3: both
};

// A call's offsets and lengths; the last two where sequences share prefixes.
struct PagedLists {
  const int32_t* q_off;
  const int32_t* kv_len;
  const int32_t* seq_off;
  const int32_t* prefix_len;
};

// First key of tile number kt of a unit's list, of tiles of TILE keys. (SH: shared prefixes
// end with a page, so that a unit's tiles start at the beginning of one, or a multiple of
// TILE keys after it.)
template <bool SH, int TILE>
__device__ __forceinline__ int key_of(const PagedUnit& u, int kt) {
  return SH ? u.base + kt * TILE : (kt < u.ns ? kt : kt - u.ns + u.w0) * TILE;
}

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
  q.base = 0;
  return q;
}

// Sequences that share prefixes. more[v]: first key that virtual sequence v goes over (a
// multiple of the page size), its row of the page table.
__device__ __forceinline__ int prefixes(const PagedShape& s) { return s.kinds & 1 ? s.S : 0; }

// Unit i of virtual sequence v. A prefix's rows see all of it: they stand behind it.
__device__ __forceinline__ PagedUnit shared_unit_at(const PagedShape& s, int v, const int4& seq, const int2& more,
                                                    int i) {
  const int row0 = i * s.step, tok = row0 / s.G;
  PagedUnit q;
  q.r = more.y;
  q.tok = seq.x + tok;
  q.g0 = row0 - tok * s.G;
  q.nrows = min(s.step, seq.y * s.G - row0);
  q.ns = v < prefixes(s) ? 0 : 1;  // the kind
  q.pos = q.ns ? seq.z - seq.y + tok : seq.z;
  q.kv_len = seq.z;
  const int last = q.pos + (q.g0 + q.nrows - 1) / s.G;
  q.hi = s.causal ? min(max(last + 1, 0), seq.z) : seq.z;
  q.lo = 0;
  q.w0 = 0;
  q.base = more.x;
  q.ntiles = max(0, (q.hi - more.x + s.tile - 1) >> s.tile_log);
  return q;
}

// Group g's sequences [s0, s1), kept inside [0, R], and its shared keys, whole pages of
// them; true where offsets or length are none.
__device__ __forceinline__ bool group_at(const PagedShape& s, const PagedLists& in, int g, int& s0, int& s1, int& P) {
  const int a = in.seq_off[g], b = in.seq_off[g + 1], p = in.prefix_len[g];
  s0 = min(max(a, 0), s.R);
  s1 = min(max(b, s0), s.R);
  P = min(max(p, 0), s.width * s.page) & -s.page;
  return s0 != a || s1 != b || (g == 0 && a != 0) || (g == s.S - 1 && b != s.R) ||
         (s1 > s0 && (p < 0 || p > s.width * s.page));
}

// Virtual sequence of group g: its tokens, keys [0, P) and the table row of its first
// sequence that has tokens (one without may be a slot out of use). Where all tokens are that
// one's, it goes over its keys by itself: P = 0 (64 sequences of up to 4000 keys, all but one
// pair in groups of one, 125 us, with their keys in two units each 130; 32 of up to 2000
// 41.4, 43.2).
__device__ __forceinline__ bool prefix_at(const PagedShape& s, const PagedLists& in, int g, int4& seq, int2& more,
                                          int& s0) {
  int s1, P;
  const bool bad = group_at(s, in, g, s0, s1, P);
  const int a = min(max(in.q_off[s0], 0), s.T), e = in.q_off[s1], n = min(max(e, a), s.T) - a;
  int row = s0;  // the first with q_off[row + 1] > a
  for (int hi = s1 - 1; row < hi;) {
    const int mid = (row + hi) >> 1;
    if (in.q_off[mid + 1] > a)
      hi = mid;
    else
      row = mid + 1;
  }
  row = min(row, s.R - 1);
  if (in.q_off[row + 1] >= e) P = 0;
  seq = make_int4(a, n, P, (n * s.G + s.step - 1) / s.step);
  more = make_int2(0, row);
  return bad;
}

// The same from sequence r's side: all tokens of its group [s0, s1) are its own.
__device__ __forceinline__ bool alone(const PagedLists& in, int r, int s0, int s1) {
  return in.q_off[r] <= in.q_off[s0] && in.q_off[r + 1] >= in.q_off[s1];
}

// Sequence r behind its group's P shared keys (prefix: the group's length as it was given).
// Flagged too where new tokens would lie in the prefix, or it is longer than the sequence.
__device__ __forceinline__ bool rest_at(const PagedShape& s, const PagedLists& in, int r, int P, int prefix, int4& seq,
                                        int2& more) {
  int a, n, L;
  const bool bad = sequence_at(s, in.q_off, in.kv_len, r, a, n, L);
  seq = make_int4(a, n, L, (n * s.G + s.step - 1) / s.step);
  more = make_int2(min(P, L & -s.page), r);
  return bad || (n > 0 && prefix > (s.causal ? max(L - n, 0) : L));
}

// The last g of n ascending starts that is at or below x.
__device__ __forceinline__ int last_at(const int32_t* starts, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (starts[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
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
// Prefixes and what follows them (SH) are units of very different lengths, so that starts
// count in small calls too: two sequences behind 1021 keys 10.7 us, 19.2 where CTAs took
// three short units in turn. (Not by a branch at run time: e4m3 steps 114.4 us for 112.5.)
template <bool SH, typename I>
struct PagedDivision {
  I total, used, extra;
  __device__ PagedDivision(const PagedShape& s, I tiles, I units) {
    used = max((I)1, min((I)s.ctas, tiles / (I)s.least));
    extra = SH || used == (I)s.ctas ? (I)s.extra : (I)0;
    total = tiles + units * (I)s.H_kv * extra;
    if constexpr (SH) used = max((I)1, min((I)s.ctas, total / (I)s.least));
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

// Limits of a CTA's own plan: sequences (kLocalChunks: chunk_kernel, whose shared
// memory is nearly full), units more than one a sequence, all units where those of
// several sequences are dealt whole (each is ranked against all others).
constexpr int kLocalSeqs = 256, kLocalChunks = 32;
constexpr int kSharedChunks = 56;  // (SH: the room of what plan_whole takes is free)
constexpr int kLocalUnits = 512;
constexpr int kWholeUnits = 320;

// The plan as one CTA makes it for itself, for a few hundred units at most and a
// total work that 32 bits hold (offsets that descend, whose spans may overlap and add
// up to more, plan nothing): every sequence into seq (first token, tokens,
// keys, units; SH: the rest of it into more), its work into work (all shared memory,
// V entries; SH: work has room for 5 S + 2 R + 2 more, R up to kLocalSeqs), the CTA's
// range into *out (shared memory). WARPS > 1: that many of its warps take a range each,
// as so many CTAs.
template <bool SH, int WARPS = 1>
__device__ __forceinline__ void plan_locally(const PagedShape& s, const PagedLists& given, int4* seq, int2* more,
                                             unsigned* work, PagedStart* out, int* err) {
  bool bad = false, descends = false, more_units = false;
  const int lane = threadIdx.x & 31;
  constexpr int kAlone = 4;  // units that a thread counts by itself
  auto unit = [&](int r, const int4& q, int i) {
    if constexpr (SH)
      return shared_unit_at(s, r, q, more[r], i);
    else
      return unit_at(s, r, q.x, q.y, q.z, i);
  };
  auto keep = [&](int r, const int4& q) {
    unsigned w = 0;
    for (int i = 0; i < q.w && q.w <= kAlone; ++i) w += max(unit(r, q, i).ntiles, 1);
    seq[r] = q;
    work[r] = w * s.H_kv;
    more_units |= q.w > kAlone;
  };
  if constexpr (SH) {
    // Offsets and lengths into shared memory, all loads at once (each one that waits for
    // another costs a microsecond), then groups, then sequences, which look for theirs there.
    int32_t* gs = reinterpret_cast<int32_t*>(work + s.V);  // groups' first sequences, shared keys, lengths as given
    int32_t *gp = gs + s.S, *gl = gp + s.S;
    const int vs = prefixes(s);
    PagedLists in = given;
    if (s.R <= kLocalSeqs) {
      int32_t *so = gl + s.S, *pl = so + s.S + 1, *qo = pl + s.S, *kl = qo + s.R + 1;
      for (int i = threadIdx.x; i <= max(s.S, s.R); i += blockDim.x) {
        const bool g = i < s.S, r = i < s.R;
        const int a = i <= s.S ? given.seq_off[i] : 0, b = g ? given.prefix_len[i] : 0;
        const int c = i <= s.R ? given.q_off[i] : 0, d = r ? given.kv_len[i] : 0;
        if (i <= s.S) so[i] = a;
        if (g) pl[i] = b;
        if (i <= s.R) qo[i] = c;
        if (r) kl[i] = d;
      }
      in = PagedLists{qo, kl, so, pl};
      __syncthreads();
    }
    for (int g = threadIdx.x; g < s.S; g += blockDim.x) {
      descends |= in.seq_off[g + 1] < in.seq_off[g];
      int s0, s1, P;
      if (vs) {
        int4 q;
        bad |= prefix_at(s, in, g, q, more[g], s0);
        P = q.z;
        keep(g, q);
      } else {
        bad |= group_at(s, in, g, s0, s1, P);
      }
      gs[g] = s0;
      gp[g] = P;
      gl[g] = in.prefix_len[g];
    }
    for (int r = threadIdx.x; r < s.R; r += blockDim.x) descends |= in.q_off[r + 1] < in.q_off[r];
    __syncthreads();
    if (s.kinds & 2)
      for (int r = threadIdx.x; r < s.R; r += blockDim.x) {
        const int g = last_at(gs, s.S, r);
        int4 q;
        int P = gp[g];
        if (!vs && alone(in, r, gs[g], min(max(in.seq_off[g + 1], gs[g]), s.R))) P = 0;
        bad |= rest_at(s, in, r, P, gl[g], q, more[vs + r]);
        keep(vs + r, q);
      }
  } else {
    const PagedLists& in = given;
    for (int r = threadIdx.x; r < s.R; r += blockDim.x) {
      int a, n, L;
      bad |= sequence_at(s, in.q_off, in.kv_len, r, a, n, L);
      descends |= in.q_off[r + 1] < in.q_off[r];
      keep(r, make_int4(a, n, L, (n * s.G + s.step - 1) / s.step));
    }
  }
  if (bad && blockIdx.x == 0) record_error(err, FM_DEV_ERR_RANGE);
  const bool none = __syncthreads_or(descends);
  // (32 steps a warp for 128 sequences, about 2 us, for nothing where none is longer)
  const bool longer = !SH || __syncthreads_or(more_units);
  for (int r = threadIdx.x >> 5; longer && r < s.V; r += blockDim.x >> 5) {  // longer ones: a lane a unit
    const int4 q = seq[r];
    if (q.w <= kAlone) continue;
    unsigned w = 0;
    for (int i = lane; i < q.w; i += 32) w += max(unit(r, q, i).ntiles, 1);
    w = __reduce_add_sync(0xffffffffu, w);
    if (lane == 0) work[r] = w * s.H_kv;
  }
  if (threadIdx.x < WARPS) out[threadIdx.x] = PagedStart{};
  __syncthreads();
  if (threadIdx.x < 32 * WARPS) {
    const int per = (s.V + 31) / 32, r0 = lane * per, r1 = min(s.V, r0 + per);
    unsigned tiles = 0, units = 0;
    for (int r = r0; r < r1; ++r) {
      tiles += work[r];
      units += seq[r].w;
    }
    const PagedDivision<SH, unsigned> div(s, __reduce_add_sync(0xffffffffu, tiles), __reduce_add_sync(0xffffffffu, units));
    const unsigned ex = div.extra * s.H_kv, mine = tiles + units * ex;
    const unsigned c = blockIdx.x * WARPS + (threadIdx.x >> 5);
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
          st.unit = unit(r, q, i);
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
          out[threadIdx.x >> 5] = st;
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
__device__ __forceinline__ void plan_whole(const PagedShape& s, const PagedLists& in, int4* seq, uint16_t* first,
                                           uint16_t* order, uint16_t* sizes, PagedStart* out, int* err) {
  bool bad = false;
  for (int r = threadIdx.x; r < s.R; r += blockDim.x) {
    int a, n, L;
    bad |= sequence_at(s, in.q_off, in.kv_len, r, a, n, L);
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
template <bool SH>
struct PagedWalk {
  const PagedShape& s;
  const PagedUnit* units;  // the plan kernel's list
  const int4* seq;         // or this CTA's own sequences
  const int2* more;        // (SH) and what else belongs to them
  const uint16_t* first;   // (whole) their first units
  const uint16_t* order;   // (whole) the units, largest first
  int left, at, i, h, kt, n;  // current segment: tiles [kt, kt + n) of head h (n 0: a unit without keys)
  int extra;
  PagedUnit u;

  __device__ PagedWalk(const PagedShape& s_, const PagedUnit* units_, const int4* seq_, const int2* more_,
                       const uint16_t* first_, const uint16_t* order_, const PagedStart& st)
      : s(s_), units(units_), seq(seq_), more(more_), first(first_), order(order_), left(st.count), at(st.u), i(st.i),
        h(st.h), kt(st.kt), extra(st.extra), u(st.unit) {
    if (dealt() && left > 0) deal();
    n = dealt() ? u.ntiles : min(u.ntiles - kt, left);
  }
  __device__ bool going() const { return left > 0; }
  __device__ bool dealt() const { return !SH && s.whole; }
  // the segment covers its unit wholly
  __device__ bool whole() const { return dealt() || (kt == 0 && n == u.ntiles); }
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
    left -= dealt() ? 1 : max(n, 1) + extra;
    if (left <= 0) return;
    if (dealt()) {
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
          while (q.w == 0 && at + 1 < s.V);
        }
        if constexpr (SH)
          u = shared_unit_at(s, at, q, more[at], i);
        else
          u = unit_at(s, at, q.x, q.y, q.z, i);
      } else {
        u = units[++at];
      }
    }
    n = min(u.ntiles, left);
  }
};

// Where results of rows with a shared prefix go: row i = token * H_q + head of kind k (0: over the
// prefix, 1: over the rest) to where[k * rows + i], a mark. kMarkWhole: all of it is in full (rows
// of d sums) and full_ml; else it is in the partial slots of CTAs first .. first + n - 1 at `row`.
struct SharedOut {
  float* full;
  float2* full_ml;
  uint32_t* where;
  long long rows;  // T * H_q
};

// A mark: 12 bits each of the first CTA and the parts, 8 of the row.
constexpr uint32_t kMarkWhole = 0xffffffffu;
constexpr int kMarkCtas = 0xfff, kMarkRows = 256;
__host__ __device__ constexpr uint32_t mark_of(int first, int parts) {
  return (uint32_t)first << 20 | (uint32_t)parts << 8;
}
__host__ __device__ constexpr int mark_first(uint32_t w) { return (int)(w >> 20); }
__host__ __device__ constexpr int mark_parts(uint32_t w) { return (int)(w >> 8 & 0xfffu); }
__host__ __device__ constexpr int mark_row(uint32_t w) { return (int)(w & 0xffu); }

// Workers with a range each of a launch that leaves marks, `warps` a CTA: those of all the CTAs
// that the SMs hold, but no more than a mark can name (on 152 SMs 1824 at most).
constexpr int marked_workers(int ctas, int warps) {
  return (ctas * warps < kMarkCtas ? ctas : kMarkCtas / warps) * warps;
}

// Which of a segment's rows' entries of `where` this CTA writes: whole units', and divided ones'
// that it is the second CTA of (0: none). c: its number.
__device__ __forceinline__ uint32_t shared_mark(bool whole, int kt, const PagedStart& st, int c) {
  if (whole) return kMarkWhole;
  return kt > 0 && st.first == c - 1 ? mark_of(st.first, st.last - st.first + 1) : 0u;
}

// Workspace of one call: units, the running sum of their work, CTA starts, the
// partial slots (two a CTA: rows x d sums, then rows x (m, l)).
struct PagedWork {
  int32_t* first;      // (V + 1) first unit of each sequence
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
  w.first = reinterpret_cast<int32_t*>(take(sizeof(int32_t) * ((size_t)s.V + 1)));
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
static_assert(kChunkRows <= kMarkRows, "a mark's row");
// (sh: sequences share prefixes, results go there)
cudaError_t launch_paged_chunk(const PagedShape& s, const PagedWork& w, const fm_kv_cache& c, const PagedLists& in,
                               const int32_t* table, const fm_rows& q, const PagedOut& out, const SharedOut* sh,
                               float scale, cudaStream_t st, int* err);

}  // namespace fm
