// Shared by the tensor-core forms of dflash_attend: units, their chunks, and each CTA's share of them.
//
// The chunks of all units, in (sequence, tile, head) order, form one index space; CTA b of a
// one-CTA-per-SM grid takes slots [b W / n, (b + 1) W / n) of it, sized on the device from the
// lengths.  G: a form's geometry - keys of a chunk, slots a unit occupies beside its chunks (the cost of
// opening a segment: queries, pipeline restart, output), slots of a chunk with two tiles and with one, threads of a CTA.
//
// Trees in units of two tiles: a chunk takes a CTA 2.3 us, or 1.55 where the unit's second tile has no token (33 to 48
// nodes of 8 heads to a K/V head have one such unit of two), so that chunks occupy three slots or two, and belong to
// the CTA that has their first: 32 trees of 33 nodes 155 -> 137 us, of 48 158 -> 145, of 64 (all two tiles) 161 as
// before.  (Slots of 5 and 3: 163 for trees of mixed sizes; of 4 and 3 1 to 2 us less than of 3 and 2 there, 3 to 4 more
// for 33 to 40 nodes, whose units gain most.  Over 8-bit pages a chunk with one tile takes nearly as long as one with
// two, and every chunk is one slot: by 3 and 2 32 trees of 33 nodes took 213 us for 191, of 64 186 for 181, of mixed
// sizes 305 for 296.  So it is without trees, where a cut elsewhere would round results differently from before.)
#pragma once

#include <cuda_bf16.h>

#include "serve_attend.cuh"

namespace dflash {
namespace plan {

struct Seg {
  int s, r0, n, kv;     // sequence, its first row, rows, key rows
  int tile, g, t0;      // query tile, kv head, its first token
  int k0, nch;          // first key (page aligned), chunks of the unit
  int c_lo, c_hi;       // this CTA's chunks of it
};

// Tokens of a unit's tile and the chunks it visits.
struct Shape {
  int group, T, TT;     // query heads per kv head, tokens of a 128-row tile, of a unit
};
__device__ __forceinline__ Shape shape_of(const AttendParams& p, int NT) {
  Shape h;
  h.group = p.group;
  h.T = p.tokens;
  h.TT = h.T * NT;
  return h;
}
template <class G, bool kTree>
__device__ __forceinline__ int unit_chunks(const AttendParams& p, const Shape& h, int n, int kv, int tile, int* k0) {
  const int t0 = tile * h.TT, t1 = min(n, t0 + h.TT);
  const int end = !kTree && p.causal ? min(kv, max(0, kv - n + t1)) : kv;
  int lo = p.window > 0 ? max(0, kv - n + (kTree ? 0 : t0) - p.window + 1) : 0;
  lo &= ~(kPage - 1);
  *k0 = lo;
  return max(1, (end - lo + G::kKeys - 1) / G::kKeys);  // a unit without keys still writes its zeros
}

// Slots of a chunk of a unit, and of a unit beside its chunks.
template <class G, bool kTree>
__device__ __forceinline__ int chunk_slots(const Shape& h, int n, int tile) {
  return !kTree || h.TT == h.T ? 1 : tile * h.TT + h.T < n ? G::kTwo : G::kOne;
}
template <class G, bool kTree>
__device__ __forceinline__ int cost_slots(const Shape& h) { return G::kUnitCost * (!kTree || h.TT == h.T ? 1 : G::kTwo); }
template <class G, bool kTree>
__device__ __forceinline__ int unit_slots(const AttendParams& p, const Shape& h, int n, int kv, int tile) {
  int k0;
  return unit_chunks<G, kTree>(p, h, n, kv, tile, &k0) * chunk_slots<G, kTree>(h, n, tile) + cost_slots<G, kTree>(h);
}
// CTAs that the W slots are cut for: each has the first slot of a chunk wherever a unit goes on on both its sides.
template <class G, bool kTree>
__device__ __forceinline__ int ctas_of(const Shape& h, long long W) {
  return (int)min((long long)gridDim.x, !kTree || h.TT == h.T ? W : W / G::kTwo);
}

// The segments of index range [lo, hi), from unit (s, tile, g) whose first slot is pu.
template <class G, bool kTree>
struct Walk {
  long long lo, hi, pu;
  int s, tile, g;

  __device__ bool next(const AttendParams& p, const Shape& h, Seg& q) {
    while (pu < hi && s < p.nb) {
      bool bad;
      if (!seq_of<kTree>(p, s, &q.r0, &q.n, &q.kv, &bad)) {
        ++s;
        tile = g = 0;
        continue;
      }
      q.nch = unit_chunks<G, kTree>(p, h, q.n, q.kv, tile, &q.k0);
      q.s = s, q.tile = tile, q.g = g, q.t0 = tile * h.TT;
      const int w = chunk_slots<G, kTree>(h, q.n, tile);
      const long long first = pu + cost_slots<G, kTree>(h);
      pu = first + (long long)q.nch * w;
      if (++g == p.nkv) {
        g = 0;
        if (++tile * h.TT >= q.n) tile = 0, ++s;
      }
      if (hi <= first || lo >= pu) continue;  // only cost slots of it are in range
      auto chunks = [&](int slots) { return w == 1 ? slots : w == G::kOne ? (slots + G::kOne - 1) / G::kOne : (slots + G::kTwo - 1) / G::kTwo; };
      q.c_lo = lo > first ? chunks((int)(lo - first)) : 0;
      q.c_hi = hi < pu ? chunks((int)(hi - first)) : q.nch;
      if (kTree && q.c_lo >= q.c_hi) continue;  // only later slots of a chunk
      return true;
    }
    return false;
  }
};

template <class G>
struct PlanCtl {
  int s0, tile0, found;
  long long red[G::kThreads / 32], base;
};

// Slots of tiles [a, b) of a sequence for one kv head, by this thread.
template <class G, bool kTree>
__device__ __forceinline__ long long tile_slots(const AttendParams& p, const Shape& h, int n, int kv, int a, int b, int step) {
  long long r = 0;
  for (int t = a; t < b; t += step) r += unit_slots<G, kTree>(p, h, n, kv, t);
  return r;
}

// This CTA's walk.  `scratch`: nb long longs of shared memory.  All threads.
template <class G, bool kTree>
__device__ Walk<G, kTree> make(const AttendParams& p, const Shape& h, PlanCtl<G>& c, long long* scratch, bool wide, long long* W_out) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (p.nb <= 32 && !wide) {
    // a lane per sequence, every warp for itself: no barrier (a step's first 3.5 us went by in the
    // general form's)
    int r0, n = 0, kv = 0;
    bool bad = false;
    const bool has = lane < p.nb && seq_of<kTree>(p, lane, &r0, &n, &kv, &bad);
    if (bad && blockIdx.x == 0 && warp == 0 && p.status) atomicOr(p.status, DFLASH_DEV_BAD_CTX);
    const int tiles = has ? (n + h.TT - 1) / h.TT : 0;
    const long long mine = tile_slots<G, kTree>(p, h, n, kv, 0, tiles, 1) * p.nkv;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const long long W = __shfl_sync(0xffffffffu, inc, 31);
    const int ctas = ctas_of<G, kTree>(h, W), b = blockIdx.x;
    Walk<G, kTree> w;
    w.lo = b < ctas ? (long long)b * W / ctas : 0;
    w.hi = b < ctas ? (long long)(b + 1) * W / ctas : 0;
    w.s = p.nb, w.tile = w.g = 0, w.pu = w.hi;
    *W_out = W;
    if (w.lo >= w.hi) return w;
    const int s0 = __ffs(__ballot_sync(0xffffffffu, inc > w.lo)) - 1;  // the sequence that holds slot lo
    long long at = __shfl_sync(0xffffffffu, inc - mine, s0);
    const int n0 = __shfl_sync(0xffffffffu, n, s0), kv0 = __shfl_sync(0xffffffffu, kv, s0);
    w.s = s0;
    for (;;) {  // its tile: at most a few
      const int slots = unit_slots<G, kTree>(p, h, n0, kv0, w.tile);
      if (w.lo < at + (long long)slots * p.nkv) {
        w.g = (int)((w.lo - at) / slots);
        w.pu = at + (long long)w.g * slots;
        return w;
      }
      at += (long long)slots * p.nkv;
      ++w.tile;
    }
  }
  // slots of each sequence (all kv heads): a thread per sequence, or a warp where chunks are long
  for (int s = wide ? warp : t; s < p.nb; s += wide ? (G::kThreads / 32) : G::kThreads) {
    int r0, n, kv;
    bool bad;
    long long m = 0;
    if (seq_of<kTree>(p, s, &r0, &n, &kv, &bad)) {
      const int tiles = (n + h.TT - 1) / h.TT;
      m = wide ? tile_slots<G, kTree>(p, h, n, kv, lane, tiles, 32) : tile_slots<G, kTree>(p, h, n, kv, 0, tiles, 1);
    } else if (bad && blockIdx.x == 0 && p.status && (!wide || lane == 0)) {
      atomicOr(p.status, DFLASH_DEV_BAD_CTX);
    }
    if (wide) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    }
    if (!wide || lane == 0) scratch[s] = m * p.nkv;
  }
  if (t == 0) c.found = 0;
  __syncthreads();
  // thread t sums sequences [t per, (t + 1) per)
  const int per = (p.nb + G::kThreads - 1) / G::kThreads, s_lo = min(p.nb, t * per), s_hi = min(p.nb, s_lo + per);
  auto scan = [&](long long v, long long* all) {  // exclusive sum over the threads before this one
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) c.red[warp] = inc;
    __syncthreads();
    long long b = inc - v, a = 0;
    for (int w = 0; w < (G::kThreads / 32); ++w) {
      if (w < warp) b += c.red[w];
      a += c.red[w];
    }
    __syncthreads();
    *all = a;
    return b;
  };
  long long mine = 0, W;
  for (int s = s_lo; s < s_hi; ++s) mine += scratch[s];
  long long at = scan(mine, &W);
  const int ctas = ctas_of<G, kTree>(h, W), b = blockIdx.x;
  Walk<G, kTree> w;
  w.lo = b < ctas ? (long long)b * W / ctas : 0;
  w.hi = b < ctas ? (long long)(b + 1) * W / ctas : 0;
  w.s = p.nb, w.tile = w.g = 0, w.pu = w.hi;
  *W_out = W;
  if (w.lo >= w.hi) return w;
  if (at <= w.lo && w.lo < at + mine) {
    for (int s = s_lo; s < s_hi; ++s) {
      if (w.lo < at + scratch[s]) {
        c.s0 = s, c.base = at;
        break;
      }
      at += scratch[s];
    }
  }
  __syncthreads();
  const int s0 = c.s0;
  long long base = c.base;
  int r0, n, kv;
  bool bad;
  seq_of<kTree>(p, s0, &r0, &n, &kv, &bad);
  const int tiles = (n + h.TT - 1) / h.TT;
  for (int b0 = 0; b0 < tiles; b0 += G::kThreads) {  // the tile that holds slot lo
    const int tile = b0 + t;
    const long long v = tile < tiles ? (long long)unit_slots<G, kTree>(p, h, n, kv, tile) * p.nkv : 0;
    long long all;
    const long long x = base + scan(v, &all);
    if (v > 0 && x <= w.lo && w.lo < x + v) c.tile0 = tile, c.base = x, c.found = 1;
    base += all;
    __syncthreads();
    if (c.found) break;
  }
  w.s = s0, w.tile = c.tile0;
  const int slots = unit_slots<G, kTree>(p, h, n, kv, w.tile);
  w.g = (int)((w.lo - c.base) / slots);
  w.pu = c.base + (long long)w.g * slots;
  return w;
}

// Which of 32 keys from `key` on a tree's row sees: context [lo, ctx), of the rows [ctx, kv) those with a bit in
// its mask of n words.
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* mask, int n, int key, int lo, int ctx, int kv) {
  const int at = key - ctx;  // bit of the mask that the first key has
  auto word = [&](int w) { return w >= 0 && w < n ? __ldg(mask + w) : w < 0 ? 0xffffffffu : 0u; };  // (the context: ones)
  uint32_t m = at <= -32 ? 0xffffffffu : __funnelshift_r(word(at >> 5), word((at >> 5) + 1), at & 31);
  if (lo > key) m = lo - key >= 32 ? 0u : m & 0xffffffffu << (lo - key);
  if (kv < key + 32) m = kv <= key ? 0u : m & 0xffffffffu >> (key + 32 - kv);
  return m;
}

// ---- Pages in 8 bits.

// Codes 0, 1 and 2, 3 of a word as pairs of bf16, times 2^-120: sign, exponent and mantissa << 4.  NaN (seven ones) becomes
// 480, which no number's code does: `met` keeps the largest magnitudes, by one instruction a pair beside the
// permutes' pipe, for is_nan() and spread_nan() below.  (By sums and masks of the codes: 158 us for 152, see serve_attend8.cu.)
__device__ __forceinline__ uint2 widen(uint32_t w, uint32_t& met) {
  uint32_t a, b;  // each byte with its sign in the byte above, moved up by 4
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(a) : "r"(w));
  asm("prmt.b32 %0, %1, 0, 0xb3a2;" : "=r"(b) : "r"(w));
  asm("mad.lo.u32 %0, %0, 16, 0;" : "+r"(a));  // (a shift, off the pipe of the permutes)
  asm("mad.lo.u32 %0, %0, 16, 0;" : "+r"(b));
  a &= 0x87f087f0u, b &= 0x87f087f0u;
  asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(met) : "r"(a));
  asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(met) : "r"(b));
  return make_uint2(a, b);
}
__device__ __forceinline__ bool is_nan(uint32_t met) { return (met & 0x7fffu) == 0x7f0u || (met >> 16 & 0x7fffu) == 0x7f0u; }

// Is one of 16 codes NaN's, of either sign?
__device__ __forceinline__ bool nan_codes(const uint4& w) {
  auto flip = [](uint32_t x) { return (x + 0x01010101u) ^ x; };  // bit 7 of a byte changes where the seven below are ones
  return (flip(w.x) | flip(w.y) | flip(w.z) | flip(w.w)) & 0x80808080u;
}

// Where is_nan() has met one, a warp goes through keys [lo, hi) of its unit once more, and rows that see a NaN get it; the
// others keep what they have.  A lane has token `tk` of the sequence (-1: none) and of its output the dims [d, d + run) of
// every `step` from d_lo on, at `out` or, of a part, `part`; lse, or a part's (m, l), or NULL.  Every lane comes to the
// votes, with a token or not.
template <int HD, bool kTree>
__device__ __forceinline__ void spread_nan(const AttendParams& p, const Seg& q, int lo, int hi, int tk, int d_lo, int run, int step,
                                           __nv_bfloat16* out, float* part, float* lse, float2* ml) {
  const int lane = threadIdx.x & 31, ctx = q.kv - q.n;
  const int pos = !kTree ? ctx + tk : tk >= 0 && p.window > 0 ? max(ctx, __ldg(p.positions + q.r0 + tk)) : 0;
  const int from = p.window > 0 ? max(0, kTree ? min(ctx, pos - p.window + 1) : pos - p.window + 1) : 0;
  const int to = p.causal ? min(q.kv, pos + 1) : q.kv;
  const uint32_t* mask = kTree ? reinterpret_cast<const uint32_t*>(p.masks + (int64_t)(q.r0 + max(tk, 0)) * p.words) : nullptr;
  const int32_t* table = p.page_tables + (int64_t)q.s * p.mpps;
#pragma unroll 1
  for (int lp = lo / kPage; lp * kPage < hi; ++lp) {
    const int id = __ldg(table + lp), page = id < 0 || id >= p.num_pages ? 0 : id;  // (reported by the copy)
    const uint8_t* tile = static_cast<const uint8_t*>(p.pool) + page * p.page_stride + (int64_t)q.g * (32 * HD + 32);
    bool any = false;
#pragma unroll 1
    for (int u = lane; u < 2 * HD; u += 32) any |= nan_codes(reinterpret_cast<const uint4*>(tile)[u]);
    if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll 1
    for (int j = 0; tk >= 0 && j < kPage; ++j) {
      const int key = lp * kPage + j;
      if (!(kTree ? mask_bits(mask, 2 * p.words, key, from, ctx, q.kv) & 1 : key >= from && key < to)) continue;
      bool all = false;
#pragma unroll 1
      for (int d = 0; d < HD; d += 16) all |= nan_codes(*reinterpret_cast<const uint4*>(tile + k8_in_tile(j, d)));
#pragma unroll 1
      for (int a = d_lo; a < HD; a += step)
#pragma unroll 1
        for (int d = a; d < a + run; ++d) {
          if (!all && (tile[16 * HD + v8_in_tile(j, d)] & 127) != 127) continue;
          if (out) out[d] = __ushort_as_bfloat16(0x7fff); else part[d] = NAN;
        }
      if (all && lse) *lse = NAN;
      if (all && ml) ml->y = NAN;
    }
    __syncwarp();
  }
}

}  // namespace plan
}  // namespace dflash
