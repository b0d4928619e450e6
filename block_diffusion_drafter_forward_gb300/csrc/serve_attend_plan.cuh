// Shared by the tensor-core forms of dflash_attend: units, their chunks, and each CTA's share of them.
//
// The chunks of all units, in (sequence, tile, head) order, form one index space; CTA b of a
// one-CTA-per-SM grid takes slots [b W / n, (b + 1) W / n) of it, sized on the device from the
// lengths.  G: a form's geometry - keys of a chunk, slots a unit occupies beside its chunks (the cost of
// opening a segment: queries, pipeline restart, output), threads of a CTA.
//
// Trees in units of two tiles: a chunk takes a CTA 2.3 us, or 1.55 where the unit's second tile has no token (33 to 48
// nodes of 8 heads to a K/V head have one such unit of two), so that chunks occupy three slots or two, and belong to
// the CTA that has their first: 32 trees of 33 nodes 155 -> 137 us, of 48 158 -> 145, of 64 (all two tiles) 161 as
// before.  (Slots of 5 and 3: 163 for trees of mixed sizes, of 4 and 3 152, of 3 and 2 154.  Without trees a chunk is
// one slot: a cut elsewhere would round results differently from before.)
#pragma once

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
constexpr int kTwo = 3, kOne = 2;
template <bool kTree>
__device__ __forceinline__ int chunk_slots(const Shape& h, int n, int tile) {
  return !kTree || h.TT == h.T ? 1 : tile * h.TT + h.T < n ? kTwo : kOne;
}
template <class G, bool kTree>
__device__ __forceinline__ int cost_slots(const Shape& h) { return G::kUnitCost * (!kTree || h.TT == h.T ? 1 : kTwo); }
template <class G, bool kTree>
__device__ __forceinline__ int unit_slots(const AttendParams& p, const Shape& h, int n, int kv, int tile) {
  int k0;
  return unit_chunks<G, kTree>(p, h, n, kv, tile, &k0) * chunk_slots<kTree>(h, n, tile) + cost_slots<G, kTree>(h);
}
// CTAs that the W slots are cut for: each has the first slot of a chunk wherever a unit goes on on both its sides.
template <bool kTree>
__device__ __forceinline__ int ctas_of(const Shape& h, long long W) {
  return (int)min((long long)gridDim.x, !kTree || h.TT == h.T ? W : W / kTwo);
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
      const int w = chunk_slots<kTree>(h, q.n, tile);
      const long long first = pu + cost_slots<G, kTree>(h);
      pu = first + (long long)q.nch * w;
      if (++g == p.nkv) {
        g = 0;
        if (++tile * h.TT >= q.n) tile = 0, ++s;
      }
      if (hi <= first || lo >= pu) continue;  // only cost slots of it are in range
      auto chunks = [&](int slots) { return w == 1 ? slots : w == kOne ? (slots + kOne - 1) / kOne : (slots + kTwo - 1) / kTwo; };
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
    const int ctas = ctas_of<kTree>(h, W), b = blockIdx.x;
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
  const int ctas = ctas_of<kTree>(h, W), b = blockIdx.x;
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

}  // namespace plan
}  // namespace dflash
