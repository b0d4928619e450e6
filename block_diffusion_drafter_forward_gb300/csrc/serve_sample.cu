// One token per row of logits by temperature, top-k, top-p and min-p (dflash_sample).
//
// A cluster of C CTAs owns a row: each keeps its slice of the row in shared memory, so the logits
// are read from HBM once whatever the number of passes.  In falling order of the logits every
// filter keeps a prefix, and the prefix is short in most rows:
//   1. largest logit m (and its lowest index: the answer where T == 0);
//   2. a histogram of t = (m - x) log2(e) / T in 1024 equal bins of [0, 20) (of [0, 40) if that
//      does not reach far enough) and, for top-p alone, the row's mass: the counts give the bin in
//      which top-k ends, the bounds on a bin's mass (2 %) the last bin that top-p can reach;
//   3. the logits up to that bin, usually a few dozen, go to the first CTA, which sorts them, sums
//      their weights in fixed point and finds the kept prefix and the token.
// Rows whose prefix does not fit in the list (flat ones) find the border by bisection on the
// logits' order-preserving keys; those, and rows without top-k and top-p, then sum the kept mass of
// every warp's segment in index order, and the warp whose segment holds u * total walks it.  Passes
// skip vectors whose largest logit is below what the pass looks at.
// The token is a whole number that a sum's last bit can change, so weights are pairs of floats
// (exp2 by a 128-entry table and a short polynomial on the compensated argument, about 2^-41)
// and sums are compensated: in plain fp32 one row in a few hundred would differ.  Weights below
// 2^-20 enter top-p's total mass in plain fp32 (they hold a small part of it).
#include <cooperative_groups.h>
#include <float.h>
#include <string.h>

#include <cmath>

#include <atomic>

#include "launch_util.cuh"
#include "serve.cuh"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kMaxC = 8;
constexpr int kList = 2048;                  // logits that the sorted list holds
constexpr float kCut = 40.f;                 // weights below 2^-40 are 0
constexpr float kNear = 20.f;                // the histogram's first range of t
constexpr int kSliceBytes = 184 * 1024;      // shared memory for a CTA's slice

struct SampleParams {
  const void* logits;
  int64_t stride;  // elements
  int rows, vocab;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* tokens;
  float* probs;
  int per;  // elements of a slice (a multiple of 8)
  float2 table[128];  // 2^(j / 128) as pairs
};

// ------------------------------------------------------------------ pairs of floats
struct F2 {
  float h, l;
};
// sum of two pairs, renormalised
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  const float s = a.h + b.h, bb = s - a.h;
  const float e = (a.h - (s - bb)) + (b.h - bb) + (a.l + b.l);
  const float h = s + e;
  return {h, e - (h - s)};
}
__device__ __forceinline__ bool below(F2 a, float b) { return a.h < b || (a.h == b && a.l < 0.f); }
// Masses as whole numbers of 2^-B: sums and comparisons are exact and cost integer operations
// (fp64 runs at 1/64 of the fp32 rate here).  B = 52 where at most 2048 weights are added, 43 for
// a row's.
template <int B>
__device__ __forceinline__ unsigned long long fix(F2 a) {
  constexpr float k = (float)(1ull << B);
  return (unsigned long long)(__float2ll_rn(a.h * k) + __float2ll_rn(a.l * k));
}
// floor(a f) for 0 <= f (at least 1 counts as 1), exactly; *inexact where there is a remainder
__device__ __forceinline__ unsigned long long part_of(unsigned long long a, float f, bool* inexact = nullptr) {
  if (inexact) *inexact = false;
  if (!(f > 0.f)) return 0;
  if (f >= 1.f) return a;
  int e;
  const unsigned long long m = (unsigned long long)ldexpf(frexpf(f, &e), 24);  // f = m 2^(e - 24), e <= 0
  const unsigned long long hi = __umul64hi(a, m), lo = a * m;
  const int sh = 24 - e;
  unsigned long long r, rem;
  if (sh < 64) {
    r = hi << (64 - sh) | lo >> sh;
    rem = lo << (64 - sh);
  } else {
    r = sh - 64 < 64 ? hi >> (sh - 64) : 0;
    rem = lo | (sh - 64 < 64 ? (sh == 64 ? 0 : hi << (128 - sh)) : hi);
  }
  if (inexact) *inexact = rem != 0;
  return r;
}
__device__ __forceinline__ F2 shfl_add(F2 a, int o) {
  F2 b = {__shfl_xor_sync(0xffffffffu, a.h, o), __shfl_xor_sync(0xffffffffu, a.l, o)};
  // the same operand order on both lanes, so that both get the same sum
  return (threadIdx.x & o) ? add(b, a) : add(a, b);
}

__device__ __forceinline__ unsigned key_of(float x) {
  const unsigned b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(unsigned k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// What a row's weights depend on.
struct Scale {
  float m, c_hi, c_lo;     // largest logit; log2(e) / T as a pair
  const float2* table;     // 2^(j / 128)
};
// t = (m - x) log2(e) / T, never falling as x falls; 0 at x == m, infinity at x == -inf
__device__ __forceinline__ float t_of(const Scale& s, float x) { return x == s.m ? 0.f : (s.m - x) * s.c_hi; }

// w = exp((x - m) / T) as a pair; 0 below 2^-40.  Exactly 1 at x == m.
__device__ __forceinline__ F2 weight(const Scale& s, float x) {
  if (x == s.m) return {1.f, 0.f};
  // d = x - m without error
  const float d = x - s.m, bb = d - x;
  const float dl = (x - (d - bb)) - (s.m + bb);
  const float t = d * s.c_hi;
  if (!(t >= -kCut)) return {0.f, 0.f};
  const float tl = fmaf(d, s.c_hi, -t) + fmaf(d, s.c_lo, dl * s.c_hi);
  const float k = rintf(t * 128.f);
  const float r0 = fmaf(k, -1.f / 128.f, t);  // exact
  const float rh = r0 + tl, rl = tl - (rh - r0);
  const int ki = (int)k, j = ki & 127, e = ki >> 7;
  // y = r ln 2, 2^r = 1 + y + y^2 (1/2 + y (1/6 + y / 24)), |y| < 0.0028
  const float kL = 0.693147182464599609f, kLl = -1.90465429995776e-9f;
  const float yh = rh * kL;
  const float yl = fmaf(rh, kL, -yh) + fmaf(rh, kLl, rl * kL);
  const float q = fmaf(yh * yh, fmaf(yh, fmaf(yh, 1.f / 24.f, 1.f / 6.f), 0.5f), yl);
  const float2 T = s.table[j];
  const float a = T.x * yh, ae = fmaf(T.x, yh, -a);
  const float h = T.x + a;
  const float lo = (a - (h - T.x)) + (ae + fmaf(T.x, q, fmaf(T.y, yh, T.y)));
  const float sc = __int_as_float((e + 127) << 23);
  const float hh = h + lo;
  // the cut on the exponent itself, with its low part: w < 2^-40 iff t + tl < -40
  if (t + tl < -kCut) return {0.f, 0.f};
  return {hh * sc, (lo - (hh - h)) * sc};
}

// ------------------------------------------------------------------ shared state
struct Slot {  // what a CTA tells the others, double-buffered by exchange
  unsigned long long d[2];
  float f;
  unsigned u[4];
};
struct Shared {
  float2 table[128];
  unsigned hist[kBins];      // the slice's histogram
  Slot slot[2];
  unsigned long long wsum[kWarps];  // kept mass of each warp's segment
  unsigned wties[kWarps];    // logits equal to tau in it
  unsigned long long all_sum[kMaxC * kWarps];
  unsigned all_ties[kMaxC * kWarps];
  float red_f[2][kWarps];
  unsigned red_u[4][kWarps];
  unsigned long long red_l[2][kWarps];
  int pick[4];
  unsigned n_list;
  unsigned index[kList];               // of the sorted list: vocabulary index
  unsigned long long list[kList];      // (~key, index), then fixed-point weights
};

// 16 bytes of logits: their largest (NaN counts as nothing), and the values.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr unsigned kPad = 0xff80ff80u;  // -inf twice
  __device__ static float top(const uint4& r) {
    const __nv_bfloat162 a = __hmax2(reinterpret_cast<const __nv_bfloat162&>(r.x), reinterpret_cast<const __nv_bfloat162&>(r.y));
    const __nv_bfloat162 b = __hmax2(reinterpret_cast<const __nv_bfloat162&>(r.z), reinterpret_cast<const __nv_bfloat162&>(r.w));
    const __nv_bfloat162 m = __hmax2(a, b);
    return fmaxf(__low2float(m), __high2float(m));
  }
  __device__ static void get(const uint4& r, float (&v)[8]) {
    const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static constexpr unsigned kPad = 0xff800000u;
  __device__ static float top(const uint4& r) {
    return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
  __device__ static void get(const uint4& r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
  }
};

template <typename T, int C>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p) {
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(16) uint8_t smem[];
  T* xs = reinterpret_cast<T*>(smem);
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int rank = C > 1 ? (int)cl.block_rank() : 0, row = blockIdx.x / C;
  int phase = 0;
  auto sync_row = [&] {
    if (C > 1) cl.sync(); else __syncthreads();
  };
  auto peer = [&](auto* ptr, int r) { return C > 1 ? cl.map_shared_rank(ptr, r) : ptr; };

  // ---- the slice.  Positions count from the 16-byte boundary at or before the row's first logit
  // (`skip` of them lie before it), so that vectors are aligned whatever the row's address;
  // position i of this CTA's slice is logit first + i.  Positions outside the row hold -inf.
  const T* src = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
  const int skip = (int)(reinterpret_cast<uintptr_t>(src) & 15) / (int)sizeof(T);
  const int first = rank * p.per - skip;
  const int count = max(0, min(p.per, p.vocab - first)), begin = max(0, -first);
  const int padded = (count + N * 32 * kWarps - 1) / (N * 32 * kWarps) * (N * 32 * kWarps);
  float best = -INFINITY;
#pragma unroll 4
  for (int i = t * N; i < padded; i += kThreads * N) {
    uint4 r;
    if (i >= begin && i + N <= count) {
      r = __ldcs(reinterpret_cast<const uint4*>(src + first + i));
    } else {  // the row's ends
      r = make_uint4(Vec<T>::kPad, Vec<T>::kPad, Vec<T>::kPad, Vec<T>::kPad);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (i + e >= begin && i + e < count) reinterpret_cast<T*>(&r)[e] = src[first + i + e];
    }
    best = fmaxf(best, Vec<T>::top(r));
    *reinterpret_cast<uint4*>(xs + i) = r;
  }
  if (t < 128) sh.table[t] = p.table[t];
  for (int b = t; b < kBins; b += kThreads) sh.hist[b] = 0;
  if (t == 0) sh.n_list = 0;

  // reductions over the row; every thread of every CTA gets the same result
  auto row_max = [&](float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (lane == 0) sh.red_f[0][warp] = v;
    __syncthreads();
    if (t == 0) {
      float r = sh.red_f[0][0];
      for (int w = 1; w < kWarps; ++w) r = fmaxf(r, sh.red_f[0][w]);
      sh.slot[phase].f = r;
    }
    sync_row();
    float r = -INFINITY;
#pragma unroll
    for (int c = 0; c < C; ++c) r = fmaxf(r, peer(&sh.slot[phase], c)->f);
    phase ^= 1;
    return r;
  };
  // op 0: sum, 1: min, 2: max of unsigned values
  auto row_u = [&](unsigned (&v)[2], int op0, int op1) {
    const int op[2] = {op0, op1};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const unsigned r = op[k] == 0 ? __reduce_add_sync(0xffffffffu, v[k])
                                    : op[k] == 1 ? __reduce_min_sync(0xffffffffu, v[k]) : __reduce_max_sync(0xffffffffu, v[k]);
      if (lane == 0) sh.red_u[k][warp] = r;
    }
    __syncthreads();
    if (t < 2) {
      unsigned r = sh.red_u[t][0];
      for (int w = 1; w < kWarps; ++w) {
        const unsigned x = sh.red_u[t][w];
        r = op[t] == 0 ? r + x : op[t] == 1 ? min(r, x) : max(r, x);
      }
      sh.slot[phase].u[t] = r;
    }
    sync_row();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      unsigned r = peer(&sh.slot[phase], 0)->u[k];
#pragma unroll
      for (int c = 1; c < C; ++c) {
        const unsigned x = peer(&sh.slot[phase], c)->u[k];
        r = op[k] == 0 ? r + x : op[k] == 1 ? min(r, x) : max(r, x);
      }
      v[k] = r;
    }
    phase ^= 1;
  };
  auto row_sum2 = [&](F2 a, F2 b, unsigned long long (&out)[2]) {  // in units of 2^-43
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = shfl_add(a, o), b = shfl_add(b, o);
    if (lane == 0) sh.red_l[0][warp] = fix<43>(a), sh.red_l[1][warp] = fix<43>(b);
    __syncthreads();
    if (t < 2) {
      unsigned long long r = 0;
      for (int w = 0; w < kWarps; ++w) r += sh.red_l[t][w];
      sh.slot[phase].d[t] = r;
    }
    sync_row();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      unsigned long long r = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) r += peer(&sh.slot[phase], c)->d[k];
      out[k] = r;
    }
    phase ^= 1;
  };
  // f(position, logit) over this thread's elements of vectors whose largest is at least `from`: warp
  // w has the contiguous segment of `seg` positions from w * seg on, lanes take vectors of it in
  // turn.  NaN and -0 come as -inf and +0 (equal logits have equal keys).
  const int seg = padded / kWarps;
  auto each = [&](float from, auto&& f) {
    for (int i = warp * seg + lane * N; i < (warp + 1) * seg; i += 32 * N) {
      const uint4 r = *reinterpret_cast<const uint4*>(xs + i);
      if (!(Vec<T>::top(r) >= from)) continue;
      float v[N];
      Vec<T>::get(r, v);
#pragma unroll
      for (int e = 0; e < N; ++e) f(i + e, v[e] == v[e] ? v[e] + 0.f : -INFINITY);
    }
  };

  const float m = row_max(best);  // also: the slice, the table and the zeroed bins are visible
  const float T_row = p.temperature ? p.temperature[row] : 1.f;
  const int k_row = p.top_k ? p.top_k[row] : 0;
  const float p_row = p.top_p ? p.top_p[row] : 1.f;
  const float lo_row = p.min_p ? p.min_p[row] : 0.f;
  float u_row = p.u[row];
  u_row = u_row > 0.f ? u_row : 0.f;
  const bool valid = m > -INFINITY && T_row >= 0.f && T_row <= FLT_MAX;
  if (!valid || T_row == 0.f) {
    unsigned v[2] = {0xffffffffu, 0};
    if (valid)
      each(m, [&](int i, float x) { v[0] = x == m && i < count ? min(v[0], (unsigned)(first + i)) : v[0]; });
    row_u(v, 1, 0);
    if (rank == 0 && t == 0) {
      p.tokens[row] = valid ? (int)v[0] : -1;
      if (p.probs) p.probs[row] = valid ? 1.f : 0.f;
    }
    sync_row();  // no CTA leaves while another reads its shared memory
    return;
  }
  // log2(e) / T as a pair: quotient, and the exact remainder's quotient
  constexpr float kE = 1.44269502162933349609375f, kEl = 1.92596299e-8f;  // log2(e)
  Scale sc;
  sc.m = m;
  sc.c_hi = kE / T_row;
  sc.c_lo = isinf(sc.c_hi) ? 0.f : (fmaf(-sc.c_hi, T_row, kE) + kEl) / T_row;
  sc.table = sh.table;
  // a logit from which on t can be below r (rounding allowed for)
  auto reach = [&](float r) { return isinf(sc.c_hi) || isinf(m) ? m : m - r / sc.c_hi * 1.00001f - fabsf(m) * 1e-6f; };

  // ---- (tau, n): keys above tau are kept, and the n first of those equal to it
  unsigned tau = key_of(-INFINITY), n_tau = 0;  // -inf itself is never drawn
  bool use_k = k_row > 0 && k_row < p.vocab;
  const bool use_p = p_row < 1.f;
  const float p_pos = fmaxf(p_row, 0.f);
  if (use_k || use_p) {
    const bool had_k = use_k;
    constexpr int kB = kBins / kThreads;  // thread t owns bins kB t .. of the falling logits
    float bin_scale = 0.f;
    int bin_k = 0, bin_end = 0;           // top-k's last bin; the last bin that the prefix can reach
    unsigned above_k = 0, n_list = 0, cnt[kB], cum0 = 0;
    unsigned long long mass = 0, tail = 0;  // of the row and of its logits past the range (top-p without top-k)
    auto bin_of = [&](float x) {
      const float b = t_of(sc, x) * bin_scale;
      return b < kBins ? (int)b : kBins;
    };
    auto before_u = [&](unsigned v, unsigned* all) {  // sum over lower threads
      unsigned inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      if (lane == 31) sh.red_u[0][warp] = inc;
      __syncthreads();
      unsigned b = inc - v, a = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) b += sh.red_u[0][w];
        a += sh.red_u[0][w];
      }
      __syncthreads();
      *all = a;
      return b;
    };
    // sums over the bins of lower threads (bounds, loose enough for fp32 sums)
    auto before_f = [&](float v, int slot, float* all) {
      float inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      if (lane == 31) sh.red_f[slot][warp] = inc;
      __syncthreads();
      float b = inc - v, a = 0.f;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) b += sh.red_f[slot][w];
        a += sh.red_f[slot][w];
      }
      *all = a;
      return b;
    };
    auto lo_of = [&](int bin) { return exp2f(-(bin + 1.001f) / bin_scale) * 0.999f; };
    auto up_of = [&](int bin) { return exp2f(-(bin - 0.001f) / bin_scale) * 1.001f; };

    for (int far = 0;; ++far) {  // t in [0, 20), then in [0, 40)
      const float range = far ? kCut : kNear;
      bin_scale = kBins / range;
      F2 near = {0, 0};
      float rest = 0.f;
      const bool sum = use_p && !use_k && !far;
      each(reach(sum ? kCut : range), [&](int, float x) {
        const int b = bin_of(x);
        if (b < kBins) {
          atomicAdd(&sh.hist[b], 1u);
          if (sum) near = add(near, weight(sc, x));
        } else if (sum) {
          const float tt = t_of(sc, x);
          rest += tt <= kCut ? exp2f(-tt) : 0.f;
        }
      });
      if (sum) {
        unsigned long long s2[2];
        row_sum2(near, F2{rest, 0.f}, s2);  // (and the row's histograms are complete)
        mass = s2[0] + s2[1];
        tail = s2[1];
      } else {
        sync_row();
        tail = 0;
      }
      unsigned mine = 0, n_all;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        cnt[b] = 0;
#pragma unroll
        for (int r = 0; r < C; ++r) cnt[b] += peer(sh.hist, r)[t * kB + b];
        mine += cnt[b];
      }
      if (t < 4) sh.pick[t] = t < 2 ? -1 : kBins - 1;
      cum0 = before_u(mine, &n_all);
      unsigned cum = cum0;
      bool found;
      if (use_k) {  // the bin in which the count reaches k
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          if (cum < (unsigned)k_row && cum + cnt[b] >= (unsigned)k_row) sh.pick[0] = t * kB + b, sh.pick[1] = (int)cum;
          cum += cnt[b];
        }
        __syncthreads();
        bin_k = bin_end = sh.pick[0];
        above_k = (unsigned)sh.pick[1];
        found = bin_k >= 0;
      } else {      // the first bin by which the goal is surely reached: by what lies before, or what is left
        float lo_s = 0.f, up_s = 0.f, lo_all, up_all;
#pragma unroll
        for (int b = 0; b < kB; ++b) lo_s += cnt[b] * lo_of(t * kB + b), up_s += cnt[b] * up_of(t * kB + b);
        float lo_run = before_f(lo_s, 0, &lo_all), up_run = before_f(up_s, 1, &up_all);
        const float whole = (float)mass * 0x1p-43f, left = (float)tail * 0x1.001p-43f;
        const float goal = p_pos * whole * 1.0001f, spare = (1.f - p_pos) * whole * 0.999f;
        bool any = false;
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          lo_run += cnt[b] * lo_of(t * kB + b);
          up_run += cnt[b] * up_of(t * kB + b);
          if (cnt[b] > 0 && (lo_run >= goal || (up_all - up_run) + up_all * 1e-5f + left <= spare)) {
            atomicMin(&sh.pick[2], t * kB + b);
            any = true;
          }
        }
        found = __syncthreads_or(any);
        bin_end = sh.pick[2];
      }
      if (found || far) {
        if (!found) {  // every weight above 0 counts
          bin_end = kBins - 1;
          use_k = false;
        }
        // logits in bins up to bin_end
        cum = cum0;
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          cum += cnt[b];
          if (t * kB + b == bin_end) sh.pick[3] = (int)cum;
        }
        __syncthreads();
        n_list = (unsigned)sh.pick[3];
        if (n_list <= kList || far) break;
      }
      // look further: zero the histogram once every CTA has read it
      sync_row();
      for (int b = t; b < kBins; b += kThreads) sh.hist[b] = 0;
      __syncthreads();
    }

    if (n_list <= kList) {
      // ---- the list, in the first CTA
      unsigned long long* list = peer(sh.list, 0);
      unsigned* n_at = peer(&sh.n_list, 0);
      each(reach((bin_end + 1) / bin_scale), [&](int i, float x) {
        if (bin_of(x) <= bin_end)
          list[atomicAdd(n_at, 1u)] = (unsigned long long)~key_of(x) << 32 | (unsigned)(first + i);
      });
      sync_row();
      if (rank != 0) return;  // nothing of the other CTAs' is read from here on
      const int n = (int)n_list;
      int n2 = 64;
      while (n2 < n) n2 *= 2;
      for (int i = n + t; i < n2; i += kThreads) sh.list[i] = ~0ull;
      __syncthreads();
      // bitonic sort by (falling logit, index)
      if (n2 > 64 || warp == 0) {
        for (int len = 2; len <= n2; len *= 2) {
          for (int d = len / 2; d > 0; d /= 2) {
            for (int i = t; i < n2 / 2; i += kThreads) {
              const int a = 2 * i - (i & (d - 1)), b = a + d;
              const unsigned long long va = sh.list[a], vb = sh.list[b];
              if ((va > vb) == ((a & len) == 0)) sh.list[a] = vb, sh.list[b] = va;
            }
            if (n2 > 64) __syncthreads(); else __syncwarp();
          }
        }
      }
      __syncthreads();
      // thread t has items [t per, (t + 1) per): weights and their running sum
      const int per = max(1, n2 / kThreads), i0 = t * per;
      constexpr int kPer = kList / kThreads;
      unsigned long long w[kPer], mine = 0;
      unsigned idx[kPer];
      bool low[kPer];  // below min-p
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        w[e] = 0, idx[e] = 0, low[e] = false;
        if (e < per && i0 + e < n) {
          const unsigned long long it = sh.list[i0 + e];
          const F2 f = weight(sc, of_key(~(unsigned)(it >> 32)));
          w[e] = fix<52>(f);
          low[e] = below(f, lo_row);
          idx[e] = (unsigned)it;
        }
        mine += w[e];
      }
      auto scan_l = [&](unsigned long long v) {  // sum over lower threads
        unsigned long long inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        if (lane == 31) sh.red_l[0][warp] = inc;
        __syncthreads();
        unsigned long long b = inc - v;
        for (int q = 0; q < warp; ++q) b += sh.red_l[0][q];
        __syncthreads();
        return b;
      };
      const unsigned long long before = scan_l(mine);
      const int k_end = use_k ? min(n, k_row) : n;
      unsigned long long goal = ~0ull;  // kept: what lies before is below it
      if (use_p) {
        int up = 9;  // the row's mass is in units of 2^-43
        if (had_k) {  // that left by top-k is all in the list
          unsigned long long run = before;
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            run += w[e];
            if (e < per && i0 + e == k_end - 1) sh.red_l[1][0] = run;
          }
          __syncthreads();
          mass = sh.red_l[1][0];
          up = 0;
        } else if (mass < 1ull << 54) {
          mass <<= up;
          up = 0;
        }
        bool more;
        goal = part_of(mass, p_pos, &more);
        goal += more;
        goal = goal >> (64 - up - 1) > 1 ? ~0ull : goal << up;  // (a prefix in the list is below 2^63)
      }
      // the kept prefix: its length and mass
      unsigned long long run = before, kept_w = 0;
      int kept_n = 0;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int i = i0 + e;
        const bool in = e < per && i < k_end && (i == 0 || run < goal) && !low[e] && w[e] > 0;
        run += w[e];
        if (in) ++kept_n, kept_w += w[e];
      }
      int n_kept = __reduce_add_sync(0xffffffffu, kept_n);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) kept_w += __shfl_xor_sync(0xffffffffu, kept_w, o);
      if (lane == 0) sh.red_u[0][warp] = n_kept, sh.red_l[0][warp] = kept_w;
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (e < per && i0 + e < n) sh.index[i0 + e] = idx[e], sh.list[i0 + e] = w[e];
      if (t == 0) sh.pick[0] = 0x7fffffff, sh.pick[1] = -1;
      __syncthreads();
      n_kept = 0;
      kept_w = 0;
      for (int q = 0; q < kWarps; ++q) n_kept += sh.red_u[0][q], kept_w += sh.red_l[0][q];
      const unsigned long long target = part_of(kept_w, u_row);
      // the lowest index at which the running sum by index exceeds the target, else the last one
      // (packed with the item's place: below 2^20 and 2^11)
      if (n_kept <= 128) {
        if (t < n_kept) {
          const unsigned me = sh.index[t];
          unsigned long long s = 0;
          for (int j = 0; j < n_kept; ++j) s += sh.index[j] <= me ? sh.list[j] : 0ull;
          const int at = (int)(me << 11 | t);
          if (s > target) atomicMin(&sh.pick[0], at);
          atomicMax(&sh.pick[1], at);
        }
      } else {
        int m2 = 256;
        while (m2 < n_kept) m2 *= 2;
        unsigned* by = reinterpret_cast<unsigned*>(xs);  // the slice is not read any more
        for (int i = t; i < m2; i += kThreads) by[i] = i < n_kept ? sh.index[i] << 11 | i : 0xffffffffu;
        __syncthreads();
        for (int len = 2; len <= m2; len *= 2) {
          for (int d = len / 2; d > 0; d /= 2) {
            for (int i = t; i < m2 / 2; i += kThreads) {
              const int a = 2 * i - (i & (d - 1)), b = a + d;
              const unsigned va = by[a], vb = by[b];
              if ((va > vb) == ((a & len) == 0)) by[a] = vb, by[b] = va;
            }
            __syncthreads();
          }
        }
        const int q = max(1, m2 / kThreads), j0 = t * q;
        unsigned long long s = 0;
        for (int e = 0; e < q; ++e)
          if (j0 + e < n_kept) s += sh.list[by[j0 + e] & 2047];
        s = scan_l(s);
        for (int e = 0; e < q; ++e) {
          if (j0 + e >= n_kept) break;
          s += sh.list[by[j0 + e] & 2047];
          if (s > target) {
            atomicMin(&sh.pick[0], (int)by[j0 + e]);
            break;
          }
        }
        if (t == 0) sh.pick[1] = (int)by[n_kept - 1];
      }
      __syncthreads();
      if (t == 0) {
        const int at = sh.pick[0] != 0x7fffffff ? sh.pick[0] : sh.pick[1];
        p.tokens[row] = at >= 0 ? at >> 11 : -1;
        if (p.probs) p.probs[row] = at >= 0 ? (float)((double)sh.list[at & 2047] / (double)kept_w) : 0.f;
      }
      return;
    }

    // ---- the list is too long (the histogram is that of [0, 40)): bisection
    if (use_k) {
      // smallest and largest key in top-k's bin, then the largest tau with count(key >= tau) >= k
      unsigned v[2] = {0xffffffffu, 0u};
      const float from = reach((bin_k + 1) / bin_scale);
      each(from, [&](int, float x) {
        if (bin_of(x) == bin_k) v[0] = min(v[0], key_of(x)), v[1] = max(v[1], key_of(x));
      });
      row_u(v, 1, 2);
      unsigned lo = v[0], hi = v[1], above = above_k;
      while (lo < hi) {
        const unsigned mid = lo + (hi - lo + 1) / 2;
        unsigned n[2] = {0, 0};
        each(of_key(mid), [&](int, float x) { n[0] += bin_of(x) == bin_k && key_of(x) >= mid; });
        row_u(n, 0, 0);
        if (above_k + n[0] >= (unsigned)k_row) lo = mid; else hi = mid - 1, above = above_k + n[0];
      }
      n_tau = (unsigned)k_row - above;
      tau = lo;
    }
    if (use_p) {
      // bounds on the mass of every bin, cut at k: the bins in which the goal can be reached
      float lo_m = 0.f, up_m = 0.f, lo_b[kB], up_b[kB];
      unsigned cum = cum0;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const int bin = t * kB + b;
        const unsigned kept = !use_k ? cnt[b] : cum >= (unsigned)k_row ? 0u : min(cnt[b], (unsigned)k_row - cum);
        cum += cnt[b];
        lo_b[b] = kept * lo_of(bin);
        up_b[b] = kept * up_of(bin);
        lo_m += lo_b[b], up_m += up_b[b];
      }
      float lo_all, up_all;
      float lo_c = before_f(lo_m, 0, &lo_all), up_c = before_f(up_m, 1, &up_all);
      __syncthreads();
      if (t < 2) sh.pick[2 + t] = kBins - 1;
      __syncthreads();
      const float p_lo = p_pos * lo_all * 0.999f, p_up = p_pos * up_all * 1.001f;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        lo_c += lo_b[b], up_c += up_b[b];
        if (up_c >= p_lo) atomicMin(&sh.pick[2], t * kB + b);
        if (lo_c >= p_up) atomicMin(&sh.pick[3], t * kB + b);
      }
      __syncthreads();
      const int b0 = sh.pick[2], b1 = sh.pick[3];
      // the mass left by top-k, and its part in the bins before b0
      const unsigned tau_k = tau, n_k = n_tau;
      const bool tie_in = n_k > 0;
      const unsigned long long w_k = tie_in ? n_k * fix<43>(weight(sc, of_key(tau_k))) : 0ull;  // the ties' mass
      F2 all = {0, 0}, head = {0, 0};
      unsigned v[2] = {0xffffffffu, 0u};
      each(fmaxf(reach(kCut), of_key(tau_k)), [&](int, float x) {
        const unsigned key = key_of(x);
        if (key < tau_k || (key == tau_k && n_k == 0)) return;
        const int b = bin_of(x);
        if (b >= b0 && b <= b1) v[0] = min(v[0], key), v[1] = max(v[1], key);
        if (key > tau_k) {
          const F2 w = weight(sc, x);
          all = add(all, w);
          if (b < b0) head = add(head, w);
        }
      });
      unsigned long long sums[2];
      row_sum2(all, head, sums);
      row_u(v, 1, 2);
      const int bin_tau = tie_in ? bin_of(of_key(tau_k)) : kBins;
      const unsigned long long base = sums[1] + (bin_tau < b0 ? w_k : 0ull);
      bool rem;
      unsigned long long goal = part_of(sums[0] + w_k, p_pos, &rem);
      goal += rem;
      unsigned lo = v[0], hi = v[1];
      if (lo <= hi) {
        unsigned long long above = base;  // mass of the keys above hi
        while (lo < hi) {
          const unsigned mid = lo + (hi - lo + 1) / 2;
          F2 s = {0, 0};
          each(of_key(mid), [&](int, float x) {
            const unsigned key = key_of(x);
            if (key < mid || key <= tau_k) return;
            const int b = bin_of(x);
            if (b >= b0 && b <= b1) s = add(s, weight(sc, x));
          });
          unsigned long long r[2];
          row_sum2(s, F2{0, 0}, r);
          const unsigned long long f = base + r[0] + (tau_k >= mid && bin_tau >= b0 ? w_k : 0ull);
          if (f >= goal) lo = mid; else hi = mid - 1, above = f;
        }
        // of the keys equal to tau: those before which less than the goal lies
        if (t == 0) {
          const F2 w = weight(sc, of_key(lo));
          const double need = goal > above ? (double)(goal - above) * 0x1p-43 : 0.0;
          const double more = w.h > 0.f ? ceil(need / ((double)w.h + (double)w.l)) : 1.0;
          sh.pick[0] = (int)fmin(more, 2e9);
        }
        __syncthreads();
        const unsigned more = (unsigned)sh.pick[0];
        const unsigned n_p = more == 0 && goal == 0 && lo == key_of(m) ? 1u : more;  // the first always stays
        n_tau = lo == tau_k && tie_in ? min(n_k, n_p) : n_p;
        tau = lo;
      }
    }
  }

  // ---- ties at tau before each warp's segment
  const bool ties = use_k || use_p;
  unsigned my_ties = 0;
  if (ties) {
    each(of_key(tau), [&](int i, float x) { my_ties += key_of(x) == tau && i >= begin && i < count; });
    my_ties = __reduce_add_sync(0xffffffffu, my_ties);
  }
  unsigned ties_before = 0;
  if (ties) {
    if (lane == 0) sh.wties[warp] = my_ties;
    sync_row();
    if (t < C * kWarps) sh.all_ties[t] = peer(sh.wties, t / kWarps)[t % kWarps];
    __syncthreads();
    for (int w = 0; w < rank * kWarps + warp; ++w) ties_before += sh.all_ties[w];
  }
  // f(index, logit, kept weight) over this warp's segment in order, a vector per lane at a time
  // (a weight has to reach min-p; the largest one does, or none)
  const float from = fmaxf(fmaxf(reach(kCut), of_key(tau)), lo_row > 0.f && lo_row < 1.f ? reach(-log2f(lo_row) + 0.01f) : -INFINITY);
  auto kept = [&](auto&& f) {
    unsigned rank0 = ties_before;
    const bool some = ties && ties_before < n_tau && ties_before + my_ties > n_tau;  // the n-th tie is here
    const bool whole = ties && ties_before + my_ties <= n_tau;
    for (int i0 = warp * seg; i0 < (warp + 1) * seg; i0 += 32 * N) {
      const uint4 r = *reinterpret_cast<const uint4*>(xs + i0 + lane * N);
      if (!__any_sync(0xffffffffu, Vec<T>::top(r) >= from)) continue;  // nothing kept here
      float v[N];
      Vec<T>::get(r, v);
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = v[e] == v[e] ? v[e] + 0.f : -INFINITY;
      unsigned eq = 0, at = 0;
      if (some) {
#pragma unroll
        for (int e = 0; e < N; ++e) eq += key_of(v[e]) == tau && i0 + lane * N + e >= begin && i0 + lane * N + e < count;
        unsigned inc = eq;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        at = rank0 + inc - eq;
        rank0 += __shfl_sync(0xffffffffu, inc, 31);
      }
      F2 w[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const unsigned key = key_of(v[e]);
        bool in = key > tau;
        if (ties && key == tau) in = some ? at++ < n_tau : whole;
        w[e] = F2{0.f, 0.f};
        if (in) {
          w[e] = weight(sc, v[e]);
          if (below(w[e], lo_row)) w[e] = F2{0.f, 0.f};
        }
      }
      if (!f(i0, w)) break;
    }
  };
  F2 sum = {0, 0};
  kept([&](int, F2 (&w)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) sum = add(sum, w[e]);
    return true;
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum = shfl_add(sum, o);
  if (lane == 0) sh.wsum[warp] = fix<43>(sum);
  sync_row();
  if (t < C * kWarps) sh.all_sum[t] = peer(sh.wsum, t / kWarps)[t % kWarps];
  __syncthreads();
  // the first segment whose running sum exceeds the target (else the last with any mass): lane l
  // has segments [l kS, (l + 1) kS)
  constexpr int kS = (C * kWarps + 31) / 32;
  unsigned long long seg_w[kS], inc = 0;
#pragma unroll
  for (int e = 0; e < kS; ++e) {
    seg_w[e] = lane * kS + e < C * kWarps ? sh.all_sum[lane * kS + e] : 0ull;
    inc += seg_w[e];
  }
  unsigned long long run = inc;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  const unsigned long long total = __shfl_sync(0xffffffffu, inc, 31);
  const unsigned long long target = part_of(total, u_row);
  run = inc - run;
  int mine_at = -1;  // this lane's first segment past the target, else its last with any mass
  unsigned long long mine_before = 0;
  bool past = false;
#pragma unroll
  for (int e = 0; e < kS; ++e) {
    if (seg_w[e] > 0 && !past) mine_at = lane * kS + e, mine_before = run, past = run + seg_w[e] > target;
    run += seg_w[e];
  }
  const unsigned hit_lanes = __ballot_sync(0xffffffffu, past), any_lanes = __ballot_sync(0xffffffffu, mine_at >= 0);
  int owner = -1;
  unsigned long long before = 0;
  if (any_lanes) {
    const int from_lane = hit_lanes ? __ffs(hit_lanes) - 1 : 31 - __clz(any_lanes);
    owner = __shfl_sync(0xffffffffu, mine_at, from_lane);
    before = __shfl_sync(0xffffffffu, mine_before, from_lane);
  }
  if (owner < 0 && rank == 0 && t == 0) {  // min-p above 1: nothing is left
    p.tokens[row] = -1;
    if (p.probs) p.probs[row] = 0.f;
  }
  if (owner == rank * kWarps + warp) {
    int token = -1;  // so far: the last kept position seen
    float wt = 0.f;
    kept([&](int i0, F2 (&w)[N]) {
      unsigned long long f[N], mine = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] = fix<43>(w[e]), mine += f[e];
      unsigned long long inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      // this lane's first position past the target, else its last kept one
      unsigned long long cum = before + (inc - mine);
      float my_w = 0.f;
      int my = -1;
      bool hit = false;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        cum += f[e];
        if (f[e] > 0 && !hit) {
          my = i0 + lane * N + e;
          my_w = w[e].h;
          hit = cum > target;
        }
      }
      const unsigned hits = __ballot_sync(0xffffffffu, hit), any = __ballot_sync(0xffffffffu, my >= 0);
      if (any) {
        const int from_lane = hits ? __ffs(hits) - 1 : 31 - __clz(any);
        token = __shfl_sync(0xffffffffu, my, from_lane);
        wt = __shfl_sync(0xffffffffu, my_w, from_lane);
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
      return hits == 0;
    });
    if (lane == 0) {
      p.tokens[row] = token >= 0 ? first + token : -1;
      if (p.probs) p.probs[row] = token >= 0 ? wt / ((float)total * 0x1p-43f) : 0.f;
    }
  }
  sync_row();  // no CTA leaves while another reads its shared memory
}

struct Powers {  // 2^(j / 128) as pairs of floats
  float2 table[128];
  Powers() {
    for (int j = 0; j < 128; ++j) {
      const double w = std::exp2(j / 128.0);
      table[j].x = (float)w;
      table[j].y = (float)(w - (double)table[j].x);
    }
  }
};

template <typename T, int C>
cudaError_t launch(const SampleParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  if (cudaError_t e = smem_attr_once(sample_kernel<T, C>, kSliceBytes, attr); e != cudaSuccess) return e;
  constexpr int step = Vec<T>::N * kThreads;
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = C;
  a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
  c.gridDim = dim3(p.rows * C);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = (p.per + step - 1) / step * step * sizeof(T);
  c.stream = st;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, sample_kernel<T, C>, p);
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" int dflash_sample(const void* logits, int64_t row_stride, int32_t dtype, int32_t rows, int32_t vocab,
                             const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                             const float* min_p, int32_t* tokens, float* probs, dflash_stream stream) {
  if (dtype != DFLASH_BF16 && dtype != DFLASH_F32) return call_error(DFLASH_EINVAL, "sample: dtype must be bf16 or f32");
  if (rows < 0 || vocab < 1 || row_stride < vocab) return call_error(DFLASH_EINVAL, "sample: rows >= 0, vocab >= 1 and row_stride >= vocab");
  if (vocab > (dtype == DFLASH_F32 ? 376000 : 752000))
    return call_error(DFLASH_EUNSUPPORTED, "sample: vocab above 376000 (fp32) or 752000 (bf16)");
  if (rows > (1 << 28) - 1) return call_error(DFLASH_ECAPACITY, "sample: too many rows for one call");
  if (rows == 0) return DFLASH_OK;
  if (!logits || !u || !tokens) return call_error(DFLASH_EINVAL, "sample: null pointer");
  SampleParams p{logits, row_stride, rows, vocab, u, temperature, top_p, min_p, top_k, tokens, probs, 0, {}};
  static const Powers powers;
  memcpy(p.table, powers.table, sizeof p.table);
  p.per = (vocab + 7 + kMaxC - 1) / kMaxC;  // (up to 7 positions before an unaligned row)
  p.per = (p.per + 7) / 8 * 8;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DFLASH_F32 ? launch<float, kMaxC>(p, st) : launch<__nv_bfloat16, kMaxC>(p, st);
  if (e != cudaSuccess) return call_error(DFLASH_ECUDA, "sample", e);
  return DFLASH_OK;
}
