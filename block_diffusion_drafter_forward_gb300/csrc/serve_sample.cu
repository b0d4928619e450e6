// One token per row of logits by temperature, top-k, top-p and min-p (dflash_sample).
//
// A cluster of C CTAs owns a row: each keeps its slice of the row in shared memory, so the logits
// are read from HBM once whatever the number of passes.  All filters reduce to one pair (tau, n):
// logits above tau are kept, and of those equal to tau the n of lowest index.
//   1. largest logit m (and its lowest index: the answer where T == 0);
//   2. a histogram of t = (m - x) log2(e) / T in 2048 equal bins of [0, 40): exact counts give
//      top-k's bin, and bounds on the mass (a bin spans 1.4 %) give the few bins in which top-p's
//      border can lie;
//   3. bisection on the logits' order-preserving keys inside those bins: counts for top-k, masses
//      for top-p (the mass above the bins and the total come from one pass);
//   4. the kept mass of every warp's segment, in index order; the warp whose segment holds
//      u * total walks it.
// The token is a whole number that a sum's last bit can change, so weights are pairs of floats
// (exp2 by a 128-entry table and a short polynomial on the compensated argument, about 2^-41)
// and sums are compensated: in plain fp32 one row in a few hundred would differ.
#include <cooperative_groups.h>
#include <float.h>

#include <atomic>

#include "launch_util.cuh"
#include "serve.cuh"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxC = 8;
constexpr float kCut = 40.f;                 // weights below 2^-40 are 0
constexpr float kBinScale = kBins / kCut;    // 51.2 bins per unit of t
constexpr int kSliceBytes = 200 * 1024;      // shared memory for a CTA's slice

struct SampleParams {
  const void* logits;
  int64_t stride;  // elements
  int rows, vocab;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* tokens;
  float* probs;
  int per;  // elements of a slice (a multiple of 8)
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
__device__ __forceinline__ double dbl(F2 a) { return (double)a.h + (double)a.l; }
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
__device__ __forceinline__ float t_of(const Scale& s, float x) { return (s.m - x) * s.c_hi; }

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
  double d[2];
  float f;
  unsigned u[4];
};
struct Shared {
  float2 table[128];
  unsigned hist[kBins];
  Slot slot[2];
  double wsum[kWarps];       // kept mass of each warp's segment
  unsigned wties[kWarps];    // logits equal to tau in it
  double all_sum[kMaxC * kWarps];
  unsigned all_ties[kMaxC * kWarps];
  float red_f[kWarps];
  double red_d[2][kWarps];
  unsigned red_u[4][kWarps];
  unsigned total[kBins];     // the row's histogram
  int pick[4];
};

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void load(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
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
  __device__ static void load(const float* p, float (&v)[4]) {
    const float4 r = *reinterpret_cast<const float4*>(p);
    v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
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

  // ---- the slice: elements [first, first + count) of the row; NaN and the padding as -inf,
  // -0 as +0 (equal logits have equal keys)
  const T* src = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
  const int first = rank * p.per, count = max(0, min(p.per, p.vocab - first));
  const int padded = (count + N * 32 * kWarps - 1) / (N * 32 * kWarps) * (N * 32 * kWarps);
  float best = -INFINITY;
  {
    const bool wide = (reinterpret_cast<uintptr_t>(src + first) & 15) == 0;
    for (int i = t * N; i < padded; i += kThreads * N) {
      float v[N];
      if (wide && i + N <= count) {
        Vec<T>::load(src + first + i, v);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = i + e < count ? Elem<T>::to_f(src[first + i + e]) : -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        v[e] = v[e] == v[e] ? v[e] + 0.f : -INFINITY;
        best = fmaxf(best, v[e]);
        xs[i + e] = Elem<T>::from_f(v[e]);
      }
    }
  }
  // 2^(j / 128) as a pair, from the double function
  if (t < 128) {
    const double w = exp2((double)t / 128.0);
    const float h = (float)w;
    sh.table[t] = make_float2(h, (float)(w - (double)h));
  }
  for (int b = t; b < kBins; b += kThreads) sh.hist[b] = 0;

  // reductions over the row; every thread of every CTA gets the same result
  auto row_max = [&](float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (lane == 0) sh.red_f[warp] = v;
    __syncthreads();
    if (t == 0) {
      float r = sh.red_f[0];
      for (int w = 1; w < kWarps; ++w) r = fmaxf(r, sh.red_f[w]);
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
  auto row_sum2 = [&](F2 a, F2 b, double (&out)[2]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = shfl_add(a, o), b = shfl_add(b, o);
    if (lane == 0) sh.red_d[0][warp] = dbl(a), sh.red_d[1][warp] = dbl(b);
    __syncthreads();
    if (t < 2) {
      double r = 0;
      for (int w = 0; w < kWarps; ++w) r += sh.red_d[t][w];
      sh.slot[phase].d[t] = r;
    }
    sync_row();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      double r = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) r += peer(&sh.slot[phase], c)->d[k];
      out[k] = r;
    }
    phase ^= 1;
  };
  // f(index in the slice, logit) over this thread's elements: warp w has the contiguous segment of
  // `seg` elements from w * seg on, lanes take vectors of it in turn
  const int seg = padded / kWarps;
  auto each = [&](auto&& f) {
    for (int i = warp * seg + lane * N; i < (warp + 1) * seg; i += 32 * N) {
      float v[N];
      Vec<T>::load(xs + i, v);
#pragma unroll
      for (int e = 0; e < N; ++e) f(i + e, v[e]);
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
      each([&](int i, float x) { v[0] = x == m && i < count ? min(v[0], (unsigned)(first + i)) : v[0]; });
    row_u(v, 1, 0);
    if (rank == 0 && t == 0) {
      p.tokens[row] = valid ? (int)v[0] : -1;
      if (p.probs) p.probs[row] = valid ? 1.f : 0.f;
    }
    sync_row();  // no CTA leaves while another reads its shared memory
    return;
  }
  const double c = 1.4426950408889634074 / (double)T_row;
  Scale sc;
  sc.m = m;
  sc.c_hi = (float)c;
  sc.c_lo = isinf(sc.c_hi) ? 0.f : (float)(c - (double)sc.c_hi);
  sc.table = sh.table;
  auto bin_of = [&](float x) {
    const float b = x == m ? 0.f : t_of(sc, x) * kBinScale;
    return b < kBins - 1 ? (int)b : kBins - 1;
  };

  // ---- (tau, n): keys above tau are kept, and the n first of those equal to it
  unsigned tau = key_of(-INFINITY), n_tau = 0;  // -inf itself is never drawn
  const bool use_k = k_row > 0 && k_row < p.vocab, use_p = p_row < 1.f;
  if (use_k || use_p) {
    each([&](int, float x) { if (x > -INFINITY) atomicAdd(&sh.hist[bin_of(x)], 1u); });
    sync_row();
    for (int b = t; b < kBins; b += kThreads) {
      unsigned s = 0;
#pragma unroll
      for (int r = 0; r < C; ++r) s += peer(sh.hist, r)[b];
      sh.total[b] = s;
    }
    if (t < 4) sh.pick[t] = t < 2 ? -1 : kBins - 1;
    __syncthreads();
    // thread t owns bins 4 t .. 4 t + 3, in falling order of the logits
    constexpr int kB = kBins / kThreads;
    unsigned cnt[kB], mine = 0;
#pragma unroll
    for (int b = 0; b < kB; ++b) cnt[b] = sh.total[t * kB + b], mine += cnt[b];
    auto before_u = [&](unsigned v) {  // sum over lower threads
      unsigned inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      if (lane == 31) sh.red_u[0][warp] = inc;
      __syncthreads();
      unsigned b = inc - v;
      for (int w = 0; w < warp; ++w) b += sh.red_u[0][w];
      __syncthreads();
      return b;
    };
    const unsigned cum0 = before_u(mine);
    const unsigned limit = use_k ? (unsigned)k_row : 0xffffffffu;
    if (use_k) {  // top-k's bin: the one in which the count reaches k (if it does)
      unsigned cum = cum0;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        if (cum < limit && cum + cnt[b] >= limit) sh.pick[0] = t * kB + b, sh.pick[1] = (int)cum;
        cum += cnt[b];
      }
    }
    __syncthreads();
    const int bin_k = sh.pick[0];
    const unsigned above_k = (unsigned)sh.pick[1];  // logits in the bins before it
    if (use_k && bin_k >= 0) {  // (fewer than k candidates: all stay)
      // smallest and largest key in the bin, then the largest tau with count(key >= tau) >= k
      unsigned v[2] = {0xffffffffu, 0u};
      each([&](int, float x) {
        if (x > -INFINITY && bin_of(x) == bin_k) v[0] = min(v[0], key_of(x)), v[1] = max(v[1], key_of(x));
      });
      row_u(v, 1, 2);
      unsigned lo = v[0], hi = v[1], above = above_k;
      while (lo < hi) {
        const unsigned mid = lo + (hi - lo + 1) / 2;
        unsigned n[2] = {0, 0};
        each([&](int, float x) { n[0] += bin_of(x) == bin_k && key_of(x) >= mid; });
        row_u(n, 0, 0);
        if (above_k + n[0] >= limit) lo = mid; else hi = mid - 1, above = above_k + n[0];
      }
      n_tau = limit - above;
      tau = lo;
    }
    if (use_p) {
      // mass bounds per bin (2^-((b+1)/51.2) .. 2^-(b/51.2), widened for rounding), cut at k
      float lo_m = 0.f, up_m = 0.f, lo_b[kB], up_b[kB];
      unsigned cum = cum0;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const int bin = t * kB + b;
        const unsigned kept = cum >= limit ? 0u : min(cnt[b], limit - cum);
        cum += cnt[b];
        lo_b[b] = bin == kBins - 1 ? 0.f : kept * exp2f(-(bin + 1.001f) / kBinScale) * 0.999f;
        up_b[b] = kept * exp2f(-(bin - 0.001f) / kBinScale) * 1.001f;
        lo_m += lo_b[b], up_m += up_b[b];
      }
      // running sums over the bins (the bounds are loose enough for fp32 sums: 0.1 % against 2^-13)
      auto before_f = [&](float v, int slot, float* all) {
        float inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        if (lane == 31) sh.red_d[slot][warp] = inc;
        __syncthreads();
        float b = inc - v, a = 0.f;
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) b += (float)sh.red_d[slot][w];
          a += (float)sh.red_d[slot][w];
        }
        *all = a;
        return b;
      };
      float lo_all, up_all;
      float lo_c = before_f(lo_m, 0, &lo_all), up_c = before_f(up_m, 1, &up_all);
      const float p_lo = fmaxf(p_row, 0.f) * lo_all * 0.999f, p_up = fmaxf(p_row, 0.f) * up_all * 1.001f;
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
      const double w_k = tau_k == key_of(-INFINITY) ? 0.0 : dbl(weight(sc, of_key(tau_k)));
      F2 all = {0, 0}, head = {0, 0};
      unsigned v[2] = {0xffffffffu, 0u};
      each([&](int, float x) {
        const unsigned key = key_of(x);
        if (key < tau_k || (key == tau_k && n_k == 0)) return;
        const int b = bin_of(x);
        if (b >= b0 && b <= b1 && x > -INFINITY) v[0] = min(v[0], key), v[1] = max(v[1], key);
        if (key > tau_k) {
          const F2 w = weight(sc, x);
          all = add(all, w);
          if (b < b0) head = add(head, w);
        }
      });
      double sums[2];
      row_sum2(all, head, sums);
      row_u(v, 1, 2);
      const bool tie_in = n_k > 0;
      const double mass = sums[0] + (tie_in ? n_k * w_k : 0.0);
      const int bin_tau = tie_in ? bin_of(of_key(tau_k)) : kBins;
      const double base = sums[1] + (tie_in && bin_tau < b0 ? n_k * w_k : 0.0);
      const double goal = (double)fmaxf(p_row, 0.f) * mass;
      unsigned lo = v[0], hi = v[1];
      if (lo <= hi) {
        double above = base;  // mass of the keys above hi
        while (lo < hi) {
          const unsigned mid = lo + (hi - lo + 1) / 2;
          F2 s = {0, 0};
          each([&](int, float x) {
            const unsigned key = key_of(x);
            if (key < mid || key <= tau_k) return;
            const int b = bin_of(x);
            if (b >= b0 && b <= b1) s = add(s, weight(sc, x));
          });
          double r[2];
          row_sum2(s, F2{0, 0}, r);
          const double f = base + r[0] + (tie_in && tau_k >= mid && bin_tau >= b0 ? n_k * w_k : 0.0);
          if (f >= goal) lo = mid; else hi = mid - 1, above = f;
        }
        // of the keys equal to tau: those before which less than the goal lies
        const double w = dbl(weight(sc, of_key(lo)));
        const double more = w > 0 ? ceil((goal - above) / w) : 1.0;
        const unsigned n_p = more < 1.0 ? (goal <= 0 && lo == key_of(m) ? 1u : 0u) : more > 4e9 ? 0xffffffffu : (unsigned)more;
        n_tau = lo == tau_k && tie_in ? min(n_k, n_p) : n_p;
        tau = lo;
      }
    }
  }

  // ---- ties at tau before each warp's segment
  const bool ties = use_k || use_p;
  unsigned my_ties = 0;
  if (ties) {
    each([&](int i, float x) { my_ties += key_of(x) == tau && i < count; });
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
  const double lo_p = (double)lo_row;
  auto kept = [&](auto&& f) {
    unsigned rank0 = ties_before;
    const bool some = ties && ties_before < n_tau && ties_before + my_ties > n_tau;  // the n-th tie is here
    const bool whole = ties && ties_before + my_ties <= n_tau;
    for (int i0 = warp * seg; i0 < (warp + 1) * seg; i0 += 32 * N) {
      float v[N];
      Vec<T>::load(xs + i0 + lane * N, v);
      unsigned eq = 0, at = 0;
      if (some) {
#pragma unroll
        for (int e = 0; e < N; ++e) eq += key_of(v[e]) == tau && i0 + lane * N + e < count;
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
          if (dbl(w[e]) < lo_p) w[e] = F2{0.f, 0.f};
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
  if (lane == 0) sh.wsum[warp] = dbl(sum);
  sync_row();
  if (t < C * kWarps) sh.all_sum[t] = peer(sh.wsum, t / kWarps)[t % kWarps];
  __syncthreads();
  double total = 0;
  for (int w = 0; w < C * kWarps; ++w) total += sh.all_sum[w];
  const double target = (double)u_row * total;
  // the first segment whose running sum exceeds the target (else the last with any mass)
  int owner = -1;
  double before = 0, run = 0;
  for (int w = 0; w < C * kWarps; ++w) {
    const double s = sh.all_sum[w];
    if (s > 0) {
      owner = w, before = run;
      run += s;
      if (run > target) break;
    }
  }
  if (owner < 0 && rank == 0 && t == 0) {  // min-p above 1: nothing is left
    p.tokens[row] = -1;
    if (p.probs) p.probs[row] = 0.f;
  }
  if (owner == rank * kWarps + warp) {
    int token = -1;  // so far: the last kept index seen
    double wt = 0;
    kept([&](int i0, F2 (&w)[N]) {
      double mine = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) mine += dbl(w[e]);
      double inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      const double end = before + __shfl_sync(0xffffffffu, inc, 31);
      // this lane's first index past the target, else its last kept one
      double cum = before + (inc - mine), my_w = 0;
      int my = -1;
      bool hit = false;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const double we = dbl(w[e]);
        cum += we;
        if (we > 0 && !hit) {
          my = i0 + lane * N + e;
          my_w = we;
          hit = cum > target;
        }
      }
      const unsigned hits = __ballot_sync(0xffffffffu, hit), any = __ballot_sync(0xffffffffu, my >= 0);
      if (any) {
        const int from = hits ? __ffs(hits) - 1 : 31 - __clz(any);
        token = __shfl_sync(0xffffffffu, my, from);
        wt = __shfl_sync(0xffffffffu, my_w, from);
      }
      before = end;
      return hits == 0;
    });
    if (lane == 0) {
      p.tokens[row] = token >= 0 ? first + token : -1;
      if (p.probs) p.probs[row] = token >= 0 ? (float)(wt / total) : 0.f;
    }
  }
  sync_row();  // no CTA leaves while another reads its shared memory
}

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
  if (vocab > (dtype == DFLASH_F32 ? 400000 : 800000))
    return call_error(DFLASH_EUNSUPPORTED, "sample: vocab above 400000 (fp32) or 800000 (bf16)");
  if (rows > (1 << 28) - 1) return call_error(DFLASH_ECAPACITY, "sample: too many rows for one call");
  if (rows == 0) return DFLASH_OK;
  if (!logits || !u || !tokens) return call_error(DFLASH_EINVAL, "sample: null pointer");
  SampleParams p{logits, row_stride, rows, vocab, u, temperature, top_p, min_p, top_k, tokens, probs, 0};
  p.per = (vocab + kMaxC - 1) / kMaxC;
  p.per = (p.per + 7) / 8 * 8;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DFLASH_F32 ? launch<float, kMaxC>(p, st) : launch<__nv_bfloat16, kMaxC>(p, st);
  if (e != cudaSuccess) return call_error(DFLASH_ECUDA, "sample", e);
  return DFLASH_OK;
}
