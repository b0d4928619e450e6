// One token per row of logits by temperature, top-k, top-p and min-p (dflash_sample).
//
// In falling order of the logits every filter keeps a prefix, and the prefix is short in most
// rows: so the row is read once, and only the logits near its maximum are held.  A CTA (a cluster
// of up to 8, when rows are few) streams a row through a ring in shared memory:
//   - a look at the first blocks sets a floor; logits from it on go to a list, and top-p alone also
//     sums the mass of the others.  A histogram of the list (counts, masses) over
//     t = (m - x) log2(e) / T, m the largest logit, says how far the prefix reaches; that part,
//     usually a few dozen logits, is sorted, and its weights' running sums give the kept prefix and
//     the token.
//   - rows without a short prefix by right (temperature alone) sum every warp's stretches of the
//     row in index order, rescaled as m grows; the stretch that holds u * total is read again.
//     Vectors whose logits are all far below m (t > 12) go in fp32, with a bound on their error:
//     where the token could depend on it, or the probability's last bit (flat rows; a few in a
//     thousand others), the row is streamed once more with exact weights.
//   - rows whose prefix is longer than the list are streamed again (from L2, mostly): histograms
//     over the logits' order-preserving keys, 9 bits a pass, with exact counts (top-k) and masses
//     (top-p), find (tau, n): the lowest kept logit, and how many of those equal to it stay; then
//     stretches of the kept weights are summed as above.
// Bound by HBM: one read of the logits (the finishing phases of some CTAs overlap the streaming of
// others; three CTAs per SM with 32 KB of copies in flight each).  Measured, rows of 151936 bf16: 1024
// rows greedy 54 us (5.8 TB/s), min-p 84, top-k 50 95, top-p 0.95 133, temperature alone 229, of
// mixed settings 126 (205 where a row is streamed again: one call in four); flat ones (top-p 0.99 at
// temperature 1.2: prefixes of many thousands) 2.06 ms; one row 23 us, of which most is latency.
//
// The token is a whole number that a sum's last bit can change, so weights are pairs of floats
// (exp2 by a 128-entry table and a short polynomial on the compensated argument, about 2^-41)
// and masses are compensated or whole numbers: in plain fp32 one row in a few hundred would
// differ.  The mass past the list's range enters top-p's total with fp32 weights, and a bound on
// their error: where a border of the prefix lies within it (one row in a thousand), the row is
// streamed once more with exact ones.
#include <cooperative_groups.h>
#include <float.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "launch_util.cuh"
#include "serve.cuh"
#include "tc_common.cuh"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

constexpr float kCut = 40.f;                 // weights below 2^-40 are 0

struct SampleParams {
  const void* logits;
  int64_t stride;  // elements
  int rows, vocab;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* tokens;
  float* probs;
  int ctas, per;  // CTAs of a row; positions of a CTA's slice (a multiple of 8)
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
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  const float p = a.h * b.h, e = fmaf(a.h, b.h, -p) + fmaf(a.h, b.l, a.l * b.h);
  const float h = p + e;
  return {h, e - (h - p)};
}
__device__ __forceinline__ bool below(F2 a, float b) { return a.h < b || (a.h == b && a.l < 0.f); }
// Masses as whole numbers of 2^-B: sums and comparisons are exact and cost integer operations
// (fp64 runs at 1/64 of the fp32 rate here).  Equal logits round alike, so what a weight loses by
// its rounding adds up over a row: B is chosen so that a row of 2^20 loses less than 1e-11 of its
// mass (at least 1).  52 where at most 2048 weights are added in 64 bits (a sorted prefix, a stretch:
// one rounding per lane of it), 59 where a row's are added one by one (keys); sums over a row then
// have 128 bits.  43, in 64 bits over a row, is for masses rounded once per warp and for bounds.
typedef unsigned __int128 u128;
constexpr int kStretchUnit = 52, kKeyUnit = 59;
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
__device__ __forceinline__ u128 part_of(u128 a, float f, bool* inexact = nullptr) {  // a below 2^104
  if (inexact) *inexact = false;
  if (!(f > 0.f)) return 0;
  if (f >= 1.f) return a;
  int e;
  const u128 x = a * (unsigned long long)ldexpf(frexpf(f, &e), 24);  // f = m 2^(e - 24), e <= 0
  const int sh = 24 - e;
  const u128 r = sh < 128 ? x >> sh : 0;
  if (inexact) *inexact = sh < 128 ? r << sh != x : x != 0;
  return r;
}
__device__ __forceinline__ double to_double(u128 a) {
  return (double)(unsigned long long)(a >> 64) * 0x1p64 + (double)(unsigned long long)a;
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

// 16 bytes of logits: their largest and smallest (NaN counts as nothing), and the values.
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
  __device__ static float low(const uint4& r) {
    const __nv_bfloat162 a = __hmin2(reinterpret_cast<const __nv_bfloat162&>(r.x), reinterpret_cast<const __nv_bfloat162&>(r.y));
    const __nv_bfloat162 b = __hmin2(reinterpret_cast<const __nv_bfloat162&>(r.z), reinterpret_cast<const __nv_bfloat162&>(r.w));
    const __nv_bfloat162 m = __hmin2(a, b);
    return fminf(__low2float(m), __high2float(m));
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
  __device__ static float low(const uint4& r) {
    return fminf(fminf(__uint_as_float(r.x), __uint_as_float(r.y)), fminf(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
  __device__ static void get(const uint4& r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
  }
};


__device__ __forceinline__ Scale scale_of(float m, float T, const float2* table) {
  // log2(e) / T: the quotient, and the exact remainder's quotient
  constexpr float kE = 1.44269502162933349609375f, kEl = 1.92596299e-8f;  // log2(e)
  Scale s;
  s.m = m;
  s.c_hi = kE / T;
  s.c_lo = isinf(s.c_hi) ? 0.f : (fmaf(-s.c_hi, T, kE) + kEl) / T;
  s.table = table;
  return s;
}
// a logit from which on t can be below r (rounding allowed for)
__device__ __forceinline__ float reach(const Scale& s, float r) {
  return isinf(s.c_hi) || isinf(s.m) ? s.m : s.m - r / s.c_hi * 1.00001f - fabsf(s.m) * 1e-6f;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 in one register pair, and the packed operations on them (sm_100 and on)
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.f : -INFINITY; }  // NaN: -inf, -0: +0

struct Row {  // a row's settings
  float T, p, lo, u;
  int k;
  bool use_k, use_p;
};
__device__ __forceinline__ Row row_of(const SampleParams& q, int row) {
  Row r;
  r.T = q.temperature ? q.temperature[row] : 1.f;
  r.k = q.top_k ? q.top_k[row] : 0;
  r.p = q.top_p ? q.top_p[row] : 1.f;
  r.lo = q.min_p ? q.min_p[row] : 0.f;
  const float u = q.u[row];
  r.u = u > 0.f ? u : 0.f;
  r.use_k = r.k > 0 && r.k < q.vocab;
  r.use_p = r.p < 1.f;
  r.p = fmaxf(r.p, 0.f);
  return r;
}

// A CTA's part of a row.  Positions count from the 16-byte boundary at or before the row's first
// logit, so that vectors are aligned whatever the row's address; position i of the slice is logit
// first + i, and those outside [begin, count) hold -inf.
template <typename T>
struct Slice {
  const T* src;
  int first, begin, count;
  __device__ Slice(const SampleParams& q, int row, int rank) {
    src = static_cast<const T*>(q.logits) + (int64_t)row * q.stride;
    const int skip = (int)(reinterpret_cast<uintptr_t>(src) & 15) / (int)sizeof(T);
    first = rank * q.per - skip;
    begin = max(0, -first);
    count = max(0, min(q.per, q.vocab - first));
  }
  __device__ bool whole(int i) const { return i >= begin && i + Vec<T>::N <= count; }
  __device__ const T* at(int i) const { return src + (first + i); }
  __device__ uint4 vector(int i) const { return whole(i) ? *reinterpret_cast<const uint4*>(at(i)) : edge(i); }
  __device__ uint4 edge(int i) const {  // a vector at the row's ends
    uint4 r = make_uint4(Vec<T>::kPad, Vec<T>::kPad, Vec<T>::kPad, Vec<T>::kPad);
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e)
      if (i + e >= begin && i + e < count) reinterpret_cast<T*>(&r)[e] = src[first + i + e];
    return r;
  }
};

__device__ __forceinline__ float prob_of(F2 w, u128 total) {  // total in units of 2^-52
  static_assert(kStretchUnit == 52, "the unit");
  return (float)(((double)w.h + (double)w.l) / (to_double(total) * 0x1p-52));
}
__device__ __forceinline__ void put(const SampleParams& q, int row, int token, float prob) {
  q.tokens[row] = token;
  if (q.probs) q.probs[row] = prob;
}

// Keys that differ by one for neighbouring values of the type
template <typename T>
__device__ __forceinline__ unsigned digit_key(float x) {
  return sizeof(T) == 2 ? key_of(x) >> 16 : key_of(x);
}
template <typename T>
__device__ __forceinline__ float of_digit_key(unsigned k) {
  if (sizeof(T) == 2) return __uint_as_float((k & 0x8000u ? k ^ 0x8000u : ~k & 0xffffu) << 16);
  return of_key(k);
}

constexpr int kST = 256, kSW = kST / 32;     // threads, warps
constexpr int kStages = 3, kVec = 4;         // ring: blocks in flight; vectors of a thread in a block
constexpr int kStageBytes = kST * kVec * 16; // 16 KB
constexpr int kMaxC = 8;                     // CTAs of a row
constexpr int kList = 4096;                  // places that a list holds
constexpr int kAim = 3000;                   // and that the floor may aim at
constexpr int kSorted = 2048;                // logits of the sorted prefix
constexpr int kBins = 256;                   // histogram of the list
constexpr int kLook = 64;                    // bins of the look at the first blocks,
constexpr float kLookFar = 32.f;             // and their range of t below the maximum found there
// Histograms over keys: bins of a round, and the words of a bin's mass, 12 bits of every weight each
// (2^20 of them fit).  9 bits a round: two rounds for bf16's keys and four for fp32's, as by 10.
constexpr int kDigit = 9, kKeys = 1 << kDigit, kParts = 5, kPartBits = 12;
// Far masses in fp32: a bound on their relative error up to t = 20 (x - m rounded: t 2^-24 ln 2 <
// 8.3e-7; ex2 2^-22; the correction's and the tree's roundings 5 2^-24); what a logit further off can
// add to it, in units of 2^-20 ((t - 20) 2^(20 - t) is at most 1 / (e ln 2): 0.531 2^-24 ln 2); and
// the error a probability may carry
constexpr float kNear = 12.f;
constexpr float kFastError = 1.4e-6f, kFastTail = 2.2e-8f, kProbError = 8e-8f;
// Beside that bound: a far mass is taken against the largest logit met until then, so it may hold weights
// that the row's maximum puts below 2^-40, where they count as 0: up to 2^-40 each.  (The probability's
// last bit is not held to that: a row of a thousand such weights is 1e-9 off.)
// The bound for a mass in units of 2^-43, of a row of `vocab` logits
__device__ __forceinline__ unsigned long long far_error(unsigned long long far, int vocab) {
  return part_of(far, kFastError) + part_of((unsigned long long)vocab << 23, kFastTail);
}
// Shared memory beside the ring, in turn: the list's places; a list's sorted prefix; the
// stretches; the digits' histograms (the stretches are not needed yet)
constexpr int kSideBytes = 16384;
static_assert(kList * 4 == kSideBytes && kSorted * 8 == kSideBytes && kKeys * kParts * 4 <= kSideBytes, "one size");
static_assert(kKeyUnit < kParts * kPartBits, "a weight of 1 has its bits");
static_assert(kList * 8 + kSorted * 8 <= kStages * kStageBytes, "the row's list, and places by index, fit in the ring");
constexpr int kStreamSmem = kStages * kStageBytes + kSideBytes;

struct Stretch {  // mass of a warp's part of a block (2^-52: 1024 weights at most), relative to ref
  unsigned long long mass;
  unsigned ties;  // logits equal to tau ahead of it; of fp32 sums: the key of the smallest logit summed
  float ref;
};

struct Shared {
  float2 table[128];
  unsigned count[kBins];
  unsigned long long mass[kBins];
  unsigned long long red_l[kSW], rest, best, before, far, far_part;
  u128 part, above;
  unsigned red_u[kSW], ties;
  unsigned m_key, n_list, n_final, full, again, cut;
  float m_look;
  float floor, floors[kSW];
  int pick[2];
};

template <typename T>
__global__ void __launch_bounds__(kST, 3) sample_kernel(const SampleParams q) {
  constexpr int N = Vec<T>::N, kBlock = kST * kVec * N, kWarpPart = kVec * 32 * N;
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* ring = reinterpret_cast<uint4*>(smem);
  uint8_t* side = smem + kStages * kStageBytes;
  unsigned* places = reinterpret_cast<unsigned*>(side);                        // the list: vocabulary indices
  unsigned long long* list = reinterpret_cast<unsigned long long*>(side);      // the sorted prefix
  Stretch* stretch = reinterpret_cast<Stretch*>(side);
  unsigned* digits = reinterpret_cast<unsigned*>(side);                        // counts, or masses in four parts
  // once the row is through, the ring holds: the row's list as (~key, index), and places by index
  unsigned long long* final_list = reinterpret_cast<unsigned long long*>(smem);
  unsigned* index = reinterpret_cast<unsigned*>(smem + kList * 8);
  unsigned* by = index + kSorted;
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int C = q.ctas, rank = C > 1 ? (int)cl.block_rank() : 0, row = blockIdx.x / C;
  auto sync_row = [&] {
    if (C > 1) cl.sync(); else __syncthreads();
  };
  auto peer = [&](auto* ptr, int r) { return C > 1 ? cl.map_shared_rank(ptr, r) : ptr; };

  const Slice<T> sl(q, row, rank);
  const int blocks = (sl.count + kBlock - 1) / kBlock;
  // behind the stretches: vectors near the maximum
  unsigned* near_places = reinterpret_cast<unsigned*>(stretch + blocks * kSW);
  const unsigned near_room = kSideBytes / 4 - blocks * kSW * 4;
  auto pos_of = [&](int b, int v) { return b * kBlock + warp * kWarpPart + (v * 32 + lane) * N; };
  // a thread copies and reads back its own vectors, so the ring needs no barrier
  auto issue = [&](int b) {
    uint4* d = ring + b % kStages * (kVec * kST) + t;
    if (b * kBlock >= sl.begin && (b + 1) * kBlock <= sl.count) {
      const T* src = sl.at(pos_of(b, 0));
#pragma unroll
      for (int v = 0; v < kVec; ++v) tc::cp_async16(d + v * kST, src + v * 32 * N);
    } else if (b < blocks) {  // with the row's ends
      for (int v = 0; v < kVec; ++v) {
        const int i = pos_of(b, v);
        if (sl.whole(i)) tc::cp_async16(d + v * kST, sl.at(i)); else d[v * kST] = sl.edge(i);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // f(block, its vectors, their largest logits) over the slice; the first blocks are on their way
  auto stream = [&](auto&& f) {
#pragma unroll 1
    for (int b = 0; b < blocks; ++b) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      uint4 x4[kVec];
      float tops[kVec];
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        x4[v] = ring[(b % kStages * kVec + v) * kST + t];
        tops[v] = Vec<T>::top(x4[v]);
      }
      f(b, x4, tops, [&] { issue(b + kStages); });
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  };
  auto start = [&] {
    for (int b = 0; b < kStages; ++b) issue(b);
  };
  start();
  const Row r = row_of(q, row);
  if (t < 128) sh.table[t] = q.table[t];
  if (t < kBins) sh.count[t] = 0, sh.mass[t] = 0;
  if (t == 0) {
    sh.m_key = 0;
    sh.n_list = sh.n_final = sh.full = sh.again = sh.cut = 0;
    sh.rest = sh.best = sh.far = 0;
    sh.pick[0] = 0x7fffffff;
    sh.pick[1] = -1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (!(r.T >= 0.f && r.T <= FLT_MAX)) {  // the same in every CTA of the row
    if (rank == 0 && t == 0) put(q, row, -1, 0.f);
    return;
  }
  __syncthreads();
  // ---- the first blocks' maximum
  const int seen = min(blocks, kStages);
  float top = -INFINITY;
  for (int b = 0; b < seen; ++b) {
#pragma unroll
    for (int v = 0; v < kVec; ++v) top = fmaxf(top, Vec<T>::top(ring[(b * kVec + v) * kST + t]));
  }
  {
    const unsigned k = __reduce_max_sync(0xffffffffu, key_of(top + 0.f));
    if (lane == 0) atomicMax(&sh.m_key, k);
  }
  sync_row();
  float m = of_key(sh.m_key);  // this warp's maximum so far
  for (int c = 0; c < C; ++c) m = fmaxf(m, of_key(*peer(&sh.m_key, c)));
  if (t == 0) sh.m_look = m;
  Scale sc = scale_of(m, r.T, sh.table);  // (T == 0: not used)
  // rows by list: a short prefix by right
  const bool greedy = r.T == 0.f;
  const bool by_list = !greedy && (r.use_k || r.use_p || r.lo > 0.f);
  const bool sum = by_list && r.use_p && !r.use_k;
  // 2^-t of N logits, in fp32 (NaN and -inf fail the comparison with the cut; m is finite): t with
  // its low part
  auto fast_of = [&](const float (&x)[N]) {
    const uint64_t nm = pair(-m, -m), c = pair(sc.c_hi, sc.c_hi), nc = pair(-sc.c_hi, -sc.c_hi), cl2 = pair(sc.c_lo, sc.c_lo);
    const uint64_t ln2 = pair(0.693147182f, 0.693147182f);
    uint64_t s = 0;
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const uint64_t d = add2(pair(x[e], x[e + 1]), nm);
      const uint64_t tt = mul2(d, nc), lo = fma2(d, cl2, fma2(d, c, tt));
      float t0, t1, w0, w1;
      unpair(tt, t0, t1);
      const uint64_t w = pair(ex2(-t0), ex2(-t1));
      unpair(fma2(w, mul2(lo, ln2), w), w0, w1);
      s = add2(s, pair(t0 <= kCut ? w0 : 0.f, t1 <= kCut ? w1 : 0.f));
    }
    float s0, s1;
    unpair(s, s0, s1);
    return s0 + s1;
  };
  auto fast = [&](const uint4& v4) {
    float x[N];
    Vec<T>::get(v4, x);
    return fast_of(x);
  };
  float floor_x = -INFINITY;  // the list takes logits from here on
  // The share of the row seen.  The last slice may have a block less than the others, and what the
  // CTAs decide by it (which floor, hence which cluster barriers) has to be the same in all of them:
  // it is counted over every slice, not over this CTA's.
  int row_blocks = 0, row_seen = 0;
  for (int c = 0; c < C; ++c) {
    const int n = (max(0, min(q.per, q.vocab - (sl.first + (c - rank) * q.per))) + kBlock - 1) / kBlock;
    row_blocks += n, row_seen += min(n, kStages);
  }
  const float share = (float)row_seen / (float)max(row_blocks, 1);
  // A floor by rank: of the threads' largest logits in the blocks seen, the r-th is about the row's
  // r / share-th (a thread seldom has two of them).  false: the list wants more than that tells
  auto floor_by_rank = [&]() -> bool {
    if (!r.use_k && !r.use_p) {  // min-p: every t up to its own (below the row's m, not this one's: more)
      floor_x = isinf(m) || isinf(sc.c_hi) ? m : m - (fmaxf(0.f, -log2f(r.lo)) + 0.5f) / sc.c_hi;
      return true;
    }
    const float want = r.use_k ? 1.5f * r.k + 64.f : 320.f;
    const int at = max(1, (int)ceilf(want * share / (C * kSW)));  // per warp
    if (at > 16) return false;
    // each warp's at-th largest; their mean
    const unsigned mine = key_of(top + 0.f);
    int ahead = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const unsigned x = __shfl_sync(0xffffffffu, mine, i);
      ahead += x > mine || (x == mine && i < lane);
    }
    if (ahead == at - 1) sh.floors[warp] = top;
    sync_row();
    float mean = 0.f;
    for (int c = 0; c < C; ++c)
      for (int w = 0; w < kSW; ++w) mean += peer(sh.floors, c)[w];
    floor_x = mean / (C * kSW);
    if (!(floor_x < INFINITY)) floor_x = m;  // infinities among them
    return true;
  };
  // A floor by a histogram of t in the blocks seen
  auto floor_by_look = [&] {
    const float step = kLookFar / kLook;
    const float from = reach(sc, kLookFar);
    for (int b = 0; b < seen; ++b) {
#pragma unroll 1
      for (int v = 0; v < kVec; ++v) {
        const uint4 x4 = ring[(b * kVec + v) * kST + t];
        if (!(Vec<T>::top(x4) >= from)) continue;
        float x[N];
        Vec<T>::get(x4, x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float tt = t_of(sc, clean(x[e]));
          if (tt < kLookFar && x[e] > -INFINITY) atomicAdd(&sh.count[(int)(tt * (kLook / kLookFar))], 1u);
        }
      }
    }
    sync_row();
    if (rank == 0 && warp == 0) {
      // lane l: bins 2 l, 2 l + 1 of the row's first blocks.  The first bins by which, going by them,
      // the list holds what the filter needs: k and half as many more; all but 1 - p of the mass
      // (the mass left out, as the blocks seen have it, against that seen alone: the few large
      // weights of a row may lie anywhere) and some 192 logits
      unsigned a = 0, b = 0;
      for (int c = 0; c < C; ++c) a += peer(sh.count, c)[2 * lane], b += peer(sh.count, c)[2 * lane + 1];
      unsigned n = a + b;
      float w = a * exp2f(-(2 * lane + 0.5f) * step) + b * exp2f(-(2 * lane + 1.5f) * step);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, n, o);
        const float y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) n += x, w += y;
      }
      const float whole = __shfl_sync(0xffffffffu, w, 31);
      const bool enough = r.use_k ? n >= (1.5f * r.k + 64.f) * share
                                  : !r.use_p || ((whole - w) * 1.3f <= (1.f - r.p) * whole * share && n >= 192.f * share);
      const unsigned yes = __ballot_sync(0xffffffffu, enough), fits = __ballot_sync(0xffffffffu, n <= kAim * share);
      const int pairs = min(yes ? __ffs(yes) : 32, max(1, ~fits ? __ffs(~fits) - 1 : 32));
      if (lane == 0) sh.floor = isinf(m) || isinf(sc.c_hi) ? m : m - pairs * 2 * step / sc.c_hi;
    }
    sync_row();  // (the counts have been read by every CTA)
    floor_x = *peer(&sh.floor, 0);  // one floor: from_list takes it for every slice's
    if (t < kLook) sh.count[t] = 0;
    __syncthreads();
  };

  // ---- the row
  F2 rest = {0.f, 0.f};                              // mass below the floor, relative to m
  bool exact_rest = false;                           // of exact weights
  auto slow = [&](const uint4& v4, float below_x) {  // exact mass of the logits below
    float x[N];
    Vec<T>::get(v4, x);
    F2 s = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (x[e] < below_x && x[e] > -INFINITY) s = add(s, weight(sc, clean(x[e])));
    return s;
  };
  unsigned long long best = 0;                       // greedy: (key, ~index)
  bool finite;                                       // m and log2(e) / T are: fp32 masses make sense
  float cut_x, near_x;                               // vectors below weigh nothing; are far
  auto bounds = [&] {
    finite = m > -INFINITY && m < INFINITY && !isinf(sc.c_hi);
    cut_x = reach(sc, kCut);
    near_x = finite ? reach(sc, kNear) : cut_x;
  };
  auto first_pass = [&](int b, uint4 (&x4)[kVec], float (&tops)[kVec], auto&& next) {
    float top = -INFINITY;  // (a vector of NaN alone has a NaN for its largest, and NaN's key is above every number's)
#pragma unroll
    for (int v = 0; v < kVec; ++v) top = fmaxf(top, tops[v]);
    const unsigned w_key = __reduce_max_sync(0xffffffffu, key_of(top + 0.f));
    const unsigned s_key = *(volatile unsigned*)&sh.m_key;
    if (lane == 0 && w_key > s_key) atomicMax(&sh.m_key, w_key);
    next();
    const float m_new = of_key(max(w_key, __shfl_sync(0xffffffffu, s_key, 0)));
    if (m_new > m) {
      sc.m = m_new;
      if (rest.h > 0.f) rest = mul(rest, weight(sc, m));
      m = m_new;
      bounds();
    }
    if (greedy) {
      if (!(top >= m)) return;
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        if (!(tops[v] >= m)) continue;
        float x[N];
        Vec<T>::get(x4[v], x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const unsigned long long c = (unsigned long long)key_of(clean(x[e])) << 32 | ~(unsigned)(sl.first + pos_of(b, v) + e);
          if (clean(x[e]) > -INFINITY && c > best) best = c;
        }
      }
      return;
    }
    if (by_list) {
      if (!(top >= (sum ? fminf(floor_x, cut_x) : floor_x))) return;
      if (exact_rest) {
#pragma unroll 1
        for (int v = 0; v < kVec; ++v) {
          const uint4 y4 = v == 0 ? x4[0] : v == 1 ? x4[1] : v == 2 ? x4[2] : x4[3];
          const float y = Vec<T>::top(y4);
          if (y >= floor_x) {
            const unsigned at = atomicAdd(&sh.n_list, 1u);
            if (at < kList) places[at] = pos_of(b, v);
          } else if (finite && y >= cut_x) {
            rest = add(rest, slow(y4, floor_x));
          }
        }
        return;
      }
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        if (tops[v] >= floor_x) {  // its logits are looked at when the row is through, by all lanes
          const unsigned at = atomicAdd(&sh.n_list, 1u);
          if (at < kList) places[at] = pos_of(b, v);
        } else if (sum && finite && tops[v] >= cut_x) {
          rest = add(rest, F2{fast(x4[v]), 0.f});
        }
      }
      return;
    }
    float far = 0.f, low = INFINITY;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      if (!(tops[v] >= cut_x)) continue;
      if (tops[v] >= near_x) {  // exactly, when the row is through
        const unsigned at = atomicAdd(&sh.n_list, 1u);
        if (at < near_room) near_places[at] = pos_of(b, v);
      } else {
        far += fast(x4[v]);
        low = fminf(low, Vec<T>::low(x4[v]));
      }
    }
    unsigned long long mass = fix<kStretchUnit>(F2{far, 0.f});
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
    const unsigned low_key = __reduce_min_sync(0xffffffffu, key_of(low));
    if (lane == 0) stretch[b * kSW + warp] = Stretch{mass, low_key, m};
  };
  bool looked = false;  // the floor is a look's
  if (by_list && !floor_by_rank()) looked = true, floor_by_look();
  __syncthreads();      // (the list takes the place of what the floor was found with)
  bounds();
  stream(first_pass);
  if (greedy) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane == 0) atomicMax(&sh.best, best);
    sync_row();
    if (rank == 0 && t == 0) {
      for (int c = 0; c < C; ++c) best = max(best, *peer(&sh.best, c));
      put(q, row, best ? (int)~(unsigned)best : -1, best ? 1.f : 0.f);
    }
    if (C > 1) cl.sync();  // no CTA leaves while another reads its shared memory
    return;
  }

  // ---- the row's maximum
  sync_row();
  float m_row = of_key(sh.m_key);
  for (int c = 0; c < C; ++c) m_row = fmaxf(m_row, of_key(*peer(&sh.m_key, c)));
  sc.m = m_row;
  if (!(m_row > -INFINITY)) {
    if (rank == 0 && t == 0) put(q, row, -1, 0.f);
    if (C > 1) cl.sync();
    return;
  }
  auto scan_l = [&](unsigned long long v, unsigned long long* all) {  // sum over lower threads of the CTA
    unsigned long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) sh.red_l[warp] = inc;
    __syncthreads();
    unsigned long long b = inc - v, a = 0;
    for (int w = 0; w < kSW; ++w) {
      if (w < warp) b += sh.red_l[w];
      a += sh.red_l[w];
    }
    __syncthreads();
    *all = a;
    return b;
  };
  auto scan_w = [&](u128 v, u128* all) {  // the same in 128 bits (256 values: each half's sum fits in 64)
    constexpr int kHalf = 52;
    unsigned long long a_lo, a_hi;
    const unsigned long long lo = scan_l((unsigned long long)v & ((1ull << kHalf) - 1), &a_lo);
    const unsigned long long hi = scan_l((unsigned long long)(v >> kHalf), &a_hi);
    *all = ((u128)a_hi << kHalf) + a_lo;
    return ((u128)hi << kHalf) + lo;
  };

  // ---- the token from the row's list, in the first CTA
  enum { kDone, kPast, kUnsure };  // kPast: the prefix is not in it; kUnsure: a border within the total's error
  auto from_list = [&]() -> int {
    const int n_all = (int)sh.n_final;
    if (sh.full || sh.rest >= 1ull << 54) return kPast;  // too many, or a mass above 2048 largest weights
    const float scale = kBins / fmaxf(t_of(sc, floor_x), 1e-30f);
    auto bin_of = [&](float tt) { return min(kBins - 1, (int)fminf(tt * scale, kBins)); };
    for (int i = t; i < n_all; i += kST) {
      const float x = of_key(~(unsigned)(final_list[i] >> 32));
      const int b = bin_of(t_of(sc, x));
      atomicAdd(&sh.count[b], 1u);
      if (r.use_p) atomicAdd(&sh.mass[b], fix<51>(weight(sc, x)));  // (4096 of them, and the rest, below 2^64)
    }
    __syncthreads();
    // thread t: bin t.  The last bin that the prefix reaches
    unsigned long long all, goal = ~0ull;
    const unsigned cum = (unsigned)scan_l(sh.count[t], &all) + sh.count[t];
    unsigned long long whole = 0, run_m = 0;
    if (r.use_p) run_m = scan_l(sh.mass[t], &whole) + sh.mass[t];
    whole += sh.rest << 8;
    bool goal_set = sum;
    if (r.use_k && r.use_p) {
      // the mass left by top-k: the bins before the one in which the count reaches k, and the largest
      // of that one
      if (cum >= (unsigned)r.k && cum - sh.count[t] < (unsigned)r.k) {
        sh.pick[1] = t;
        sh.red_u[1] = cum - sh.count[t];
        sh.before = run_m - sh.mass[t];
      }
      if (t == 0) sh.n_list = 0;
      __syncthreads();
      const int bin_k = sh.pick[1];
      if (bin_k < 0) return kPast;
      const unsigned in_bin = sh.count[bin_k];
      if (in_bin <= kST) {
        for (int i = t; i < n_all; i += kST) {
          const unsigned long long it = final_list[i];
          if (bin_of(t_of(sc, of_key(~(unsigned)(it >> 32)))) == bin_k) list[atomicAdd(&sh.n_list, 1u)] = it;
        }
        __syncthreads();
        unsigned long long w = 0;
        if (t < in_bin) {
          const unsigned long long it = list[t];
          unsigned ahead = sh.red_u[1];
          for (unsigned j = 0; j < in_bin; ++j) ahead += list[j] < it;
          if (ahead < (unsigned)r.k) w = fix<51>(weight(sc, of_key(~(unsigned)(it >> 32))));
        }
        scan_l(w, &all);
        whole = sh.before + all;
        goal_set = true;
      }
      __syncthreads();
      if (t == 0) sh.pick[1] = -1;
    }
    bool here;
    if (goal_set) {
      bool more;
      goal = part_of(whole, r.p, &more);
      goal = max(goal + more, 1ull);  // the first always stays
      here = run_m >= goal;
      goal = goal >> 63 ? ~0ull : goal << 1;  // in the sorted prefix's units
    } else if (r.use_k) {
      here = cum >= (unsigned)r.k;
    } else {  // min-p: t <= -log2(min_p), allowing for rounding
      const float far = fmaxf(0.f, -log2f(r.lo)) + 0.01f;
      here = (t + 1) / scale > far || (t == kBins - 1 && isinf(t_of(sc, floor_x)));
    }
    if (here) atomicMin(&sh.pick[0], t);
    if (t == 0) sh.n_list = 0;
    __syncthreads();
    const int bin_end = sh.pick[0];
    if (bin_end == 0x7fffffff) return kPast;  // the prefix goes on past the list
    if (t == bin_end) sh.red_u[0] = cum;
    __syncthreads();
    const int n = (int)sh.red_u[0];
    if (n > kSorted) return kPast;
    int n2 = 64;
    while (n2 < n) n2 *= 2;
    for (int i = t; i < n_all; i += kST) {
      const unsigned long long it = final_list[i];
      if (bin_of(t_of(sc, of_key(~(unsigned)(it >> 32)))) <= bin_end) list[atomicAdd(&sh.n_list, 1u)] = it;
    }
    for (int i = n + t; i < n2; i += kST) list[i] = ~0ull;
    if (t == 0) sh.pick[0] = 0x7fffffff;
    __syncthreads();
    auto sort = [&](auto* v, int len_all) {  // ascending, bitonic; up to 64 by one warp
      if (len_all > 64 || warp == 0) {
        for (int len = 2; len <= len_all; len *= 2) {
          for (int d = len / 2; d > 0; d /= 2) {
            for (int i = t; i < len_all / 2; i += kST) {
              const int a = 2 * i - (i & (d - 1)), b = a + d;
              const auto va = v[a], vb = v[b];
              if ((va > vb) == ((a & len) == 0)) v[a] = vb, v[b] = va;
            }
            if (len_all > 64) __syncthreads(); else __syncwarp();
          }
        }
      }
      __syncthreads();
    };
    sort(list, n2);  // by (falling logit, index)
    // thread t has items [t per, (t + 1) per): weights (units of 2^-52) and their running sum
    const int per = max(1, n2 / kST), i0 = t * per;
    static_assert(kSorted / kST <= 32, "one bit per item");
    unsigned long long mine = 0;
    unsigned low = 0;  // items below min-p
#pragma unroll 1
    for (int e = 0; e < per; ++e) {
      const int i = i0 + e;
      if (i >= n) break;
      const unsigned long long it = list[i];
      const F2 f = weight(sc, of_key(~(unsigned)(it >> 32)));
      const unsigned long long w = fix<52>(f);
      low |= (unsigned)below(f, r.lo) << e;
      index[i] = (unsigned)it;
      list[i] = w;
      mine += w;
    }
    const unsigned long long before = scan_l(mine, &all);
    const int k_end = r.use_k ? min(n, r.k) : n;
    if (r.use_p && !goal_set) {  // the goal is a part of the mass left by top-k
      unsigned long long run = before;
      for (int e = 0; e < per && i0 + e < k_end; ++e) {
        run += list[i0 + e];
        if (i0 + e == k_end - 1) sh.before = run;
      }
      __syncthreads();
      bool more;
      goal = part_of(sh.before, r.p, &more);
      goal += more;
    }
    // the kept prefix: its length and mass
    unsigned long long run = before, kept_w = 0;
    int n_kept = 0;
    // the goal's error: the fp32 weights', those below the cut, and the roundings of the parts (2^-44 a warp)
    unsigned long long slack = sum && sh.rest ? 1ull << 15 : 0ull;
    if (slack && !exact_rest)
      slack += (far_error(sh.rest, q.vocab) << 9) + (sh.m_look < m_row ? (unsigned long long)q.vocab << 12 : 0ull);
    bool unsure = false;
    for (int e = 0; e < per && i0 + e < k_end; ++e) {
      const unsigned long long w = list[i0 + e];
      if ((i0 + e == 0 || run < goal) && !(low >> e & 1) && w > 0) ++n_kept, kept_w += w;
      run += w;
      unsure |= slack && (run > goal ? run - goal : goal - run) <= slack;
    }
    if (__syncthreads_or(unsure)) return kUnsure;
    n_kept = __reduce_add_sync(0xffffffffu, n_kept);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) kept_w += __shfl_xor_sync(0xffffffffu, kept_w, o);
    if (lane == 0) sh.red_u[warp] = n_kept, sh.red_l[warp] = kept_w;
    __syncthreads();
    n_kept = 0;
    kept_w = 0;
    for (int w = 0; w < kSW; ++w) n_kept += sh.red_u[w], kept_w += sh.red_l[w];
    const unsigned long long target = part_of(kept_w, r.u);
    // the lowest index at which the running sum by index exceeds the target, else the last one
    // (packed with the item's place: below 2^20 and 2^11)
    if (n_kept <= 128) {
      if (t < n_kept) {
        const unsigned me = index[t];
        unsigned long long s = 0;
        for (int j = 0; j < n_kept; ++j) s += index[j] <= me ? list[j] : 0ull;
        const int at = (int)(me << 11 | t);
        if (s > target) atomicMin(&sh.pick[0], at);
        atomicMax(&sh.pick[1], at);
      }
    } else {
      int m2 = 256;
      while (m2 < n_kept) m2 *= 2;
      for (int i = t; i < m2; i += kST) by[i] = i < n_kept ? index[i] << 11 | i : 0xffffffffu;
      __syncthreads();
      sort(by, m2);
      const int c = m2 / kST, j0 = t * c;
      unsigned long long s = 0;
      for (int e = 0; e < c && j0 + e < n_kept; ++e) s += list[by[j0 + e] & 2047];
      s = scan_l(s, &all);
      for (int e = 0; e < c && j0 + e < n_kept; ++e) {
        s += list[by[j0 + e] & 2047];
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
      put(q, row, at >= 0 ? at >> 11 : -1, at >= 0 ? (float)((double)list[at & 2047] / (double)kept_w) : 0.f);
    }
    return kDone;
  };

  // (tau, n_tau): logits above tau are kept, and the n_tau first of those equal to it (by keys)
  unsigned tau = digit_key<T>(-INFINITY), n_tau = 0;  // -inf itself is never drawn
  bool ties = false, exact = false;
  if (by_list) {
    for (;;) {
      {  // gather the row's list in the first CTA (its ring is idle: its own part of the row is through)
        if (rest.h > 0.f) rest = mul(rest, weight(sc, m));
        m = m_row;
        bounds();
        unsigned long long* dst = peer(final_list, 0);
        unsigned* n_at = peer(&sh.n_final, 0);
        const int n = (int)min(sh.n_list, (unsigned)kList);
        bool full = sh.n_list > kList;
        // (whole warps: a vector per lane, their hits counted together)
        for (int i = t; i < (n + 31) / 32 * 32; i += kST) {
          float x[N];
          const int pos = i < n ? (int)places[i] : 0;
          if (i < n) Vec<T>::get(sl.vector(pos), x);
          int hits = 0;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            if (i >= n) x[e] = -INFINITY;
            hits += x[e] >= floor_x && x[e] > -INFINITY;
          }
          int inc = hits;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
          }
          unsigned at = 0;
          if (lane == 31) at = atomicAdd(n_at, (unsigned)inc);
          at = __shfl_sync(0xffffffffu, at, 31) + inc - hits;
#pragma unroll
          for (int e = 0; e < N; ++e) {
            if (x[e] >= floor_x && x[e] > -INFINITY) {
              if (at < kList)
                dst[at++] = (unsigned long long)~key_of(x[e] + 0.f) << 32 | (unsigned)(sl.first + pos + e);
              else
                full = true;
              x[e] = -INFINITY;
            }
          }
          if (sum && finite) {
            if (!exact_rest)
              rest = add(rest, F2{fast_of(x), 0.f});
            else if (i < n)
              rest = add(rest, slow(sl.vector(pos), floor_x));
          }
        }
        if (full) atomicOr(peer(&sh.full, 0), 1u);
        if (sum) {
          F2 s = rest;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s = shfl_add(s, o);
          if (lane == 0) atomicAdd(peer(&sh.rest, 0), fix<43>(s));
        }
      }
      sync_row();
      if (rank == 0) {
        const int what = from_list();
        if (t == 0)
          for (int c = 0; c < C; ++c) *peer(&sh.again, c) = (unsigned)what;
      }
      sync_row();
      if (!sh.again) return;
      // once more, with exact weights or with a floor that a look sets
      const bool unsure = sh.again == kUnsure;
      if (unsure ? exact_rest : looked || (!r.use_k && !r.use_p)) break;
      m = m_row;
      __syncthreads();
      if (t < kBins) sh.count[t] = 0, sh.mass[t] = 0;
      if (t == 0) {
        sh.n_list = sh.n_final = sh.full = 0;
        sh.rest = 0;
        sh.m_look = m_row;
        sh.pick[0] = 0x7fffffff;
        sh.pick[1] = -1;
      }
      start();
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      if (unsure) exact_rest = true; else looked = true, floor_by_look();
      rest = {0.f, 0.f};
      bounds();
      stream(first_pass);
      sync_row();
    }

    // ---- by histograms over keys.  One border: the first key, falling, by which the count reaches
    // k (by_mass: the mass reaches p of all).  Rounds over keys [lo, hi], kDigit bits of them each;
    // keys below tau_k do not take part and n_k of those equal to it do.  false: it is not reached.
    m = m_row;
    auto border = [&](bool by_mass, unsigned tau_k, unsigned n_k, unsigned* key, u128* left) {
      unsigned hi = digit_key<T>(m_row);
      unsigned lo = max(tau_k, digit_key<T>(by_mass ? fmaxf(reach(sc, kCut), -FLT_MAX) : -FLT_MAX));
      u128 goal = (unsigned)r.k, above = 0;
      const u128 w_k = by_mass && n_k > 0 ? (u128)n_k * fix<kKeyUnit>(weight(sc, of_digit_key<T>(tau_k))) : 0;
      for (bool first = true;; first = false) {
        const int bits = 32 - __clz(hi - lo), shift = max(0, bits - kDigit);
        const bool by_count = !by_mass || shift == 0;  // (one key a bin: its mass is the count times its weight)
        for (int i = t; i < kKeys * kParts; i += kST) digits[i] = 0;
        if (t == 0) sh.pick[0] = -1;
        start();
        __syncthreads();
        const float from = of_digit_key<T>(lo);
        stream([&](int b, uint4 (&x4)[kVec], float (&tops)[kVec], auto&& next) {
          next();
#pragma unroll 1
          for (int v = 0; v < kVec; ++v) {
            const uint4 y4 = v == 0 ? x4[0] : v == 1 ? x4[1] : v == 2 ? x4[2] : x4[3];
            if (!(Vec<T>::top(y4) >= from)) continue;
            float x[N];
            Vec<T>::get(y4, x);
#pragma unroll
            for (int e = 0; e < N; ++e) {
              const unsigned k = digit_key<T>(clean(x[e]));
              if (k < lo || k > hi) continue;
              unsigned* d = digits + ((hi - k) >> shift);
              if (by_mass && k == tau_k && n_k > 0) continue;  // (w_k has them)
              if (by_count) {
                atomicAdd(d, 1u);
              } else {
                const unsigned long long w = fix<kKeyUnit>(weight(sc, clean(x[e])));
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                  const unsigned part = (unsigned)(w >> kPartBits * i) & ((1u << kPartBits) - 1);
                  if (part) atomicAdd(d + i * kKeys, part);
                }
              }
            }
          }
        });
        sync_row();
        constexpr int kB = kKeys / kST;  // thread t: bins kB t ..
        u128 v[kB], mine = 0, all;
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          v[b] = 0;
          const int at = t * kB + b;
          for (int c = 0; c < C; ++c) {
            const unsigned* d = peer(digits, c) + at;
            for (int i = 0; i < (by_count ? 1 : kParts); ++i) v[b] += (u128)d[i * kKeys] << kPartBits * i;
          }
          if (by_mass && by_count && v[b] > 0) v[b] *= fix<kKeyUnit>(weight(sc, of_digit_key<T>(hi - at)));
          if (by_mass && n_k > 0 && tau_k >= lo && tau_k <= hi && (int)((hi - tau_k) >> shift) == at) v[b] += w_k;
          mine += v[b];
        }
        u128 run = above + scan_w(mine, &all);
        if (first && by_mass) {
          bool more;
          goal = part_of(all, r.p, &more) + more;
          if (goal == 0) goal = 1;  // the first always stays
        }
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          if (run < goal && run + v[b] >= goal) sh.pick[0] = t * kB + b, sh.above = run;
          run += v[b];
        }
        sync_row();  // every CTA has read the others' bins
        const int b = sh.pick[0];
        above = b < 0 ? above : sh.above;
        __syncthreads();  // read before the next round resets it
        if (b < 0) return false;
        hi -= (unsigned)b << shift;
        lo = max(lo, hi - ((1u << shift) - 1));
        if (shift == 0) {
          *key = hi;
          *left = goal - above;
          return true;
        }
      }
    };
    u128 left;
    if (r.use_k && border(false, 0, 0, &tau, &left)) {  // (else fewer than k candidates: all stay)
      n_tau = (unsigned)left;
      ties = true;
    }
    if (r.use_p) {
      const unsigned n_k = n_tau;
      unsigned key;
      if (border(true, tau, n_k, &key, &left)) {
        // of the keys equal to it: those before which less than the goal lies (1 + the largest n of
        // which the mass is below)
        const unsigned long long w = fix<kKeyUnit>(weight(sc, of_digit_key<T>(key)));
        unsigned n = 0;
        for (unsigned bit = 1u << 20; bit > 0; bit >>= 1)
          if ((u128)(n | bit) * w < left) n |= bit;
        ++n;
        n_tau = key == tau && n_k > 0 ? min(n_k, n) : n;
        tau = key;
        ties = true;
      }
    }
    exact = true;
  }

  // ---- sums by stretch of what is kept (the first time, temperature alone: they are there)
  for (bool summed = !by_list;; summed = false, exact = true) {
    if (!summed) {
      m = m_row;
      const float from = fmaxf(fmaxf(reach(sc, kCut), of_digit_key<T>(tau)), r.lo > 0.f && r.lo < 1.f ? reach(sc, -log2f(r.lo) + 0.01f) : -INFINITY);
      if (ties) {  // ties at tau ahead of each stretch
        start();
        stream([&](int b, uint4 (&x4)[kVec], float (&tops)[kVec], auto&& next) {
          next();
          unsigned n = 0;
#pragma unroll
          for (int v = 0; v < kVec; ++v) {
            if (!(tops[v] >= from)) continue;
            float x[N];
            Vec<T>::get(x4[v], x);
#pragma unroll
            for (int e = 0; e < N; ++e) n += x[e] > -INFINITY && digit_key<T>(clean(x[e])) == tau;
          }
          n = __reduce_add_sync(0xffffffffu, n);
          if (lane == 0) stretch[b * kSW + warp].ties = n;
        });
        __syncthreads();
        const int n = blocks * kSW, per = (n + kST - 1) / kST;
        unsigned long long mine = 0, part;
        for (int i = t * per; i < min(n, (t + 1) * per); ++i) mine += stretch[i].ties;
        unsigned long long run = scan_l(mine, &part);
        if (t == 0) sh.ties = (unsigned)part;
        sync_row();
        for (int c = 0; c < rank; ++c) run += *peer(&sh.ties, c);
        for (int i = t * per; i < min(n, (t + 1) * per); ++i) {
          const unsigned x = stretch[i].ties;
          stretch[i].ties = (unsigned)run;
          run += x;
        }
        sync_row();  // (the counts have been read)
      }
      start();
      stream([&](int b, uint4 (&x4)[kVec], float (&tops)[kVec], auto&& next) {
        next();
        F2 s = {0.f, 0.f};
        unsigned at = ties ? stretch[b * kSW + warp].ties : 0u;
        const unsigned ahead = at;
#pragma unroll 1
        for (int v = 0; v < kVec; ++v) {
          const uint4 y4 = v == 0 ? x4[0] : v == 1 ? x4[1] : v == 2 ? x4[2] : x4[3];
          const bool any = Vec<T>::top(y4) >= from;
          if (!__any_sync(0xffffffffu, any)) continue;
          float x[N];
          Vec<T>::get(y4, x);
          unsigned eq = 0, inc = 0;
          if (ties) {
#pragma unroll
            for (int e = 0; e < N; ++e) eq += x[e] > -INFINITY && digit_key<T>(clean(x[e])) == tau;
            inc = eq;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
              if (lane >= o) inc += y;
            }
          }
          unsigned mine = at + inc - eq;
          if (any) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
              const float c = clean(x[e]);
              const unsigned k = digit_key<T>(c);
              if (c > -INFINITY && (k > tau || (ties && k == tau && mine++ < n_tau))) {
                const F2 w = weight(sc, c);
                if (!below(w, r.lo)) s = add(s, w);
              }
            }
          }
          if (ties) at += __shfl_sync(0xffffffffu, inc, 31);
        }
        unsigned long long mass = fix<kStretchUnit>(s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
        if (lane == 0) stretch[b * kSW + warp] = Stretch{mass, ahead, m_row};
      });
      __syncthreads();
    }
    // ---- the stretch that holds the target
    const int n = blocks * kSW, per = (n + kST - 1) / kST;
    u128 mine = 0, part;
    unsigned long long my_far = 0;  // (2^-43)
    unsigned my_cut = 0;            // logits of stretches that hold weights below the cut
    if (!exact) {
      // by the row's maximum now, and the near vectors exactly
      for (int i = t; i < n; i += kST) {
        Stretch& s = stretch[i];
        if (s.ref != m_row) {
          if (t_of(sc, of_key(s.ties)) > kCut - 0.01f) my_cut += kWarpPart;
          const float h = (float)s.mass, l = (float)(long long)(s.mass - (unsigned long long)h);
          s.mass = s.ref > -INFINITY ? fix<0>(mul(F2{h, l}, weight(sc, s.ref))) : 0ull;  // (in the same units)
        }
        my_far += (s.mass >> (kStretchUnit - 43)) + 1;
      }
      __syncthreads();
      for (int i = t; i < (int)min(sh.n_list, near_room); i += kST) {
        const int pos = near_places[i];
        float x[N];
        Vec<T>::get(sl.vector(pos), x);
        F2 s = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (clean(x[e]) > -INFINITY) s = add(s, weight(sc, clean(x[e])));
        atomicAdd(&stretch[pos / kBlock * kSW + pos % kBlock / kWarpPart].mass, fix<kStretchUnit>(s));
      }
      __syncthreads();
    }
    for (int i = t * per; i < min(n, (t + 1) * per); ++i) mine += stretch[i].mass;
    if (!exact && t == 0 && sh.n_list > near_room)  // near vectors were left out
      for (int c = 0; c < C; ++c) *peer(&sh.again, c) = 1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) my_far += __shfl_xor_sync(0xffffffffu, my_far, o);
    if (lane == 0 && my_far) atomicAdd(&sh.far, my_far);
    if (my_cut) atomicAdd(&sh.cut, my_cut);
    if (t == 0) sh.pick[0] = 0x7fffffff, sh.pick[1] = -1;
    u128 run = scan_w(mine, &part), total = part;
    unsigned long long far = sh.far;
    unsigned cut = sh.cut;
    int last = 0;  // the row's last CTA with any mass
    if (C > 1) {
      if (t == 0) sh.part = part, sh.far_part = far;
      cl.sync();
      total = far = cut = 0;
      for (int c = 0; c < C; ++c) {
        const u128 x = *peer(&sh.part, c);
        far += *peer(&sh.far_part, c);
        cut += *peer(&sh.cut, c);
        if (c < rank) run += x;
        if (x > 0) last = c;
        total += x;
      }
    }
    const bool whole = exact || !sh.again;
    const u128 target = part_of(total, r.u);
    // the fp32 sums' error, of what lies ahead (a) less u times the total's (a + b): at most
    // (1 - u) |a| + u |b|, for a and b together at most far_off; the weights below the cut, and the lanes'
    // roundings.  (Saturated: it is compared with masses of a stretch)
    const unsigned long long far_off = far_error(far, q.vocab);
    const unsigned long long slack =
        exact ? 0ull : (min(part_of(far_off, fmaxf(r.u, 1.f - r.u)), 1ull << 52) << (kStretchUnit - 43)) +
                           ((unsigned long long)cut << (kStretchUnit - (int)kCut)) + (1 << 16);
    for (int i = t * per; i < min(n, (t + 1) * per); ++i) {  // this CTA's first stretch past the target, and its last with any mass
      const unsigned long long x = stretch[i].mass;
      if (x > 0) {
        if (run <= target && run + x > target) {
          sh.pick[0] = i;
          sh.before = (unsigned long long)(target - run);  // of the target in this stretch
          sh.ties = run == 0;                              // nothing lies ahead of it
        }
        atomicMax(&sh.pick[1], i);
      }
      run += x;
    }
    __syncthreads();
    const bool mine_past = sh.pick[0] != 0x7fffffff;
    if (total == 0) {  // min-p above 1: nothing is left
      if (rank == 0 && t == 0) put(q, row, -1, 0.f);
    } else if (mine_past || (rank == last && target >= total)) {  // (u >= 1: the row's last kept one)
      // the whole CTA walks the stretch: thread t has its positions kE t .. kE t + kE - 1
      constexpr int kE = kWarpPart / kST;
      const int at = mine_past ? sh.pick[0] : sh.pick[1];
      const int i0 = at / kSW * kBlock + at % kSW * kWarpPart + t * kE;
      const unsigned long long goal = mine_past ? sh.before : ~0ull;  // masses from the stretch's start
      const bool at_start = mine_past && sh.ties;
      float x[kE];
      unsigned eq = 0;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int i = i0 + e;
        x[e] = i >= sl.begin && i < sl.count ? clean(Elem<T>::to_f(*sl.at(i))) : -INFINITY;
        eq += x[e] > -INFINITY && digit_key<T>(x[e]) == tau;
      }
      unsigned long long all;
      unsigned tie = ties ? (unsigned)scan_l(eq, &all) + stretch[at].ties : 0u;
      F2 w[kE];
      unsigned long long f[kE], sum_w = 0;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const unsigned k = digit_key<T>(x[e]);
        w[e] = F2{0.f, 0.f};
        if (x[e] > -INFINITY && (k > tau || (ties && k == tau && tie++ < n_tau))) w[e] = weight(sc, x[e]);
        if (below(w[e], r.lo)) w[e] = F2{0.f, 0.f};
        f[e] = fix<kStretchUnit>(w[e]);
        sum_w += f[e];
      }
      unsigned long long cum = scan_l(sum_w, &all);
      if (t == 0) sh.pick[0] = 0x7fffffff, sh.pick[1] = -1;
      __syncthreads();
      // the first position past the target, else the last with any mass
      int hit = -1, any = -1;
      unsigned long long from = 0, to = 0;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        if (f[e] > 0) {
          any = i0 + e;
          if (hit < 0 && cum + f[e] > goal) hit = i0 + e, from = cum, to = cum + f[e];
        }
        cum += f[e];
      }
      if (hit >= 0) atomicMin(&sh.pick[0], hit);
      if (any >= 0) atomicMax(&sh.pick[1], any);
      __syncthreads();
      const int token = sh.pick[0] != 0x7fffffff ? sh.pick[0] : sh.pick[1];
      // Nothing here counts: the fp32 sums, by the maximum as it was then, had weights in the stretch that
      // are below 2^-40 by the row's.
      if (token < 0 && t == 0)
        for (int c = 0; c < C; ++c) *peer(&sh.again, c) = 1;
      if (token >= i0 && token < i0 + kE) {
        F2 tw = w[0];
#pragma unroll
        for (int e = 1; e < kE; ++e)
          if (token == i0 + e) tw = w[e];
        // sure: the fp32 sums' error moves neither border of the token past the target, nor the
        // probability's last bit
        bool sure = exact || (whole && !mine_past) || (whole && token == hit && ((at_start && from == 0) || from + slack <= goal) && to > goal + slack);
        if (q.probs && !exact) sure = sure && (double)far_off * 0x1p9 <= to_double(total) * (double)kProbError;
        if (sure)
          put(q, row, sl.first + token, prob_of(tw, total));
        else
          for (int c = 0; c < C; ++c) *peer(&sh.again, c) = 1;  // once more, exactly
      }
    }
    sync_row();
    if (exact || !sh.again) return;
  }
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

template <typename T>
cudaError_t launch(SampleParams p, int sms, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  if (cudaError_t e = smem_attr_once(sample_kernel<T>, kStreamSmem, attr); e != cudaSuccess) return e;
  // as many CTAs per row (up to 8) as run together, three per SM, when the row is long enough to
  // be worth the exchanges: 64 rows of 262144 fp32 take 7
  const int64_t blocks = ((int64_t)p.vocab * (int)sizeof(T) + kStageBytes - 1) / kStageBytes;
  p.ctas = (int)std::max<int64_t>(1, std::min<int64_t>({(int64_t)kMaxC, 3ll * sms / p.rows, blocks / 2}));
  p.per = (p.vocab + 7 + p.ctas - 1) / p.ctas;  // (up to 7 positions before an unaligned row)
  p.per = (p.per + 7) / 8 * 8;
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = p.ctas;
  a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
  c.gridDim = dim3(p.rows * p.ctas);
  c.blockDim = dim3(kST);
  c.dynamicSmemBytes = kStreamSmem;
  c.stream = st;
  c.attrs = a;
  c.numAttrs = p.ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&c, sample_kernel<T>, p);
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
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == DFLASH_F32 ? 4 : 2)) return call_error(DFLASH_EINVAL, "sample: logits not whole elements");
  SampleParams p{logits, row_stride, rows, vocab, u, temperature, top_p, min_p, top_k, tokens, probs, 1, 0, {}};
  static const Powers powers;
  memcpy(p.table, powers.table, sizeof p.table);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e == cudaSuccess) e = dtype == DFLASH_F32 ? launch<float>(p, sms, st) : launch<__nv_bfloat16>(p, sms, st);
  if (e != cudaSuccess) return call_error(DFLASH_ECUDA, "sample", e);
  return DFLASH_OK;
}
