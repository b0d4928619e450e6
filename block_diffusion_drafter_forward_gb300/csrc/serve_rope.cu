// Rotary positions of a step's queries and keys (dflash_rotate) and their table (dflash_rope_turns).
#include <math.h>

#include <algorithm>

#include "launch_util.cuh"
#include "serve.cuh"

namespace dflash {
namespace {

struct RotateParams {
  const uint8_t* src[2];
  uint8_t* dst[2];
  int64_t ss[2], ds[2];  // bytes between rows
  const int32_t* positions;
  const unsigned long long* turns;
  int rows, q_heads, heads, groups, rotated;  // groups of 16 dims in a head, of them rotated
  int slots, per_row;                         // heads that a block takes at once, of one row
  float scale, sign;
  bool copy[2];  // the other dims, unless they are in place already
};

template <typename T> struct Eight;  // eight elements of a row in registers
template <> struct Eight<__nv_bfloat16> {
  uint4 w;
  __device__ void load(const void* p) { w = *static_cast<const uint4*>(p); }
  __device__ void store(void* p) const { *static_cast<uint4*>(p) = w; }
  __device__ float get(int i) const {
    const uint32_t x = (&w.x)[i >> 1];
    return __uint_as_float(i & 1 ? x & 0xffff0000u : x << 16);
  }
  __device__ void put(int i, float a, float b) {  // elements i, i + 1
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    (&w.x)[i >> 1] = *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <> struct Eight<float> {
  float4 w[2];
  __device__ void load(const void* p) { w[0] = static_cast<const float4*>(p)[0], w[1] = static_cast<const float4*>(p)[1]; }
  __device__ void store(void* p) const { static_cast<float4*>(p)[0] = w[0], static_cast<float4*>(p)[1] = w[1]; }
  __device__ float get(int i) const { return (&w[i >> 2].x)[i & 3]; }
  __device__ void put(int i, float a, float b) { (&w[i >> 2].x)[i & 3] = a, (&w[i >> 2].x)[(i & 3) + 1] = b; }
};

// A thread has one group of 16 dims (8 pairs) of one row and goes through every per_row-th head, so
// that an angle's sine and cosine serve many heads.  The angle is exact: position times the
// frequency in 2^-64 turns, modulo a turn, is one integer product, of which 32 bits stay.  The nearest quarter turn comes
// off as a whole number; the rest, an eighth of a turn at most, goes to fp32 with an error of 2^-28 turns, 2.3e-8 in sine
// and cosine, where their own last place is 6e-8 (the whole angle in fp32 would be off by 9.4e-8).  Rotating in fp32 and
// rounding once is the plain definition.
// Bound by HBM: 16 Ki rows of 64 + 8 heads of 128 in bf16 94.9 us, 6.4 TB/s (94 % of the copy rate); by latency where
// rows are few: then every head of a row has threads of its own (64 rows of 32 + 4 heads 2.9 us).
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(256) rotate_kernel(const RotateParams p) {
  const int g = threadIdx.x % p.groups, slot = threadIdx.x / p.groups;
  if (slot >= p.slots) return;
  const int64_t row = (int64_t)blockIdx.x * (p.slots / p.per_row) + slot / p.per_row;
  if (row >= p.rows) return;
  int h = slot % p.per_row;
  const int hd = p.groups * 16;
  // the group's two runs of eight dims
  const int a = kInterleaved || g >= p.rotated ? 16 * g : 8 * g;
  const int b = kInterleaved || g >= p.rotated ? a + 8 : a + 8 * p.rotated;
  float c[8], s[8];
  if (g < p.rotated) {
    const long long pos = p.positions[row];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t turn = (unsigned long long)pos * __ldg(p.turns + 8 * g + i) >> 32, quarter = turn + (1u << 29) >> 30;
      float x, y;  // sine and cosine of the rest
      sincospif((float)(int)(turn - (quarter << 30)) * 0x1p-31f, &x, &y);  // half turns in [-1/4, 1/4]
      c[i] = __uint_as_float(__float_as_uint((quarter & 1 ? x : y) * p.scale) ^ (quarter + 1 & 2) << 30);
      s[i] = __uint_as_float(__float_as_uint((quarter & 1 ? y : x) * p.sign) ^ (quarter & 2) << 30);
    }
  }
#pragma unroll 2
  for (; h < p.heads; h += p.per_row) {
    const bool key = h >= p.q_heads;
    const int64_t at = (int64_t)(key ? h - p.q_heads : h) * hd * sizeof(T);
    const uint8_t* src = (key ? p.src[1] + row * p.ss[1] : p.src[0] + row * p.ss[0]) + at;
    uint8_t* dst = (key ? p.dst[1] + row * p.ds[1] : p.dst[0] + row * p.ds[0]) + at;
    if (g >= p.rotated && !(key ? p.copy[1] : p.copy[0])) continue;
    Eight<T> u, v;
    u.load(src + a * sizeof(T));
    v.load(src + b * sizeof(T));
    if (g < p.rotated) {
      if (kInterleaved) {
        auto turn = [&](Eight<T>& e, int i0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float xa = e.get(2 * i), xb = e.get(2 * i + 1);
            e.put(2 * i, xa * c[i0 + i] - xb * s[i0 + i], xb * c[i0 + i] + xa * s[i0 + i]);
          }
        };
        turn(u, 0);
        turn(v, 4);
      } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float a0 = u.get(i), a1 = u.get(i + 1), b0 = v.get(i), b1 = v.get(i + 1);
          u.put(i, a0 * c[i] - b0 * s[i], a1 * c[i + 1] - b1 * s[i + 1]);
          v.put(i, b0 * c[i] + a0 * s[i], b1 * c[i + 1] + a1 * s[i + 1]);
        }
      }
    }
    u.store(dst + a * sizeof(T));
    v.store(dst + b * sizeof(T));
  }
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" int dflash_rope_turns(int32_t rotary_dim, double theta, double linear, int32_t yarn, double yarn_factor,
                                 double yarn_orig_max_pos, double yarn_beta_fast, double yarn_beta_slow,
                                 uint64_t* turns, float* mscale) {
  if (!turns || !mscale) return call_error(DFLASH_EINVAL, "rope_turns: null pointer");
  if (rotary_dim < 16 || rotary_dim > 512 || rotary_dim % 16) return call_error(DFLASH_EUNSUPPORTED, "rope_turns: rotary_dim must be a multiple of 16 up to 512");
  if (!(theta > 1.) || !isfinite(theta) || !(linear >= 1.) || !isfinite(linear))
    return call_error(DFLASH_EINVAL, "rope_turns: theta must be above 1, linear at least 1");
  if (yarn && (linear != 1. || !(yarn_factor >= 1.) || !isfinite(yarn_factor) || !(yarn_orig_max_pos > 0.) ||
               !isfinite(yarn_orig_max_pos) || !(yarn_beta_fast > 0.) || !(yarn_beta_slow > 0.)))
    return call_error(DFLASH_EINVAL, "rope_turns: bad YaRN parameters");
  const double d = rotary_dim;
  double low = 0, denom = 1;
  *mscale = 1.f;
  if (yarn) {
    auto pair_of = [&](double beta) { return d * log(yarn_orig_max_pos / (beta * 2.0 * M_PI)) / (2.0 * log(theta)); };
    low = fmax(floor(pair_of(yarn_beta_fast)), 0.0);
    const double high = fmin(ceil(pair_of(yarn_beta_slow)), d - 1.0);
    denom = fabs(high - low) < 1e-6 ? high - low + 0.001 : high - low;
    *mscale = (float)(0.1 * log(yarn_factor) + 1.0);
  }
  for (int j = 0; j < rotary_dim / 2; ++j) {
    double f = pow(theta, -2.0 * j / d) / linear;
    if (yarn) {
      const double ramp = fmin(fmax((j - low) / denom, 0.0), 1.0);
      f = f / yarn_factor * ramp + f * (1.0 - ramp);
    }
    turns[j] = (uint64_t)ldexp(f / (2.0 * M_PI), 64);  // f <= 1: below 2^62
  }
  return DFLASH_OK;
}

extern "C" int dflash_rotate(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int32_t q_heads,
                             const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride, int32_t k_heads,
                             int32_t dtype, int32_t rows, int32_t head_dim, int32_t rotary_dim, int32_t interleaved,
                             int32_t inverse, const int32_t* positions, const uint64_t* turns, float mscale,
                             dflash_stream stream) {
  if (dtype != DFLASH_BF16 && dtype != DFLASH_F32) return call_error(DFLASH_EINVAL, "rotate: dtype must be bf16 or f32");
  if (head_dim < 16 || head_dim > 512 || head_dim % 16 || rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16)
    return call_error(DFLASH_EUNSUPPORTED, "rotate: head_dim must be a multiple of 16 up to 512, rotary_dim one up to head_dim");
  if (q_heads < 1 || k_heads < 0 || (int64_t)q_heads + k_heads > 4096)
    return call_error(DFLASH_EINVAL, "rotate: q_heads >= 1, k_heads >= 0, at most 4096 together");
  if (rows < 0) return call_error(DFLASH_EINVAL, "rotate: rows must be >= 0");
  if (rows > 1 << 30) return call_error(DFLASH_ECAPACITY, "rotate: rows above 2^30");
  if (!(fabsf(mscale) <= 3.4e38f)) return call_error(DFLASH_EINVAL, "rotate: mscale must be finite");
  if (rows == 0) return DFLASH_OK;
  if (!q || !q_out || !positions || !turns || (k_heads > 0 && (!k || !k_out))) return call_error(DFLASH_EINVAL, "rotate: null pointer");
  const int es = dtype == DFLASH_F32 ? 4 : 2;
  auto bad = [&](const void* p, int64_t stride, int heads) {
    return stride < (int64_t)heads * head_dim || stride > INT64_MAX / 8 || (stride * es) % 16 || !aligned16(p);
  };
  if (bad(q, q_stride, q_heads) || bad(q_out, q_out_stride, q_heads) ||
      (k_heads > 0 && (bad(k, k_stride, k_heads) || bad(k_out, k_out_stride, k_heads))))
    return call_error(DFLASH_EINVAL, "rotate: rows below their heads, or an address or a stride not whole 16 bytes");
  if ((q == q_out && q_stride != q_out_stride) || (k_heads > 0 && k == k_out && k_stride != k_out_stride))
    return call_error(DFLASH_EINVAL, "rotate: in place needs one stride");
  RotateParams p;
  p.src[0] = static_cast<const uint8_t*>(q), p.dst[0] = static_cast<uint8_t*>(q_out), p.ss[0] = q_stride * es, p.ds[0] = q_out_stride * es;
  p.src[1] = static_cast<const uint8_t*>(k), p.dst[1] = static_cast<uint8_t*>(k_out), p.ss[1] = k_stride * es, p.ds[1] = k_out_stride * es;
  p.copy[0] = q != q_out, p.copy[1] = k != k_out;
  p.positions = positions;
  p.turns = reinterpret_cast<const unsigned long long*>(turns);
  p.rows = rows, p.q_heads = q_heads, p.heads = q_heads + k_heads;
  p.groups = head_dim / 16, p.rotated = rotary_dim / 16;
  p.scale = mscale, p.sign = inverse ? -mscale : mscale;
  int sms = 0;
  if (cudaError_t e = sm_count(&sms); e != cudaSuccess) return call_error(DFLASH_ECUDA, "rotate", e);
  const int most = 256 / p.groups;  // heads of a block at once
  const int64_t fill = ((int64_t)sms * 1024 + (int64_t)rows * p.groups - 1) / ((int64_t)rows * p.groups);
  p.per_row = (int)std::min<int64_t>(std::min(most, p.heads), std::max<int64_t>(fill, 4));
  const int per_block = most / p.per_row;  // rows
  p.slots = per_block * p.per_row;
  const unsigned blocks = (unsigned)(((int64_t)rows + per_block - 1) / per_block);
  auto kern = dtype == DFLASH_F32 ? (interleaved ? rotate_kernel<float, true> : rotate_kernel<float, false>)
                                  : (interleaved ? rotate_kernel<__nv_bfloat16, true> : rotate_kernel<__nv_bfloat16, false>);
  kern<<<blocks, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return call_error(DFLASH_ECUDA, "rotate", e);
  return DFLASH_OK;
}
