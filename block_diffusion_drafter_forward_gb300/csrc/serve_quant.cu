// K/V rows into pages of 8 bits (dflash_append_kv_quant) and out of them (dflash_read_kv_quant).
//
// A row of a head becomes hd e4m3 codes of x 2^-k and the byte k + 127, k the smallest integer with
// max |x| <= 448 2^k.  A power of two instead of max / 448 costs at most one bit of e4m3's exponent
// range and no precision, and makes every stored value a bf16 number: reading rounds nothing, and
// attention over these pages is attention over bf16 pages that hold those numbers.
//
// Both kernels take a block of 16 consecutive rows and a warp per entry: a run of eight rows whose
// slots fill one half page in order (a step's rows of a sequence follow one another), or a single row.
// A lane has eight dims of a row (16 bytes of bf16): K moves as it is, 8 codes at a time; of V a lane
// has eight dims of four rows, and the transpose of those is byte permutes in registers, so that a run
// reads and writes whole sectors.  A single row's V goes byte by byte.  With heads of 64 a warp has two
// heads at a time.  Rounding: e4m3 to nearest even, by definition; the power of two is exact.
// Bound by HBM, from which instructions and the chain of a run (slots, rows, maxima, codes) still keep them: 16.7 Ki rows
// of 8 heads of 128 in bf16 25.8 us in and 21.7 us out, 3.9 and 4.6 TB/s (1024 rows of 4 heads 3.9 us each way).
#include <cuda_fp8.h>

#include <algorithm>
#include <cstdio>

#include "launch_util.cuh"
#include "serve.cuh"

namespace dflash {
namespace {

constexpr int kRows = 16, kWarps = 8;

struct QuantParams {
  const uint8_t *k, *v;  // rows (append) ...
  uint8_t *ko, *vo;      // ... or where they go (read)
  int64_t ks, vs;        // bytes between rows
  uint8_t* pool;
  int64_t page_bytes;
  const int32_t* slots;
  uint32_t* status;
  int n, nkv, num_pages;
};

// What a warp finds out by itself of the block's rows (every warp alike, without a barrier: with one, seven warps of
// eight waited for the first at 30 % of HBM).  Lane l holds the slot of row r0 - 7 + l - the rows here, and seven on
// either side that a run may reach - and the l-th entry: its row, | 64 for a run.
struct Entries {
  int slot, entry, n;
  unsigned none;  // rows without a place, a bit each
};
__device__ __forceinline__ Entries find_entries(const QuantParams& p, int r0) {
  Entries e;
  const int lane = threadIdx.x & 31, r = r0 - 7 + lane;
  e.slot = lane < kRows + 14 && r >= 0 && r < p.n ? p.slots[r] : -1;
  const bool good = e.slot >= 0 && e.slot / kPage < p.num_pages;
  if (threadIdx.x < 32 && blockIdx.y == 0 && p.status && lane >= 7 && lane < 7 + kRows && e.slot >= 0 && !good)
    atomicOr(p.status, DFLASH_DEV_BAD_PAGE);
  const int before = __shfl_up_sync(0xffffffffu, e.slot, 1);
  const unsigned next = __ballot_sync(0xffffffffu, lane > 0 && good && before >= 0 && e.slot == before + 1);  // one behind the row before
  const unsigned first = __ballot_sync(0xffffffffu, good && (e.slot & 7) == 0);
  const int o = e.slot & 7, s = lane - o;  // a row's run is decided alike in every block that sees it
  const bool run = good && s >= 0 && (first >> s & 1) && (next >> s >> 1 & 0x7f) == 0x7f;
  const bool here = lane >= 7 && lane < 7 + kRows && r < p.n;
  const unsigned take = __ballot_sync(0xffffffffu, here && good && (!run || o == 0));  // a run belongs to the block of its first row
  const unsigned runs = __ballot_sync(0xffffffffu, run);
  e.none = __ballot_sync(0xffffffffu, here && !good) >> 7;
  e.n = __popc(take);
  const int at = (int)__fns(take, 0, lane + 1);  // (-1: no such entry)
  e.entry = at < 0 ? 0 : (at - 7) | (runs >> at & 1 ? 64 : 0);
  return e;
}

// Eight dims of a row as they are loaded, and as fp32.
template <typename T> struct Raw { uint4 w[sizeof(T) / 2]; };
template <typename T>
__device__ __forceinline__ void load8(const uint8_t* p, Raw<T>& x) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) x.w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
}
__device__ __forceinline__ void open8(const Raw<__nv_bfloat16>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float((&r.w[0].x)[i] << 16), x[2 * i + 1] = __uint_as_float((&r.w[0].x)[i] & 0xffff0000u);
}
__device__ __forceinline__ void open8(const Raw<float>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float((&r.w[i >> 2].x)[i & 3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {  // (bf16 numbers: no rounding)
  uint4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) (&w.x)[i] = __byte_perm(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]), 0x7632);
  *reinterpret_cast<uint4*>(p) = w;
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Codes of a row held eight dims a lane by kLanes neighbouring lanes; *e: its exponent byte.  NaN become NaN by the
// conversion and are no maximum; rows with infinities (a maximum of infinity) are looked at once more.
template <int kLanes, typename T>
__device__ __forceinline__ uint2 encode(const Raw<T>& raw, int* e) {
  float x[8];
  open8(raw, x);
  float m = fmaxf(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))),
                  fmaxf(fmaxf(fabsf(x[4]), fabsf(x[5])), fmaxf(fabsf(x[6]), fabsf(x[7]))));
  m = m == m ? m : 0.f;  // (all of them NaN)
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (__any_sync(0xffffffffu, m == INFINITY)) {
    m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (fabsf(x[i]) == INFINITY) x[i] = __uint_as_float(0x7fc00000u);
      m = fmaxf(m, fabsf(x[i]));
    }
    m = m == m ? m : 0.f;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  const uint32_t top = __float_as_uint(m);
  // max = 1.m 2^(E - 127) <= 448 2^k = 1.75 2^(k + 8)
  const int k = min(max((int)(top >> 23) - 135 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), -118), 119);
  *e = k + 127;
  const float f = pow2i(-k);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * f, x[2 * i + 1] * f), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
__device__ __forceinline__ void decode4(uint32_t w, float f, float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16 * i), __NV_E4M3);
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = v.x * f, x[2 * i + 1] = v.y * f;
  }
}

// Four words of four bytes, transposed.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
  const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
  w[0] = __byte_perm(a, b, 0x5410), w[1] = __byte_perm(a, b, 0x7632);
  w[2] = __byte_perm(c, d, 0x5410), w[3] = __byte_perm(c, d, 0x7632);
}

// The units (entry, heads) of a warp: every kWarps-th, entries first.
struct Units {
  int entry, head, de, dh, n;
  __device__ __forceinline__ Units(int warp, int n) : entry(warp % max(n, 1)), head(warp / max(n, 1)), de(kWarps % max(n, 1)), dh(kWarps / max(n, 1)), n(n) {}
  __device__ __forceinline__ void next() {
    entry += de, head += dh;
    if (entry >= n) entry -= n, ++head;
  }
};
// Bytes of a half page's rows (j = 0 or 8) in a tile, d a multiple of 8: K of row j + 2 r + half, and V of rows j + 4 half .. + 3
// of dim d + x.  (k8_in_tile and v8_in_tile with what is known of j and d.)
__device__ __forceinline__ int k_of_run(int j, int half, int r, int d) {
  return (d >> 6) * 1024 + (d & 8) + (j + half) * 64 + r * 128 + (((d >> 4 & 3) ^ r) * 16);
}
__device__ __forceinline__ int v_of_run(int j, int half, int d, int x) {
  return (d >> 5) * 512 + (d >> 3 & 3) * 4 + x * 64 + (((j >> 2) + half) ^ (x >> 1)) * 16;
}

template <typename T, int HD>
__global__ void __launch_bounds__(32 * kWarps) append_quant_kernel(const QuantParams p) {
  constexpr int kPieces = HD / 8, kHeads = 16 / kPieces;  // lanes of a row; heads of a warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r0 = blockIdx.x * kRows;
  const Entries e = find_entries(p, r0);
  const int half = lane >> 4, sub = (lane & 15) / kPieces, d = lane % kPieces * 8;
  const int groups = (p.nkv + kHeads - 1) / kHeads, per = gridDim.y, mine = (groups - (int)blockIdx.y + per - 1) / per;
  if (e.n == 0) return;
  for (Units u(warp, e.n); u.head < mine; u.next()) {
    const int en = __shfl_sync(0xffffffffu, e.entry, u.entry), h = (blockIdx.y + u.head * per) * kHeads + sub;
    const bool on = h < p.nkv;  // (lanes past the last head follow its neighbours' shuffles)
    const int i = en & 63, slot = __shfl_sync(0xffffffffu, e.slot, 7 + i), j = slot % kPage;
    const int64_t row = r0 + i;
    uint8_t* tile = p.pool + (int64_t)(slot / kPage) * p.page_bytes + (int64_t)h * (32 * HD + 32);
    const uint8_t* src[2] = {p.k + row * p.ks, p.v + row * p.vs};
    const int64_t at = ((int64_t)h * HD + d) * sizeof(T);
    auto fetch = [&](int side, int r, Raw<T>& x) {
      if (on) {
        load8(src[side] + r * (side ? p.vs : p.ks) + at, x);
      } else {
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) x.w[k] = make_uint4(0, 0, 0, 0);
      }
    };
    if (en & 64) {
      Raw<T> x[4], y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) fetch(0, 2 * r + half, x[r]);
#pragma unroll
      for (int r = 0; r < 4; ++r) fetch(1, 4 * half + r, y[r]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        int ex;
        const uint2 c = encode<kPieces>(x[r], &ex);
        if (on) *reinterpret_cast<uint2*>(tile + k_of_run(j, half, r, d)) = c;
        if (on && d == 0) tile[32 * HD + j + 2 * r + half] = (uint8_t)ex;
      }
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        int ex;
        const uint2 c = encode<kPieces>(y[r], &ex);
        lo[r] = c.x, hi[r] = c.y;
        if (on && d == 0) tile[32 * HD + 16 + j + 4 * half + r] = (uint8_t)ex;
      }
      transpose4(lo);
      transpose4(hi);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (!on) continue;
        *reinterpret_cast<uint32_t*>(tile + 16 * HD + v_of_run(j, half, d, r)) = lo[r];
        *reinterpret_cast<uint32_t*>(tile + 16 * HD + v_of_run(j, half, d, 4 + r)) = hi[r];
      }
    } else {  // K by the lower lanes, V by the upper ones
      Raw<T> x;
      fetch(half, 0, x);
      int ex;
      const uint2 c = encode<kPieces>(x, &ex);
      if (!on) continue;
      if (half == 0) {
        *reinterpret_cast<uint2*>(tile + k8_in_tile(j, d)) = c;
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) tile[16 * HD + v8_in_tile(j, d + k)] = (uint8_t)((k < 4 ? c.x : c.y) >> 8 * (k & 3));
      }
      if (d == 0) tile[32 * HD + 16 * half + j] = (uint8_t)ex;
    }
  }
}

template <typename T, int HD>
__global__ void __launch_bounds__(32 * kWarps) read_quant_kernel(const QuantParams p) {
  constexpr int kPieces = HD / 8, kHeads = 16 / kPieces;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r0 = blockIdx.x * kRows;
  const Entries e = find_entries(p, r0);
  const int half = lane >> 4, sub = (lane & 15) / kPieces, d = lane % kPieces * 8;
  const int groups = (p.nkv + kHeads - 1) / kHeads, per = gridDim.y, mine = (groups - (int)blockIdx.y + per - 1) / per;
  auto put = [&](int side, int64_t row, int h, const float (&x)[8]) {
    uint8_t* dst = (side ? p.vo + row * p.vs : p.ko + row * p.ks) + ((int64_t)h * HD + d) * sizeof(T);
    store8(reinterpret_cast<T*>(dst), x);
  };
  for (Units u(warp, e.n); e.n > 0 && u.head < mine; u.next()) {
    const int en = __shfl_sync(0xffffffffu, e.entry, u.entry), h = (blockIdx.y + u.head * per) * kHeads + sub;
    const int i = en & 63, slot = __shfl_sync(0xffffffffu, e.slot, 7 + i), j = slot % kPage;
    if (h >= p.nkv) continue;
    const int64_t row = r0 + i;
    const uint8_t* tile = p.pool + (int64_t)(slot / kPage) * p.page_bytes + (int64_t)h * (32 * HD + 32);
    float x[8];
    if (en & 64) {
      uint2 c[4];
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        c[r] = *reinterpret_cast<const uint2*>(tile + k_of_run(j, half, r, d));
        lo[r] = *reinterpret_cast<const uint32_t*>(tile + 16 * HD + v_of_run(j, half, d, r));
        hi[r] = *reinterpret_cast<const uint32_t*>(tile + 16 * HD + v_of_run(j, half, d, 4 + r));
      }
      const uint2 ek = *reinterpret_cast<const uint2*>(tile + 32 * HD + j), ev = *reinterpret_cast<const uint2*>(tile + 32 * HD + 16 + j);
      auto scale = [&](const uint2& b, int r) { return pow2i((int)((r < 4 ? b.x : b.y) >> 8 * (r & 3) & 255) - 127); };
      transpose4(lo);
      transpose4(hi);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float f = scale(ek, 2 * r + half);
        decode4(c[r].x, f, x);
        decode4(c[r].y, f, x + 4);
        put(0, row + 2 * r + half, h, x);
        const float g = scale(ev, 4 * half + r);
        decode4(lo[r], g, x);
        decode4(hi[r], g, x + 4);
        put(1, row + 4 * half + r, h, x);
      }
    } else {
      uint2 c;
      if (half == 0) {
        c = *reinterpret_cast<const uint2*>(tile + k8_in_tile(j, d));
      } else {
        c = make_uint2(0, 0);
#pragma unroll
        for (int k = 0; k < 8; ++k) (k < 4 ? c.x : c.y) |= (uint32_t)tile[16 * HD + v8_in_tile(j, d + k)] << 8 * (k & 3);
      }
      const float f = pow2i((int)tile[32 * HD + 16 * half + j] - 127);
      decode4(c.x, f, x);
      decode4(c.y, f, x + 4);
      put(half, row, h, x);
    }
  }
  for (unsigned none = e.none; none; none &= none - 1) {  // rows without a place: zeros
    const float x[8] = {};
    for (int u = warp; u < mine; u += kWarps) {
      const int h = (blockIdx.y + u * per) * kHeads + sub;
      if (h < p.nkv) put(half, r0 + __ffs(none) - 1, h, x);
    }
  }
}

template <typename T, int HD>
void launch(const QuantParams& p, bool read, dim3 grid, cudaStream_t st) {
  if (read) read_quant_kernel<T, HD><<<grid, 32 * kWarps, 0, st>>>(p);
  else append_quant_kernel<T, HD><<<grid, 32 * kWarps, 0, st>>>(p);
}

int run(const char* name, const dflash_kv_pages* kv, int32_t dtype, QuantParams& p, int64_t ks, int64_t vs, bool read, dflash_stream stream) {
  auto refuse = [&](int code, const char* why) {
    char text[160];
    snprintf(text, sizeof text, "%s: %s", name, why);
    return call_error(code, text);
  };
  if (int rc = check_pages(kv, true)) return rc;
  if (kv->dtype != DFLASH_FP8E4M3_ROWEXP) return refuse(DFLASH_EINVAL, "pages must be e4m3 with row exponents");
  if (dtype != DFLASH_BF16 && dtype != DFLASH_F32) return refuse(DFLASH_EINVAL, "rows must be bf16 or f32");
  if (p.n < 0) return refuse(DFLASH_EINVAL, "n must be >= 0");
  if (p.n == 0) return DFLASH_OK;
  const void *k = read ? p.ko : p.k, *v = read ? p.vo : p.v;
  if (!k || !v || !p.slots) return refuse(DFLASH_EINVAL, "null pointer");
  const int es = dtype == DFLASH_F32 ? 4 : 2;
  const int64_t row = (int64_t)kv->n_kv_heads * kv->head_dim;
  if (ks < row || vs < row || ks > INT64_MAX / 8 || vs > INT64_MAX / 8 || (ks * es) % 16 || (vs * es) % 16 || !aligned16(k) || !aligned16(v))
    return refuse(DFLASH_EINVAL, "rows below n_kv_heads * head_dim, or k, v or a stride not whole 16 bytes");
  p.ks = ks * es, p.vs = vs * es;
  p.pool = static_cast<uint8_t*>(kv->pool), p.page_bytes = kv->page_stride;
  p.status = kv->status, p.nkv = kv->n_kv_heads, p.num_pages = kv->num_pages;
  int sms = 0;
  if (cudaError_t e = sm_count(&sms); e != cudaSuccess) return call_error(DFLASH_ECUDA, name, e);
  const int64_t blocks = (p.n + (int64_t)kRows - 1) / kRows;
  const int groups = (p.nkv + 128 / kv->head_dim - 1) / (128 / kv->head_dim);
  const dim3 grid((unsigned)blocks, (unsigned)std::min<int64_t>(groups, std::max<int64_t>(1, 16 * sms / blocks)));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == DFLASH_F32)
    kv->head_dim == 128 ? launch<float, 128>(p, read, grid, st) : launch<float, 64>(p, read, grid, st);
  else
    kv->head_dim == 128 ? launch<__nv_bfloat16, 128>(p, read, grid, st) : launch<__nv_bfloat16, 64>(p, read, grid, st);
  if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return call_error(DFLASH_ECUDA, name, e);
  return DFLASH_OK;
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" int dflash_append_kv_quant(const dflash_kv_pages* kv, int32_t src_dtype, const void* k, int64_t k_stride,
                                      const void* v, int64_t v_stride, const int32_t* slots, int32_t n,
                                      dflash_stream stream) {
  QuantParams p{};
  p.k = static_cast<const uint8_t*>(k), p.v = static_cast<const uint8_t*>(v), p.slots = slots, p.n = n;
  return run("append_kv_quant", kv, src_dtype, p, k_stride, v_stride, false, stream);
}

extern "C" int dflash_read_kv_quant(const dflash_kv_pages* kv, int32_t dst_dtype, const int32_t* slots, int32_t n, void* k,
                                    int64_t k_stride, void* v, int64_t v_stride, dflash_stream stream) {
  QuantParams p{};
  p.ko = static_cast<uint8_t*>(k), p.vo = static_cast<uint8_t*>(v), p.slots = slots, p.n = n;
  return run("read_kv_quant", kv, dst_dtype, p, k_stride, v_stride, true, stream);
}
