// Shared by the two forms of dflash_attend (serve_attend.cu: fp32 on the CUDA cores;
// serve_attend_tc.cu: bf16 on the tensor cores).
#pragma once

#include "serve.cuh"

namespace dflash {

struct AttendParams {
  const void* q;
  void* out;
  float* lse;
  const void* pool;
  const int32_t *page_tables, *kv_lens, *row_starts;
  uint32_t* status;
  int64_t q_stride, out_stride, page_stride;  // elements
  int nb, n_rows, mpps, num_pages, nh, nkv, window, causal;
  bool wide_out;     // rows of out start on 32 bytes
  float scale_log2;  // scale * log2(e): scores are exponents of 2
  int group, tokens; // query heads of a kv head; tokens of a tile of 128 rows
  unsigned inv;      // row / group = row * inv >> 16 for rows below 128
  // trees: masks of a sequence's rows over its rows (words of 64 bits each), positions; or NULL
  const unsigned long long* masks;
  const int32_t* positions;
  int words;
  bool quant;        // pages in 8 bits
};

// Workspace of the tensor-core form: split units' partials.
struct AttendWork {
  float* o;        // [2 sms][rows][head_dim] unnormalised O
  float2* ml;      // [2 sms][rows] (maximum in log2 units, sum)
  int4* meta;      // [sms] the unit that starts in a CTA and ends in a later one: (CTAs, its first row, tokens, g)
  int long_chunks; // many query tiles per sequence
  int spread;      // merge: rows before parts where that waits less
};

// Row r of partial slot `slot` (rows of fp32, as many as a unit of `rows` has): a warp merges a row,
// a row-per-thread writer stores whole sectors.
__device__ __forceinline__ float* part_row(const AttendWork& w, int slot, int r, int rows, int hd) {
  return w.o + ((int64_t)slot * rows + r) * hd;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Sequence s: its rows [*r0, *r0 + *n), key rows *kv.  false: no rows, or out of range (*bad).
template <bool kTree = false>
__device__ __forceinline__ bool seq_of(const AttendParams& p, int s, int* r0, int* n, int* kv, bool* bad) {
  const int a = __ldg(p.row_starts + s), b = __ldg(p.row_starts + s + 1), k = __ldg(p.kv_lens + s);
  *bad = a < 0 || b < a || b > p.n_rows || k < 0 || (long long)k > (long long)p.mpps * kPage ||
         (kTree && b - a > 64 * p.words);
  *r0 = a;
  *n = b - a;
  *kv = k;
  return !*bad && b > a;
}

int64_t attend_tc_workspace(int head_dim, int sms);
// The workspace's parts; long_chunks: many query tiles per sequence.
AttendWork attend_work(void* workspace, int head_dim, int sms, bool long_chunks);
// Merges the partials of split units (rows of p.tokens tokens, 128 rows a slot).
cudaError_t launch_attend_combine(const AttendParams& p, const AttendWork& w, int head_dim, int sms, cudaStream_t st);
// Pages in 8 bits, bf16 queries, at most 16 query heads of a kv head: units of 16 rows.
cudaError_t launch_attend8(const AttendParams& p, int head_dim, void* workspace, int sms, cudaStream_t st);
cudaError_t launch_attend_tc(const AttendParams& p, int head_dim, int max_new, void* workspace, int sms, cudaStream_t st);

}  // namespace dflash
