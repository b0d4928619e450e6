// Attention of a chunk of new tokens per sequence over its paged K/V rows (dflash_attend): the C
// entries, and the fp32 form on the CUDA cores (as the fp32 drafter's path).  The bf16 form is
// serve_attend_tc.cu.
#include <float.h>

#include "launch_util.cuh"
#include "serve_attend.cuh"

namespace dflash {
namespace {

__device__ __forceinline__ int page_id(const AttendParams& p, int s, int lp) {
  const int page = __ldg(p.page_tables + (int64_t)s * p.mpps + lp);
  if (page >= 0 && page < p.num_pages) return page;
  if (p.status) atomicOr(p.status, DFLASH_DEV_BAD_PAGE);
  return 0;
}

// CUDA-core form: one warp per (row, query head), online softmax over pages of 16 keys.  Lane l
// takes key l % 16 and one half of the dims of q . k, and dims l, l + 32, ... of the output.
template <int HD>
__global__ void __launch_bounds__(128) attend_simple_kernel(const AttendParams p) {
  __shared__ float s_q[4][HD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && p.status) {  // every sequence is checked, also those that no row leads to
    for (int s = threadIdx.x; s < p.nb; s += blockDim.x) {
      int r0, n, kv;
      bool bad;
      seq_of(p, s, &r0, &n, &kv, &bad);
      if (bad) atomicOr(p.status, DFLASH_DEV_BAD_CTX);
    }
  }
  const int64_t x = (int64_t)blockIdx.x * 4 + warp;
  const int i = (int)(x / p.nh), h = (int)(x % p.nh), g = h / (p.nh / p.nkv);
  if (i >= p.n_rows) return;
  int lo = 0, hi = p.nb;  // the last sequence that starts at or before row i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.row_starts + mid) <= i) lo = mid; else hi = mid;
  }
  const int s = lo;
  int r0, n, kv;
  bool bad;
  const bool rows = seq_of(p, s, &r0, &n, &kv, &bad);
  if (!rows || i < r0 || i >= r0 + n) return;
  const float* q = static_cast<const float*>(p.q) + i * p.q_stride + h * HD;
#pragma unroll
  for (int e = 0; e < HD / 32; ++e) s_q[warp][lane + 32 * e] = q[lane + 32 * e] * p.scale_log2;
  __syncwarp();
  const int pos = kv - n + (i - r0);
  const int k_end = p.causal ? min(kv, pos + 1) : kv;
  const int k_begin = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  float m = -INFINITY, l = 0.f, acc[HD / 32];
#pragma unroll
  for (int e = 0; e < HD / 32; ++e) acc[e] = 0.f;
  const int half = lane >> 4, j = lane & 15;
  for (int lp = k_begin / kPage; lp * kPage < k_end; ++lp) {
    const float* tile = static_cast<const float*>(p.pool) + page_id(p, s, lp) * p.page_stride + (int64_t)g * 2 * kPage * HD;
    float sc = 0.f;
#pragma unroll
    for (int c = 0; c < HD / 16; ++c) {
      const int d8 = half * (HD / 16) + c;
      const float* k = tile + k_in_tile(j, d8 * 8, HD);
#pragma unroll
      for (int e = 0; e < 8; ++e) sc = fmaf(s_q[warp][d8 * 8 + e], k[e], sc);
    }
    sc += __shfl_xor_sync(0xffffffffu, sc, 16);
    const int key = lp * kPage + j;
    const bool see = key >= k_begin && key < k_end;
    sc = see ? sc : -INFINITY;
    float mx = sc;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float m_new = fmaxf(m, mx);
    const float base = m_new == -INFINITY ? 0.f : m_new;
    const float alpha = exp2f(m - base), pr = see ? exp2f(sc - base) : 0.f;
    float sum = pr;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * alpha + sum;
    m = m_new;
#pragma unroll
    for (int e = 0; e < HD / 32; ++e) acc[e] *= alpha;
    const float* v = tile + kPage * HD;
    for (int jj = max(0, k_begin - lp * kPage); jj < min(kPage, k_end - lp * kPage); ++jj) {  // seen keys only
      const float w = __shfl_sync(0xffffffffu, pr, jj);
#pragma unroll
      for (int e = 0; e < HD / 32; ++e) acc[e] = fmaf(w, v[v_in_tile(jj, lane + 32 * e, HD)], acc[e]);
    }
  }
  float* out = static_cast<float*>(p.out) + i * p.out_stride + h * HD;
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
  for (int e = 0; e < HD / 32; ++e) out[lane + 32 * e] = acc[e] * inv;
  if (p.lse && lane == 0) p.lse[(int64_t)i * p.nh + h] = lse_of(m, l);
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" int64_t dflash_attend_workspace(const dflash_kv_pages* kv) {
  if (int rc = check_pages(kv)) return rc;
  if (kv->dtype == DFLASH_F32) return 0;
  int sms = 0;
  if (cudaError_t e = sm_count(&sms); e != cudaSuccess) return call_error(DFLASH_ECUDA, "attend_workspace", e);
  return attend_tc_workspace(kv->head_dim, sms);
}

extern "C" int dflash_attend(const dflash_kv_pages* kv, const void* q, int64_t q_stride, const int32_t* page_tables,
                             int32_t max_pages_per_seq, const int32_t* kv_lens, const int32_t* row_starts, int32_t nb,
                             int32_t n_rows, int32_t max_new, int32_t n_q_heads, float scale, int32_t window,
                             int32_t causal, void* out, int64_t out_stride, float* lse, void* workspace,
                             int64_t workspace_bytes, dflash_stream stream) {
  if (int rc = check_pages(kv)) return rc;
  if (nb < 1 || n_rows < 0 || max_new < 0) return call_error(DFLASH_EINVAL, "attend: nb >= 1, n_rows >= 0 and max_new >= 0");
  if (nb > 16384 || n_rows > 1 << 30) return call_error(DFLASH_ECAPACITY, "attend: nb above 16384 or n_rows above 2^30");
  if (max_pages_per_seq < 1 || max_pages_per_seq >= 1 << 26)  // key indices stay below 2^30
    return call_error(DFLASH_EINVAL, "attend: max_pages_per_seq must be in [1, 2^26)");
  if (n_q_heads < 1 || n_q_heads % kv->n_kv_heads || n_q_heads / kv->n_kv_heads > 128)
    return call_error(DFLASH_EINVAL, "attend: n_q_heads must be a multiple of n_kv_heads, at most 128 times it");
  if (window < 0) return call_error(DFLASH_EINVAL, "attend: window must be >= 0");
  if (!(scale > 0.f) || !(scale <= FLT_MAX)) return call_error(DFLASH_EINVAL, "attend: scale must be positive and finite");
  if (n_rows == 0) return DFLASH_OK;
  if (!q || !out || !page_tables || !kv_lens || !row_starts) return call_error(DFLASH_EINVAL, "attend: null pointer");
  const int es = kv->dtype == DFLASH_F32 ? 4 : 2;
  const int64_t row = (int64_t)n_q_heads * kv->head_dim;
  if (q_stride < row || out_stride < row || (q_stride * es) % 16 || (out_stride * es) % 16 || !aligned16(q) || !aligned16(out))
    return call_error(DFLASH_EINVAL, "attend: rows below n_q_heads * head_dim, or q, out or a stride not whole 16 bytes");
  const int64_t need = dflash_attend_workspace(kv);
  if (need < 0) return (int)need;
  if (workspace_bytes < need || (need > 0 && (!workspace || !aligned16(workspace))))
    return call_error(DFLASH_EINVAL, "attend: workspace below dflash_attend_workspace() bytes, or not 16-byte aligned");
  if (window >= 1 << 30) window = 0;  // longer than any sequence; positions less the window stay in 32 bits
  AttendParams p{q, out, lse, kv->pool, page_tables, kv_lens, row_starts, kv->status, q_stride, out_stride, kv->page_stride,
                 nb, n_rows, max_pages_per_seq, kv->num_pages, n_q_heads, kv->n_kv_heads, window, causal != 0,
                 reinterpret_cast<uintptr_t>(out) % 32 == 0 && (out_stride * es) % 32 == 0, scale * 1.4426950408889634f};
  p.group = n_q_heads / kv->n_kv_heads;
  p.tokens = 128 / p.group;
  p.inv = (65536 + p.group - 1) / p.group;  // (exact: 127 (inv group - 65536) < 65536)
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (kv->dtype == DFLASH_BF16) {
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e == cudaSuccess) e = launch_attend_tc(p, kv->head_dim, max_new, workspace, sms, st);
    return e == cudaSuccess ? DFLASH_OK : call_error(DFLASH_ECUDA, "attend", e);
  }
  const int64_t blocks = ((int64_t)n_rows * n_q_heads + 3) / 4;
  if (blocks > 0x7fffffff) return call_error(DFLASH_ECAPACITY, "attend: too many rows for one call");
  if (kv->head_dim == 128)
    attend_simple_kernel<128><<<(unsigned)blocks, 128, 0, st>>>(p);
  else
    attend_simple_kernel<64><<<(unsigned)blocks, 128, 0, st>>>(p);
  if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return call_error(DFLASH_ECUDA, "attend", e);
  return DFLASH_OK;
}
