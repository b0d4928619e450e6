// Page tables and row map of a step, and the copy of its K/V rows into the pages.
//
// extend_tables: two prefix sums over the sequences (pages needed, rows added), then one thread
// per row finds its sequence by binary search.  Bound by latency: a step of 1024 rows moves 14 KB.
// The scan is repeated by every CTA of the one cluster that runs it, so no CTA waits for another
// before it maps its rows; the cluster barrier at the end lets the lengths and the stack position
// be written in place of the inputs.
#include <cooperative_groups.h>

#include <atomic>

#include "launch_util.cuh"
#include "serve.cuh"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

constexpr int kTabThreads = 1024;
constexpr int kTabMaxSeqs = 16384;

struct TablesParams {
  const int32_t *ctx_lens, *new_rows, *free_pages, *free_begin;
  int32_t *page_tables, *free_end, *kv_lens, *row_starts, *row_seq, *row_index, *slots;
  uint32_t* status;
  int nb, mpps, n_free, max_rows;
};

__global__ void __launch_bounds__(kTabThreads) extend_tables_kernel(const TablesParams p) {
  extern __shared__ int32_t sm[];
  int32_t* s_row = sm;                // [nb + 1] first row of each sequence
  int32_t* s_ctx = s_row + p.nb + 1;  // [nb] rows held
  int32_t* s_pg = s_ctx + p.nb;       // [nb] position in the stack of its first new page
  __shared__ long long s_sum[2][kTabThreads / 32];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const unsigned rank = blockIdx.x, nctas = gridDim.x;
  const long long begin = *p.free_begin;
  const bool begin_ok = begin >= 0;
  long long rows0 = 0, pages0 = 0;    // sums over the sequences before this tile
  int granted_rows = 0, granted_pages = 0;
  bool no_room = false, bad = false;
  for (int s0 = 0; s0 < p.nb; s0 += kTabThreads) {
    const int s = s0 + t;
    int ctx = 0, n = 0, need = 0;
    if (s < p.nb) {
      ctx = p.ctx_lens[s];
      n = p.new_rows[s];
      if (ctx < 0 || n < 0 || (long long)ctx + n > (long long)p.mpps * kPage) {
        n = 0;
        bad = true;
      } else {
        need = (ctx + n + kPage - 1) / kPage - (ctx + kPage - 1) / kPage;
      }
    }
    long long r = n, g = need;  // inclusive sums: warp, then across warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, r, o), b = __shfl_up_sync(0xffffffffu, g, o);
      if (lane >= o) r += a, g += b;
    }
    if (lane == 31) s_sum[0][warp] = r, s_sum[1][warp] = g;
    __syncthreads();
    if (warp == 0) {
      long long a = s_sum[0][lane], b = s_sum[1][lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long c = __shfl_up_sync(0xffffffffu, a, o), d = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) a += c, b += d;
      }
      s_sum[0][lane] = a, s_sum[1][lane] = b;
    }
    __syncthreads();
    r += rows0 + (warp ? s_sum[0][warp - 1] : 0);
    g += pages0 + (warp ? s_sum[1][warp - 1] : 0);
    rows0 += s_sum[0][kTabThreads / 32 - 1];
    pages0 += s_sum[1][kTabThreads / 32 - 1];
    // both sums never fall, so the sequences that fit are a prefix of the batch
    const bool fits = begin_ok && begin + g <= p.n_free && r <= p.max_rows;
    if (s < p.nb) {
      s_ctx[s] = ctx;
      s_row[s] = fits ? (int)(r - n) : -1;
      s_pg[s] = fits ? (int)(begin + g - need) : 0;
      no_room |= !fits;
    }
    // the totals granted: the last sequence that fits has the largest
    const int gr = __reduce_max_sync(0xffffffffu, fits && s < p.nb ? (int)r : 0);
    const int gp = __reduce_max_sync(0xffffffffu, fits && s < p.nb ? (int)g : 0);
    __syncthreads();  // every thread has read s_sum
    if (lane == 0) s_sum[0][warp] = gr, s_sum[1][warp] = gp;
    __syncthreads();
    for (int w = 0; w < kTabThreads / 32; ++w) {
      granted_rows = max(granted_rows, (int)s_sum[0][w]);
      granted_pages = max(granted_pages, (int)s_sum[1][w]);
    }
    __syncthreads();
  }
  // sequences past the last that fits start (and end) at the total
  for (int s = t; s < p.nb; s += kTabThreads)
    if (s_row[s] < 0) s_row[s] = granted_rows;
  if (t == 0) s_row[p.nb] = granted_rows;
  __syncthreads();

  for (int i = rank * kTabThreads + t; i < p.max_rows; i += nctas * kTabThreads) {
    int seq = -1, idx = -1, slot = -1;
    if (i < granted_rows) {
      int lo = 0, hi = p.nb;  // the last sequence whose first row is <= i
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_row[mid] <= i) lo = mid; else hi = mid;
      }
      seq = lo;
      const int ctx = s_ctx[seq];
      idx = ctx + i - s_row[seq];
      const int pg = idx / kPage, held = (ctx + kPage - 1) / kPage;
      int32_t* entry = p.page_tables + (int64_t)seq * p.mpps + pg;
      int page;
      if (pg >= held) {  // a new page: entered in the table by its first row
        page = p.free_pages[s_pg[seq] + pg - held];
        if (idx % kPage == 0) *entry = page;
      } else {
        page = *entry;
      }
      slot = page >= 0 && page < (1 << 27) ? page * kPage + idx % kPage : -1;
    }
    p.row_seq[i] = seq;
    p.row_index[i] = idx;
    p.slots[i] = slot;
  }
  if (nctas > 1) cg::this_cluster().sync();  // every CTA has read the inputs
  else __syncthreads();
  if (rank == 0) {
    for (int s = t; s <= p.nb; s += kTabThreads) {
      p.row_starts[s] = s_row[s];
      if (s < p.nb) p.kv_lens[s] = s_ctx[s] + s_row[s + 1] - s_row[s];
    }
    if (t == 0) *p.free_end = (int)begin + granted_pages;
    if (p.status && (bad || no_room)) atomicOr(p.status, (bad ? DFLASH_DEV_BAD_CTX : 0u) | (no_room ? DFLASH_DEV_NO_ROOM : 0u));
  }
}

struct AppendParams {
  const uint8_t *k, *v;
  int64_t ks, vs;  // bytes between rows
  uint8_t* pool;
  int64_t page_bytes;
  const int32_t* slots;
  uint32_t* status;
  int n, nkv, num_pages;
};

// Row r, head h, dims 8 c .. 8 c + 7 of K and V: one thread each.
template <typename T, int HD>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
  constexpr int kC = HD / 8;
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int c = (int)(x % kC), h = (int)(x / kC % p.nkv);
  const int64_t r = x / kC / p.nkv;
  if (r >= p.n) return;
  const int slot = p.slots[r];
  if (slot < 0) return;
  const int page = slot / kPage, j = slot % kPage;
  if (page >= p.num_pages) {
    if (p.status && c == 0 && h == 0) atomicOr(p.status, DFLASH_DEV_BAD_PAGE);
    return;
  }
  T* tile = reinterpret_cast<T*>(p.pool + page * p.page_bytes) + (int64_t)h * 2 * kPage * HD;
  const T* k = reinterpret_cast<const T*>(p.k + r * p.ks) + h * HD + c * 8;
  const T* v = reinterpret_cast<const T*>(p.v + r * p.vs) + h * HD + c * 8;
  for (int e = 0; e < 8; ++e) {
    tile[k_in_tile(j, c * 8 + e, HD)] = k[e];
    tile[kPage * HD + v_in_tile(j, c * 8 + e, HD)] = v[e];
  }
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" int dflash_extend_tables(const int32_t* ctx_lens, const int32_t* new_rows, int32_t nb,
                                    int32_t* page_tables, int32_t max_pages_per_seq, const int32_t* free_pages,
                                    int32_t n_free, const int32_t* free_begin, int32_t* free_end, int32_t* kv_lens,
                                    int32_t* row_starts, int32_t* row_seq, int32_t* row_index, int32_t* slots,
                                    int32_t max_rows, uint32_t* status, dflash_stream stream) {
  if (!ctx_lens || !new_rows || !page_tables || !free_pages || !free_begin || !free_end || !kv_lens || !row_starts ||
      !row_seq || !row_index || !slots)
    return call_error(DFLASH_EINVAL, "extend_tables: null pointer");
  if (nb < 1 || n_free < 0 || max_rows < 0) return call_error(DFLASH_EINVAL, "extend_tables: nb >= 1, n_free >= 0 and max_rows >= 0");
  if (max_pages_per_seq < 1 || max_pages_per_seq >= 1 << 27)
    return call_error(DFLASH_EINVAL, "extend_tables: max_pages_per_seq must be in [1, 2^27)");
  if (nb > kTabMaxSeqs) return call_error(DFLASH_ECAPACITY, "extend_tables: nb above 16384");
  if (max_rows > 1 << 30) return call_error(DFLASH_ECAPACITY, "extend_tables: max_rows above 2^30");
  TablesParams p{ctx_lens, new_rows, free_pages, free_begin, page_tables, free_end, kv_lens, row_starts,
                 row_seq,  row_index, slots, status, nb, max_pages_per_seq, n_free, max_rows};
  const int smem = (3 * nb + 1) * (int)sizeof(int32_t);
  static std::atomic<unsigned long long> attr{0};
  if (cudaError_t e = smem_attr_once(extend_tables_kernel, (3 * kTabMaxSeqs + 1) * (int)sizeof(int32_t), attr); e != cudaSuccess)
    return call_error(DFLASH_ECUDA, "extend_tables", e);
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute a[1];
  const int ctas = max_rows > 4096 ? 8 : 1;
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = ctas;
  a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
  c.gridDim = dim3(ctas);
  c.blockDim = dim3(kTabThreads);
  c.dynamicSmemBytes = smem;
  c.stream = reinterpret_cast<cudaStream_t>(stream);
  c.attrs = a;
  c.numAttrs = 1;
  if (cudaError_t e = cudaLaunchKernelEx(&c, extend_tables_kernel, p); e != cudaSuccess)
    return call_error(DFLASH_ECUDA, "extend_tables", e);
  return DFLASH_OK;
}

extern "C" int dflash_append_kv(const dflash_kv_pages* kv, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, const int32_t* slots, int32_t n, dflash_stream stream) {
  if (int rc = check_pages(kv)) return rc;
  if (n < 0) return call_error(DFLASH_EINVAL, "append_kv: n must be >= 0");
  if (n == 0) return DFLASH_OK;
  if (!k || !v || !slots) return call_error(DFLASH_EINVAL, "append_kv: null pointer");
  const int es = kv->dtype == DFLASH_F32 ? 4 : 2, row = kv->n_kv_heads * kv->head_dim;
  if (k_stride < row || v_stride < row || (k_stride * es) % 16 || (v_stride * es) % 16 || !aligned16(k) || !aligned16(v))
    return call_error(DFLASH_EINVAL, "append_kv: rows below n_kv_heads * head_dim, or k, v or a stride not whole 16 bytes");
  AppendParams p{static_cast<const uint8_t*>(k), static_cast<const uint8_t*>(v), k_stride * es, v_stride * es,
                 static_cast<uint8_t*>(kv->pool), kv->page_stride * es, slots, kv->status, n, kv->n_kv_heads, kv->num_pages};
  const int64_t items = (int64_t)n * row / 8, blocks = (items + 255) / 256;
  if (blocks > 0x7fffffff) return call_error(DFLASH_ECAPACITY, "append_kv: too many rows for one call");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = kv->dtype == DFLASH_F32, w = kv->head_dim == 128;
  auto kern = f32 ? (w ? append_kernel<float, 128> : append_kernel<float, 64>)
                  : (w ? append_kernel<__nv_bfloat16, 128> : append_kernel<__nv_bfloat16, 64>);
  kern<<<(unsigned)blocks, 256, 0, st>>>(p);
  if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return call_error(DFLASH_ECUDA, "append_kv", e);
  return DFLASH_OK;
}
