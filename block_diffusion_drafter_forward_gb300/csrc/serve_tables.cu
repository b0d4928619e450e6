// Page tables and row map of a step, and the copy of its K/V rows into the pages.
//
// extend_tables: two prefix sums over the sequences (pages needed, rows added), then one thread
// per row finds its sequence by binary search.  Bound by latency: a step of 1024 rows moves 14 KB and
// takes 5 us on the device.
// The scan is repeated by every CTA, so none waits for another before it maps its rows.  Lengths,
// pages held or a stack position written in place of the inputs have to wait until every CTA has read them:
// then the CTAs are one cluster (8 at most) with a barrier before the first CTA writes; else the
// rows spread over as many CTAs as they fill (134 Ki rows: 5.3 against 19.4 us in a cluster of 8).
#include <cooperative_groups.h>

#include <algorithm>
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
  int32_t* held;  // pages of each sequence, or NULL: those that its rows fill
  uint32_t* status;
  int nb, mpps, n_free, max_rows;
  bool in_place;
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
        const int filled = (ctx + kPage - 1) / kPage, held = p.held ? p.held[s] : filled;
        if (held < filled || held > p.mpps) {
          n = 0;
          bad = true;
        } else {
          need = max(0, (ctx + n + kPage - 1) / kPage - held);
        }
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
      const int pg = idx / kPage, held = p.held ? p.held[seq] : (ctx + kPage - 1) / kPage;
      int32_t* entry = p.page_tables + (int64_t)seq * p.mpps + pg;
      int page;
      if (pg >= held) {  // a new page: entered in the table by its first row
        page = p.free_pages[s_pg[seq] + pg - held];
        if (idx % kPage == 0) *entry = page;
      } else {
        page = *entry;
      }
      if (page >= 0 && page < (1 << 27)) slot = page * kPage + idx % kPage;
      else if (p.status) atomicOr(p.status, DFLASH_DEV_BAD_PAGE);
    }
    p.row_seq[i] = seq;
    p.row_index[i] = idx;
    p.slots[i] = slot;
  }
  if (p.in_place) cg::this_cluster().sync();  // every CTA has read the inputs
  else __syncthreads();
  if (rank == 0) {
    for (int s = t; s <= p.nb; s += kTabThreads) {
      p.row_starts[s] = s_row[s];
      if (s == p.nb) continue;
      const int n = s_row[s + 1] - s_row[s];
      if (p.held && n > 0) p.held[s] = max(p.held[s], (s_ctx[s] + n + kPage - 1) / kPage);
      p.kv_lens[s] = s_ctx[s] + n;
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
  int n, nkv, num_pages, heads;
  bool wide;  // tiles start on 32 bytes
};

// A block takes kRows consecutive rows and one head, or four where there are rows enough to fill
// the SMs with fewer blocks (1024 rows of 4 heads: 7.3 us by fours, 4.3 by ones; 16.7 Ki rows of 8
// heads: 30.8 us by fours, 4.5 TB/s, 32.0 by ones); a warp one entry of one head at a time.
// An entry is a run of eight rows whose slots fill one half page in order (the usual case: a
// step's rows of a sequence follow one another), or a single row.  In the tile eight keys of a
// half page lie side by side, so a run is written in whole sectors: K by lanes of 8 rows x 4
// pieces (64 contiguous bytes read per row, 128 written), V transposed in registers (a lane
// reads two dims of the eight rows and writes both dims' eight keys).  A single row writes V
// element by element.  Bound by HBM, both ways once.
constexpr int kRows = 16;

template <typename T>
__device__ __forceinline__ void copy16(T* d, const T* s) {
  *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(s);
}
__device__ __forceinline__ void put_keys(__nv_bfloat16* d, const uint32_t (&r)[8], bool wide) {  // dims x, x + 1 of 8 keys
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = __byte_perm(r[2 * i], r[2 * i + 1], 0x5410);
    w[4 + i] = __byte_perm(r[2 * i], r[2 * i + 1], 0x7632);
  }
  put32(d, w, wide);
}
__device__ __forceinline__ void put_keys(float* d, const uint2 (&r)[8], bool wide) {
  const uint32_t x[8] = {r[0].x, r[1].x, r[2].x, r[3].x, r[4].x, r[5].x, r[6].x, r[7].x};
  const uint32_t y[8] = {r[0].y, r[1].y, r[2].y, r[3].y, r[4].y, r[5].y, r[6].y, r[7].y};
  put32(d, x, wide);
  put32(d + 8, y, wide);
}
template <typename T> struct Two;  // two dims of a row
template <> struct Two<__nv_bfloat16> { using type = uint32_t; };
template <> struct Two<float> { using type = uint2; };

template <typename T, int HD>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
  using T2 = typename Two<T>::type;
  __shared__ int s_slot[kRows + 14], s_entry[kRows], s_n;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int r0 = blockIdx.x * kRows;
  if (t < kRows + 14) {  // the rows here, and seven on either side that a run may reach
    const int r = r0 - 7 + t;
    s_slot[t] = r >= 0 && r < p.n ? p.slots[r] : -1;
  }
  if (t == 0) s_n = 0;
  __syncthreads();
  if (t < 32) {
    bool take = false, run = false;
    if (t < kRows) {
      const int slot = s_slot[7 + t];
      if (slot >= 0 && slot / kPage >= p.num_pages) {
        if (p.status && blockIdx.y == 0) atomicOr(p.status, DFLASH_DEV_BAD_PAGE);
      } else if (slot >= 0) {
        const int o = slot & 7, first = 7 + t - o;  // a row's run is decided alike in every block that sees it
        run = true;
        for (int k = 0; k < 8; ++k) run = run && s_slot[first + k] == slot - o + k;
        take = !run || o == 0;  // a run belongs to the block of its first row
      }
    }
    const unsigned m = __ballot_sync(0xffffffffu, take);
    if (take) s_entry[__popc(m & ((1u << t) - 1))] = t | (run ? 64 : 0);
    if (t == 0) s_n = __popc(m);
  }
  __syncthreads();
  const int h = blockIdx.y * p.heads + warp % p.heads;
  if (h >= p.nkv) return;
  constexpr int kPer = 16 / sizeof(T);  // dims of a 16-byte piece
  for (int e = warp / p.heads; e < s_n; e += 8 / p.heads) {
    const int i = s_entry[e] & 63, slot = s_slot[7 + i];
    const int64_t row = r0 + i;
    T* tile = reinterpret_cast<T*>(p.pool + (slot / kPage) * p.page_bytes) + (int64_t)h * 2 * kPage * HD;
    const int j = slot % kPage;
    const T* k = reinterpret_cast<const T*>(p.k + row * p.ks) + h * HD;
    const T* v = reinterpret_cast<const T*>(p.v + row * p.vs) + h * HD;
    if (s_entry[e] & 64) {
      const T* kr = reinterpret_cast<const T*>(reinterpret_cast<const uint8_t*>(k) + (lane & 7) * p.ks);
      uint4 kk[HD / kPer / 4];
      T2 vv[HD / 64][8];
#pragma unroll
      for (int c = 0; c < HD / kPer / 4; ++c) kk[c] = *reinterpret_cast<const uint4*>(kr + (c * 4 + (lane >> 3)) * kPer);
#pragma unroll
      for (int c = 0; c < HD / 64; ++c) {
#pragma unroll
        for (int x = 0; x < 8; ++x)
          vv[c][x] = *reinterpret_cast<const T2*>(
              reinterpret_cast<const T*>(reinterpret_cast<const uint8_t*>(v) + x * p.vs) + c * 64 + 2 * lane);
      }
#pragma unroll
      for (int c = 0; c < HD / kPer / 4; ++c)
        *reinterpret_cast<uint4*>(tile + k_in_tile(j + (lane & 7), (c * 4 + (lane >> 3)) * kPer, HD)) = kk[c];
#pragma unroll
      for (int c = 0; c < HD / 64; ++c) put_keys(tile + kPage * HD + v_in_tile(j, c * 64 + 2 * lane, HD), vv[c], p.wide);
    } else {
#pragma unroll
      for (int c = lane; c < HD / kPer; c += 32) copy16(tile + k_in_tile(j, c * kPer, HD), k + c * kPer);
#pragma unroll
      for (int d = lane; d < HD; d += 32) tile[kPage * HD + v_in_tile(j, d, HD)] = v[d];
    }
  }
}

__global__ void take_status_kernel(uint32_t* status, uint32_t* flags) { *flags = atomicExch(status, 0u); }

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" int dflash_take_status(uint32_t* status, uint32_t* flags, dflash_stream stream) {
  if (!status || !flags) return call_error(DFLASH_EINVAL, "take_status: null pointer");
  take_status_kernel<<<1, 1, 0, reinterpret_cast<cudaStream_t>(stream)>>>(status, flags);
  if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return call_error(DFLASH_ECUDA, "take_status", e);
  return DFLASH_OK;
}

extern "C" int dflash_extend_tables(const int32_t* ctx_lens, const int32_t* new_rows, int32_t nb,
                                    int32_t* page_tables, int32_t max_pages_per_seq, const int32_t* free_pages,
                                    int32_t n_free, const int32_t* free_begin, int32_t* free_end, int32_t* kv_lens,
                                    int32_t* row_starts, int32_t* row_seq, int32_t* row_index, int32_t* slots,
                                    int32_t max_rows, uint32_t* status, dflash_stream stream) {
  return dflash_extend_tables_ex(ctx_lens, new_rows, nb, page_tables, max_pages_per_seq, free_pages, n_free, free_begin,
                                 free_end, kv_lens, row_starts, row_seq, row_index, slots, max_rows, nullptr, status, stream);
}

extern "C" int dflash_extend_tables_ex(const int32_t* ctx_lens, const int32_t* new_rows, int32_t nb,
                                       int32_t* page_tables, int32_t max_pages_per_seq, const int32_t* free_pages,
                                       int32_t n_free, const int32_t* free_begin, int32_t* free_end, int32_t* kv_lens,
                                       int32_t* row_starts, int32_t* row_seq, int32_t* row_index, int32_t* slots,
                                       int32_t max_rows, int32_t* held_pages, uint32_t* status, dflash_stream stream) {
  if (!ctx_lens || !new_rows || !page_tables || !free_pages || !free_begin || !free_end || !kv_lens || !row_starts ||
      !row_seq || !row_index || !slots)
    return call_error(DFLASH_EINVAL, "extend_tables: null pointer");
  if (nb < 1 || n_free < 0 || max_rows < 0) return call_error(DFLASH_EINVAL, "extend_tables: nb >= 1, n_free >= 0 and max_rows >= 0");
  if (max_pages_per_seq < 1 || max_pages_per_seq >= 1 << 27)
    return call_error(DFLASH_EINVAL, "extend_tables: max_pages_per_seq must be in [1, 2^27)");
  if (nb > kTabMaxSeqs) return call_error(DFLASH_ECAPACITY, "extend_tables: nb above 16384");
  if (max_rows > 1 << 30) return call_error(DFLASH_ECAPACITY, "extend_tables: max_rows above 2^30");
  TablesParams p{ctx_lens, new_rows, free_pages, free_begin, page_tables, free_end, kv_lens, row_starts,
                 row_seq,  row_index, slots, held_pages, status, nb, max_pages_per_seq, n_free, max_rows, false};
  const int smem = (3 * nb + 1) * (int)sizeof(int32_t);
  static std::atomic<unsigned long long> attr{0};
  if (cudaError_t e = smem_attr_once(extend_tables_kernel, (3 * kTabMaxSeqs + 1) * (int)sizeof(int32_t), attr); e != cudaSuccess)
    return call_error(DFLASH_ECUDA, "extend_tables", e);
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute a[1];
  auto overlap = [](const int32_t* a, int64_t n, const int32_t* b, int64_t m) { return a < b + m && b < a + n; };
  p.in_place = held_pages || free_end == free_begin || overlap(kv_lens, nb, ctx_lens, nb);
  int sms = 0;
  if (cudaError_t e = sm_count(&sms); e != cudaSuccess) return call_error(DFLASH_ECUDA, "extend_tables", e);
  const int fill = std::max(1, (max_rows + kTabThreads - 1) / kTabThreads);
  const int ctas = p.in_place ? (max_rows > 4096 ? 8 : 1) : std::min(fill, sms);
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = p.in_place ? ctas : 1;
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
                 static_cast<uint8_t*>(kv->pool), kv->page_stride * es, slots, kv->status, n, kv->n_kv_heads, kv->num_pages, 4,
                 reinterpret_cast<uintptr_t>(kv->pool) % 32 == 0 && (kv->page_stride * es) % 32 == 0};
  int sms = 0;
  if (cudaError_t e = sm_count(&sms); e != cudaSuccess) return call_error(DFLASH_ECUDA, "append_kv", e);
  const int64_t groups = (n + (int64_t)kRows - 1) / kRows;
  p.heads = groups * ((kv->n_kv_heads + 3) / 4) < 4 * sms ? 1 : 4;
  const dim3 grid((unsigned)groups, (unsigned)((kv->n_kv_heads + p.heads - 1) / p.heads));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool f32 = kv->dtype == DFLASH_F32, w = kv->head_dim == 128;
  auto kern = f32 ? (w ? append_kernel<float, 128> : append_kernel<float, 64>)
                  : (w ? append_kernel<__nv_bfloat16, 128> : append_kernel<__nv_bfloat16, 64>);
  kern<<<grid, 256, 0, st>>>(p);
  if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return call_error(DFLASH_ECUDA, "append_kv", e);
  return DFLASH_OK;
}
