// Trees of drafted tokens: positions and masks of a batch of them (dflash_draft_tree), and the move
// of an accepted branch's rows (dflash_keep_rows).
#include <algorithm>
#include <type_traits>

#include "launch_util.cuh"
#include "serve.cuh"

namespace dflash {
namespace {

constexpr int kMaxNodes = 512, kMaxWords = kMaxNodes / 64;

// A block per sequence, a thread per node (64 for every word of the masks).  Ancestors by pointer jumping: with A_i the
// node and the ancestors seen so far and J_i the first one not seen, A_i |= A_{J_i} and J_i = J_{J_i} double
// them, so log2(depth) rounds do.  Bound by latency: a round is one pass through shared memory and two
// barriers (a tree of 32 nodes 3.0 us, 32 trees of 33-64 3.7; with 512 threads whatever the masks 6.5).
// Blocks from nb on empty the rows outside the sequences.
__global__ void __launch_bounds__(kMaxNodes) draft_tree_kernel(const int32_t* parents, const int32_t* kv_lens,
                                                                  const int32_t* row_starts, int nb, int n_rows, int words,
                                                                  int32_t* positions, unsigned long long* masks,
                                                                  uint32_t* status) {
  __shared__ unsigned long long s_anc[kMaxNodes * kMaxWords];  // [word][node]
  __shared__ int s_jump[kMaxNodes];
  const int t = threadIdx.x, s = blockIdx.x;
  auto clear = [&](int64_t row) {
    positions[row] = -1;
    for (int w = 0; w < words; ++w) masks[row * words + w] = 0;
  };
  if (s >= nb) {
    const int lo = min(max(row_starts[0], 0), n_rows), hi = min(max(row_starts[nb], lo), n_rows);
    const int64_t n = (int64_t)lo + (n_rows - hi), step = (int64_t)(gridDim.x - nb) * blockDim.x;
    for (int64_t i = (int64_t)(s - nb) * blockDim.x + t; i < n; i += step) clear(i < lo ? i : hi + (i - lo));
    return;
  }
  const int r0 = row_starts[s], r1 = row_starts[s + 1], kv = kv_lens[s];
  const bool out = r0 < 0 || r1 < r0 || r1 > n_rows;
  const int n = out ? 0 : r1 - r0;
  const bool bad = out || kv < n, wide = !out && n > 64 * words;
  if (bad || wide) {
    if (t == 0 && status) atomicOr(status, (bad ? DFLASH_DEV_BAD_CTX : 0u) | (wide ? DFLASH_DEV_BAD_TREE : 0u));
    for (int i = t; i < n; i += blockDim.x) clear(r0 + i);
    return;
  }
  unsigned long long anc[kMaxWords];
  int jump = -1;
  if (t < n) {
    jump = parents[r0 + t];
    if (jump < -1 || jump >= t) {
      jump = -1;
      if (status) atomicOr(status, DFLASH_DEV_BAD_TREE);
    }
  }
#pragma unroll
  for (int w = 0; w < kMaxWords; ++w) anc[w] = w == t >> 6 && t < n ? 1ull << (t & 63) : 0ull;
  for (;;) {
    if (t < n) {
      s_jump[t] = jump;
#pragma unroll
      for (int w = 0; w < kMaxWords; ++w)
        if (w < words) s_anc[w * kMaxNodes + t] = anc[w];
    }
    if (!__syncthreads_or(jump >= 0)) break;
    if (jump >= 0) {
#pragma unroll
      for (int w = 0; w < kMaxWords; ++w)
        if (w < words) anc[w] |= s_anc[w * kMaxNodes + jump];
      jump = s_jump[jump];
    }
    __syncthreads();  // read before the next round's writes
  }
  if (t < n) {
    int depth = -1;
#pragma unroll
    for (int w = 0; w < kMaxWords; ++w) {
      depth += __popcll(anc[w]);
      if (w < words) masks[(int64_t)(r0 + t) * words + w] = anc[w];
    }
    positions[r0 + t] = kv - n + depth;
  }
}

struct KeepParams {
  uint8_t* pool;
  int64_t page_bytes, head_bytes;
  const int32_t *page_tables, *ctx_lens, *path, *path_lens;
  uint32_t* status;
  int nb, nkv, mpps, num_pages, max_path, hd;
};

// A warp has one (sequence, head) and takes the rows in order of their new places, a half page (eight rows, or what
// of them the path fills) at a time: all loads of a half page ahead of its stores.  Since the path rises, row i of it
// is read at or behind i, and no row is written before it has been read; a lane reads and writes the same dims,
// so that its own program order is enough.  V of a whole half page is stored eight rows of a dim at once:
// row by row every element is a sector of its own (256 trees, 8 heads of 128: 18.1 us, row by row 25).  Bound by
// latency (a half page is one round trip; one tree 4.7 us) and by V's gathered elements.  (K and halves of V in warps
// of their own: one tree 4.3 us, but 256 trees 22.8.)
template <int ES>  // bytes of an element: 4, 2, or 1 (codes, with their exponents)
__global__ void __launch_bounds__(128) keep_kernel(const KeepParams p) {
  using V = typename std::conditional<ES == 4, uint32_t, typename std::conditional<ES == 2, uint16_t, uint8_t>::type>::type;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int s = (int)(unit / p.nkv), h = (int)(unit % p.nkv);
  if (s >= p.nb) return;
  const int n = p.path_lens[s], ctx = p.ctx_lens[s];
  const int32_t* path = p.path + (int64_t)s * p.max_path;
  const int64_t cap = (int64_t)p.mpps * kPage;
  unsigned bad = 0;
  if (n < 0 || n > p.max_path) {
    bad = DFLASH_DEV_BAD_TREE;
  } else {
    for (int i = lane; i < n; i += 32) {
      const int x = path[i];
      if (x < 0 || (i > 0 && path[i - 1] >= x)) bad |= DFLASH_DEV_BAD_TREE;
      if ((int64_t)ctx + x >= cap) bad |= DFLASH_DEV_BAD_CTX;
    }
    if (ctx < 0 || ctx > cap - n) bad |= DFLASH_DEV_BAD_CTX;  // (also where no row moves: the rows below stay within the table's)
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (bad) {
    if (lane == 0 && p.status) atomicOr(p.status, bad & DFLASH_DEV_BAD_TREE ? DFLASH_DEV_BAD_TREE : DFLASH_DEV_BAD_CTX);
    return;
  }
  if (n == 0) return;
  const int32_t* table = p.page_tables + (int64_t)s * p.mpps;
  const int hd = p.hd, pieces = hd * ES / 16;  // K of a row: pieces of 16 bytes, at most 32
  for (int b1 = ctx & ~7; b1 < ctx + n; b1 += 32) {
    // lane l: the row that goes to b1 + l (four half pages' places are looked up at once: 5.0 -> 4.7 us for a tree)
    const int i = b1 + lane - ctx;
    uint8_t *from = nullptr, *to = nullptr;
    int jf = 0;
    bool there = false, move = false;
    if (i >= 0 && i < n) {
      const int a = ctx + path[i], b = b1 + lane;
      const int pa = table[a / kPage], pb = table[b / kPage];
      there = pa >= 0 && pa < p.num_pages && pb >= 0 && pb < p.num_pages;
      move = there && a != b;
      if (!there && a != b && p.status) atomicOr(p.status, DFLASH_DEV_BAD_PAGE);
      if (there) {
        from = p.pool + pa * p.page_bytes + h * p.head_bytes;
        to = p.pool + pb * p.page_bytes + h * p.head_bytes;
      }
      jf = a % kPage;
    }
    const unsigned movers = __ballot_sync(0xffffffffu, move), placed = __ballot_sync(0xffffffffu, there);
#pragma unroll 1
    for (int g = 0; g < 32; g += 8) {
      const unsigned moving = movers >> g & 0xff;
      if (!moving) continue;
      const bool whole = (placed >> g & 0xff) == 0xffu;  // (rows that stay are then stored as they were)
      const unsigned take = whole ? 0xffu : moving;
      uint8_t* dst = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), g + __ffs(moving) - 1));
      const int j0 = (b1 + g) % kPage;
      uint4 k[8];
      V v[8][4];
      uint8_t e[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const uint8_t* f = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(from), g + r));
        const int j = __shfl_sync(0xffffffffu, jf, g + r);
        if (!(take >> r & 1)) continue;
        if (lane < pieces)
          k[r] = *reinterpret_cast<const uint4*>(f + (ES == 1 ? k8_in_tile(j, lane * 16) : k_in_tile(j, lane * (16 / ES), hd) * ES));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int d = lane + 32 * x;
          if (d < hd) v[r][x] = reinterpret_cast<const V*>(f + 16 * hd * ES)[ES == 1 ? v8_in_tile(j, d) : v_in_tile(j, d, hd)];
        }
        if (ES == 1 && lane < 2) e[r] = f[32 * hd + 16 * lane + j];
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (!(take >> r & 1)) continue;
        const int j = j0 + r;
        if (lane < pieces)
          *reinterpret_cast<uint4*>(dst + (ES == 1 ? k8_in_tile(j, lane * 16) : k_in_tile(j, lane * (16 / ES), hd) * ES)) = k[r];
        if (!whole) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int d = lane + 32 * x;
            if (d < hd) reinterpret_cast<V*>(dst + 16 * hd * ES)[ES == 1 ? v8_in_tile(j, d) : v_in_tile(j, d, hd)] = v[r][x];
          }
        }
        if (ES == 1 && lane < 2) dst[32 * hd + 16 * lane + j] = e[r];
      }
      if (whole) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int d = lane + 32 * x;
          if (d >= hd) continue;
          if (ES == 1) {
#pragma unroll
            for (int z = 0; z < 8; z += 4)
              *reinterpret_cast<uint32_t*>(dst + 16 * hd + v8_in_tile(j0 + z, d)) = v[z][x] | (uint32_t)v[z + 1][x] << 8 | (uint32_t)v[z + 2][x] << 16 | (uint32_t)v[z + 3][x] << 24;
          } else {
            uint4* out = reinterpret_cast<uint4*>(dst + (16 * hd + v_in_tile(j0, d, hd)) * ES);
            if (ES == 2) {
              out[0] = make_uint4(v[0][x] | (uint32_t)v[1][x] << 16, v[2][x] | (uint32_t)v[3][x] << 16, v[4][x] | (uint32_t)v[5][x] << 16, v[6][x] | (uint32_t)v[7][x] << 16);
            } else {
              out[0] = make_uint4(v[0][x], v[1][x], v[2][x], v[3][x]);
              out[1] = make_uint4(v[4][x], v[5][x], v[6][x], v[7][x]);
            }
          }
        }
      }
    }
  }
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" int dflash_draft_tree(const int32_t* parents, const int32_t* kv_lens, const int32_t* row_starts, int32_t nb,
                                 int32_t n_rows, int32_t max_nodes, int32_t* positions, uint64_t* masks,
                                 uint32_t* status, dflash_stream stream) {
  if (nb < 1 || n_rows < 0) return call_error(DFLASH_EINVAL, "draft_tree: nb >= 1 and n_rows >= 0");
  if (nb > 16384 || n_rows > 1 << 30) return call_error(DFLASH_ECAPACITY, "draft_tree: nb above 16384 or n_rows above 2^30");
  if (max_nodes < 1 || max_nodes > kMaxNodes) return call_error(DFLASH_EUNSUPPORTED, "draft_tree: max_nodes must be in [1, 512]");
  if (n_rows == 0) return DFLASH_OK;
  if (!parents || !kv_lens || !row_starts || !positions || !masks) return call_error(DFLASH_EINVAL, "draft_tree: null pointer");
  const int threads = (max_nodes + 63) / 64 * 64;  // as many as the masks have bits
  const int rest = (int)std::min<int64_t>(64, ((int64_t)n_rows + threads - 1) / threads);
  draft_tree_kernel<<<nb + rest, threads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      parents, kv_lens, row_starts, nb, n_rows, (max_nodes + 63) / 64, positions, reinterpret_cast<unsigned long long*>(masks), status);
  if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return call_error(DFLASH_ECUDA, "draft_tree", e);
  return DFLASH_OK;
}

extern "C" int dflash_keep_rows(const dflash_kv_pages* kv, const int32_t* page_tables, int32_t max_pages_per_seq,
                                const int32_t* ctx_lens, int32_t nb, const int32_t* path, int32_t max_path,
                                const int32_t* path_lens, dflash_stream stream) {
  if (int rc = check_pages(kv, true)) return rc;
  if (nb < 1 || max_path < 0) return call_error(DFLASH_EINVAL, "keep_rows: nb >= 1 and max_path >= 0");
  if (nb > 16384 || max_path > kMaxNodes) return call_error(DFLASH_ECAPACITY, "keep_rows: nb above 16384 or max_path above 512");
  if (max_pages_per_seq < 1 || max_pages_per_seq >= 1 << 26)
    return call_error(DFLASH_EINVAL, "keep_rows: max_pages_per_seq must be in [1, 2^26)");
  if (!page_tables || !ctx_lens || !path_lens || (max_path > 0 && !path)) return call_error(DFLASH_EINVAL, "keep_rows: null pointer");
  const int es = page_es(kv);
  const int64_t head = es == 1 ? 32 * kv->head_dim + 32 : (int64_t)32 * kv->head_dim * es;
  KeepParams p{static_cast<uint8_t*>(kv->pool), kv->page_stride * es, head, page_tables, ctx_lens, path, path_lens, kv->status,
               nb, kv->n_kv_heads, max_pages_per_seq, kv->num_pages, max_path, kv->head_dim};
  const int64_t units = (int64_t)nb * kv->n_kv_heads;
  auto kern = es == 4 ? keep_kernel<4> : es == 2 ? keep_kernel<2> : keep_kernel<1>;
  kern<<<(unsigned)((units + 3) / 4), 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return call_error(DFLASH_ECUDA, "keep_rows", e);
  return DFLASH_OK;
}
