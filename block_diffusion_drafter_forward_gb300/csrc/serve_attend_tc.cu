// Tensor-core form of dflash_attend (bf16): paged attention of ragged chunks, stream-K.
//
// Work unit = (sequence, query tile, kv head): with G = query heads per kv head, the G heads of
// T = floor(128 / G) tokens are the rows of one 128-row UMMA tile (row = token * G + head), so a
// K/V byte feeds every query head that shares it.  Keys go in chunks of 128 (8 pages).  The
// chunks of all units, in (sequence, tile, head) order, form one index space; CTA b of a
// one-CTA-per-SM grid takes slots [b W / n, (b + 1) W / n) of it, sized on the device from the
// lengths, so prompts, blocks and single tokens share the SMs evenly and a graph replayed with
// other lengths stays balanced.  A unit cut between CTAs leaves fp32 partials (O, m, l) in the
// workspace (at most two per CTA) that attend_combine_kernel merges in key order.
//
// Two softmax streams of 128 threads (one query row each) keep the tensor cores fed, in two forms:
//   two tiles (long chunks): stream x owns query tile x of a 256-row unit, both read the same
//     K/V slots: 4 x 128 x 128 x head_dim products per 64 KB of K/V, tensor-bound;
//   one tile (short chunks): stream x takes the chunks of parity x of the same queries, and the
//     two (O, m, l) meet at the segment's end: HBM-bound, two chunks' softmax in flight.
// Per stream the order is S = Q K^T -> softmax -> O += P V -> next S; while one stream's softmax
// runs, the tensor cores work for the other.  P goes back as bf16 over its own S columns and is
// read from TMEM; O stays in TMEM and is rescaled only when a row's maximum grew by more than
// 2^8 (P <= 2^8 stays exact in range, the normalised result is the same).
//
// Bound and measured (GB300, 32 query heads on 4 kv heads of 128): single tokens and short blocks by
// HBM - 16 single tokens on 16-32 Ki rows (64 heads on 8) 243 us, 6.6 TB/s; 32 blocks of 16 on
// 0.5-8 Ki rows 64 us, 4.3 TB/s (7 us less without its copies: the chunks' chain and the segments'
// ends).  Prompts by the chain of one chunk - softmax 1.5-2.3 kcycles, P V and S 1.1 and their
// hand-overs - of which two streams fill 57 % of the tensor pipe: a prompt of 8192 499 us,
// 1.10 PFLOP/s (no single part holds it: without exponentials 2 % less, without maxima 8, without
// copies 3; 64 keys at a time, S a half ahead of the softmax, 10 more - Q is then read twice as
// often, and shared memory gives S its Q and K at 128 B a cycle).
//
// Rounding: P is bf16 (the MMA's operand type), sums and O fp32, the normaliser sums the fp32 P.
// Warp roles: 0-3 stream 0, 4-7 stream 1, 8 K pages, 10 V pages, 9 and 11 MMA issue.  The V warp
// also zeroes the key rows behind a sequence's end in its last page (never-written rows may hold
// NaN, and 0 * NaN would reach O; their scores are masked by select).  Issuing an MMA blocks its
// thread while the tensor pipe's queue is full, so with two tiles each stream has a warp of its own
// (one that issued for both left the pipe idle between the streams: 614 against 564 us for a prompt
// of 8192); with one tile a single thread keeps the chunks in order over both streams.
#include <float.h>

#include <atomic>
#include <type_traits>

#include "launch_util.cuh"
#include "serve_attend.cuh"
#include "tc_common.cuh"

namespace dflash {
namespace {

using namespace tc;

constexpr int kKeys = 128;                      // keys per chunk
constexpr int kPages = kKeys / kPage;           // 8
constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kCtl = 2944;                      // barriers, plan, row exchange

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// The wait of tc_common.cuh with its first poll ahead of the abort flag: most waits find their phase
// complete, and a shared-memory read costs hundreds of cycles while MMAs saturate its bandwidth.
__device__ __forceinline__ bool wait_ab(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_try_wait(bar, parity) || mbar_wait_ab(bar, parity, abort);
}

// Slots of the index space a unit occupies beside its chunks: the cost of opening a segment
// (queries, pipeline restart, output) in chunks.
constexpr int kUnitCost = 3;

template <int HD, int NT>
struct Cfg {
  static constexpr int kTile = kPage * HD * 2;         // a page of one head: bytes of K (or V)
  static constexpr int kQ = 128 * HD * 2;              // a query tile
  static constexpr int kSlot = kPages * kTile;         // a chunk's K (or V)
  static constexpr int kNK = HD == 128 ? 3 : 6;        // K and V slots in flight
  static constexpr int kNV = HD == 128 ? 2 : 6;
  static constexpr int kSmem = 2 * kQ + (kNK + kNV) * kSlot + kCtl;  // (queries: two tiles, or two segments' tile)
};

struct Seg {
  int s, r0, n, kv;     // sequence, its first row, rows, key rows
  int tile, g, t0;      // query tile, kv head, its first token
  int k0, nch;          // first key (page aligned), chunks of the unit
  int c_lo, c_hi;       // this CTA's chunks of it
};

// Tokens of a unit's tile and the chunks it visits.
struct Shape {
  int group, T, TT;     // query heads per kv head, tokens of a 128-row tile, of a unit
};
__device__ __forceinline__ Shape shape_of(const AttendParams& p, int NT) {
  Shape h;
  h.group = p.group;
  h.T = p.tokens;
  h.TT = h.T * NT;
  return h;
}
__device__ __forceinline__ int unit_chunks(const AttendParams& p, const Shape& h, int n, int kv, int tile, int* k0) {
  const int t0 = tile * h.TT, t1 = min(n, t0 + h.TT);
  const int end = p.causal ? min(kv, max(0, kv - n + t1)) : kv;
  int lo = p.window > 0 ? max(0, kv - n + t0 - p.window + 1) : 0;
  lo &= ~(kPage - 1);
  *k0 = lo;
  return max(1, (end - lo + kKeys - 1) / kKeys);  // a unit without keys still writes its zeros
}

// The segments of index range [lo, hi), from unit (s, tile, g) whose first slot is pu.
struct Walk {
  long long lo, hi, pu;
  int s, tile, g;

  __device__ bool next(const AttendParams& p, const Shape& h, Seg& q) {
    while (pu < hi && s < p.nb) {
      bool bad;
      if (!seq_of(p, s, &q.r0, &q.n, &q.kv, &bad)) {
        ++s;
        tile = g = 0;
        continue;
      }
      q.nch = unit_chunks(p, h, q.n, q.kv, tile, &q.k0);
      q.s = s, q.tile = tile, q.g = g, q.t0 = tile * h.TT;
      const long long first = pu + kUnitCost;
      pu = first + q.nch;
      if (++g == p.nkv) {
        g = 0;
        if (++tile * h.TT >= q.n) tile = 0, ++s;
      }
      if (hi <= first || lo >= pu) continue;  // only cost slots of it are in range
      q.c_lo = (int)(lo > first ? lo - first : 0);
      q.c_hi = (int)(hi < pu ? hi - first : q.nch);
      return true;
    }
    return false;
  }
};

struct Ctl {
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6], v_raw[6];
  uint64_t s_full[2], p_half[2], p_full[2], o_done[2], o_free[2], q_full[2];
  uint32_t tmem_slot;
  int flags[2];
  int s0, tile0, found;
  long long red[kWarps], W, base;
  float2 ml[2][128];  // one tile: the streams' (m, l) of every row
};
static_assert(sizeof(Ctl) <= kCtl, "control block overflows its slot");

// Slots of tiles [a, b) of a sequence for one kv head, by this thread.
__device__ __forceinline__ long long tile_slots(const AttendParams& p, const Shape& h, int n, int kv, int a, int b, int step) {
  long long r = 0;
  int k0;
  for (int t = a; t < b; t += step) r += unit_chunks(p, h, n, kv, t, &k0) + kUnitCost;
  return r;
}

// This CTA's walk.  `scratch`: nb long longs of shared memory.  All threads.
__device__ Walk plan(const AttendParams& p, const Shape& h, Ctl& c, long long* scratch, bool wide, long long* W_out) {
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (p.nb <= 32 && !wide) {
    // a lane per sequence, every warp for itself: no barrier (a step's first 3.5 us went by in the
    // general form's)
    int r0, n = 0, kv = 0, k0;
    bool bad = false;
    const bool has = lane < p.nb && seq_of(p, lane, &r0, &n, &kv, &bad);
    if (bad && blockIdx.x == 0 && warp == 0 && p.status) atomicOr(p.status, DFLASH_DEV_BAD_CTX);
    const int tiles = has ? (n + h.TT - 1) / h.TT : 0;
    const long long mine = tile_slots(p, h, n, kv, 0, tiles, 1) * p.nkv;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const long long W = __shfl_sync(0xffffffffu, inc, 31);
    const int G = (int)min((long long)gridDim.x, W), b = blockIdx.x;
    Walk w;
    w.lo = b < G ? (long long)b * W / G : 0;
    w.hi = b < G ? (long long)(b + 1) * W / G : 0;
    w.s = p.nb, w.tile = w.g = 0, w.pu = w.hi;
    *W_out = W;
    if (w.lo >= w.hi) return w;
    const int s0 = __ffs(__ballot_sync(0xffffffffu, inc > w.lo)) - 1;  // the sequence that holds slot lo
    long long at = __shfl_sync(0xffffffffu, inc - mine, s0);
    const int n0 = __shfl_sync(0xffffffffu, n, s0), kv0 = __shfl_sync(0xffffffffu, kv, s0);
    w.s = s0;
    for (;;) {  // its tile: at most a few
      const int slots = unit_chunks(p, h, n0, kv0, w.tile, &k0) + kUnitCost;
      if (w.lo < at + (long long)slots * p.nkv) {
        w.g = (int)((w.lo - at) / slots);
        w.pu = at + (long long)w.g * slots;
        return w;
      }
      at += (long long)slots * p.nkv;
      ++w.tile;
    }
  }
  // slots of each sequence (all kv heads): a thread per sequence, or a warp where chunks are long
  for (int s = wide ? warp : t; s < p.nb; s += wide ? kWarps : kThreads) {
    int r0, n, kv;
    bool bad;
    long long m = 0;
    if (seq_of(p, s, &r0, &n, &kv, &bad)) {
      const int tiles = (n + h.TT - 1) / h.TT;
      m = wide ? tile_slots(p, h, n, kv, lane, tiles, 32) : tile_slots(p, h, n, kv, 0, tiles, 1);
    } else if (bad && blockIdx.x == 0 && p.status && (!wide || lane == 0)) {
      atomicOr(p.status, DFLASH_DEV_BAD_CTX);
    }
    if (wide) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    }
    if (!wide || lane == 0) scratch[s] = m * p.nkv;
  }
  if (t == 0) c.found = 0;
  __syncthreads();
  // thread t sums sequences [t per, (t + 1) per)
  const int per = (p.nb + kThreads - 1) / kThreads, s_lo = min(p.nb, t * per), s_hi = min(p.nb, s_lo + per);
  auto scan = [&](long long v, long long* all) {  // exclusive sum over the threads before this one
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) c.red[warp] = inc;
    __syncthreads();
    long long b = inc - v, a = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) b += c.red[w];
      a += c.red[w];
    }
    __syncthreads();
    *all = a;
    return b;
  };
  long long mine = 0, W;
  for (int s = s_lo; s < s_hi; ++s) mine += scratch[s];
  long long at = scan(mine, &W);
  const int G = (int)min((long long)gridDim.x, W), b = blockIdx.x;
  Walk w;
  w.lo = b < G ? (long long)b * W / G : 0;
  w.hi = b < G ? (long long)(b + 1) * W / G : 0;
  w.s = p.nb, w.tile = w.g = 0, w.pu = w.hi;
  *W_out = W;
  if (w.lo >= w.hi) return w;
  if (at <= w.lo && w.lo < at + mine) {
    for (int s = s_lo; s < s_hi; ++s) {
      if (w.lo < at + scratch[s]) {
        c.s0 = s, c.base = at;
        break;
      }
      at += scratch[s];
    }
  }
  __syncthreads();
  const int s0 = c.s0;
  long long base = c.base;
  int r0, n, kv, k0;
  bool bad;
  seq_of(p, s0, &r0, &n, &kv, &bad);
  const int tiles = (n + h.TT - 1) / h.TT;
  for (int b0 = 0; b0 < tiles; b0 += kThreads) {  // the tile that holds slot lo
    const int tile = b0 + t;
    const long long v = tile < tiles ? (long long)(unit_chunks(p, h, n, kv, tile, &k0) + kUnitCost) * p.nkv : 0;
    long long all;
    const long long x = base + scan(v, &all);
    if (v > 0 && x <= w.lo && w.lo < x + v) c.tile0 = tile, c.base = x, c.found = 1;
    base += all;
    __syncthreads();
    if (c.found) break;
  }
  w.s = s0, w.tile = c.tile0;
  const int slots = unit_chunks(p, h, n, kv, w.tile, &k0) + kUnitCost;
  w.g = (int)((w.lo - c.base) / slots);
  w.pu = c.base + (long long)w.g * slots;
  return w;
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
// 64 columns of this lane's TMEM row, without the wait; ld_wait ties the registers to it
__device__ __forceinline__ void ld64(uint32_t taddr, float (&v)[64]) {
  __syncwarp();
#define R8(i) "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3]), "=f"(v[i + 4]), "=f"(v[i + 5]), "=f"(v[i + 6]), "=f"(v[i + 7])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
      : R8(0), R8(8), R8(16), R8(24), R8(32), R8(40), R8(48), R8(56)
      : "r"(taddr));
#undef R8
}
__device__ __forceinline__ void ld_wait(float (&a)[64], float (&b)[64]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) asm volatile("" : "+f"(a[i]), "+f"(b[i]));
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t (&v)[32]) {  // 32 columns, without the wait
  __syncwarp();
#define R8(i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::R8(0),
      R8(8), R8(16), R8(24), "r"(taddr)
      : "memory");
#undef R8
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The chunks of stream x, in order, as every role counts them.
template <int NT>
struct It {
  Walk w;
  Seg sg;
  int j, n;        // chunk within the segment, chunks of it
  int kc0;         // chunks of the segments before it
  int it;          // chunks this stream did before
  int seg, act;    // segments before this one: all, and those this stream works in
  bool valid;

  // does stream x work in the segment?
  __device__ static bool active(const Shape& h, const Seg& q, int x) {
    return x == 0 || (NT == 2 ? q.t0 + h.T < q.n : q.c_hi - q.c_lo > 1);
  }
  __device__ bool enter(const AttendParams& p, const Shape& h, int x) {
    while (w.next(p, h, sg)) {
      ++seg;
      n = sg.c_hi - sg.c_lo;
      if (active(h, sg, x)) {
        ++act;
        j = NT == 2 ? 0 : x;
        return true;
      }
      kc0 += n;
    }
    return false;
  }
  __device__ void start(const AttendParams& p, const Shape& h, const Walk& w0, int x) {
    w = w0;
    kc0 = it = 0;
    seg = act = -1;
    valid = enter(p, h, x);
  }
  __device__ bool first(int x) const { return j == (NT == 2 ? 0 : x); }
  __device__ void step(const AttendParams& p, const Shape& h, int x) {
    ++it;
    j += NT == 2 ? 1 : 2;
    if (j < n) return;
    kc0 += n;
    valid = enter(p, h, x);
  }
  // pages of the chunk that hold keys of the sequence
  __device__ int pages() const {
    const int k = sg.k0 + (sg.c_lo + j) * kKeys;
    return max(0, min(kPages, (sg.kv - k + kPage - 1) / kPage));
  }
};

template <int HD, int NT>
__global__ void __launch_bounds__(kThreads, 1) attend_tc_kernel(const AttendParams p, const AttendWork wk, const __grid_constant__ CUtensorMap q_map) {
  using C = Cfg<HD, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];  // (the queries' swizzle counts from 1 KB boundaries)
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + 2 * C::kQ;
  uint8_t* sV = sK + C::kNK * C::kSlot;
  Ctl& c = *reinterpret_cast<Ctl*>(sV + C::kNV * C::kSlot);
  volatile int* flags = c.flags;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const Shape h = shape_of(p, NT);

  pdl_wait();  // everything read here may come from the kernel before
  if (t == 0) wk.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
  long long W;
  const Walk walk = plan(p, h, c, reinterpret_cast<long long*>(sK), wk.long_chunks, &W);
  if (walk.lo >= walk.hi) {  // nothing for this CTA
    pdl_trigger();
    return;
  }
  if (t == 0) {
    for (int i = 0; i < 6; ++i) {
      mbar_init(&c.k_full[i], 1);
      mbar_init(&c.k_empty[i], NT);
      mbar_init(&c.v_full[i], 1);
      mbar_init(&c.v_empty[i], NT);
      mbar_init(&c.v_raw[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.s_full[i], 1);
      mbar_init(&c.p_half[i], 128);
      mbar_init(&c.p_full[i], 128);
      mbar_init(&c.o_done[i], 1);
      mbar_init(&c.o_free[i], NT == 2 ? 128 : 256);
      mbar_init(&c.q_full[i], 1);
    }
    flags[0] = 0;
    fence_barrier_init();
  }
  // rows that no query fills stay finite
  if (h.group * h.T < 128)
    for (int i = t; i < 2 * C::kQ / 16; i += kThreads) reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();  // the plan's scratch is overwritten by copies
  if (warp == 0) tmem_alloc(&c.tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem_slot;
  pdl_trigger();
  // Queries of a segment into tile b (its second query tile's: two tiles, b = 1) by TMA: rows of 64
  // dims in the 128-byte swizzle, (head, token) in the tile's row order.  One thread.  (Copied by the
  // softmax threads, 16 bytes each, they queued for thousands of cycles behind the pages.)
  auto load_q = [&](const Seg& q, int b) {
    mbar_arrive_expect_tx(&c.q_full[b], h.group * h.T * HD * 2);
    for (int d = 0; d < HD / 64; ++d)
      tma_load_3d(sQ + b * C::kQ + d * (128 * 128), &q_map, &c.q_full[b], d * 64, q.g * h.group, q.r0 + q.t0 + (NT == 2 ? b * h.T : 0));
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 8 || warp == 10) {
      // ---- page producers: lane l copies page l of a chunk.  The page ids of the next chunk are
      // fetched while the warp waits for a slot.  V of a chunk whose last page is part full (or that
      // has no page) lands on v_raw; the V warp zeroes its rows behind the end when it has come,
      // between its other work.
      const int kv = warp == 10;
      uint64_t* full = kv ? c.v_full : c.k_full;
      uint64_t* empty = kv ? c.v_empty : c.k_empty;
      uint8_t* ring = kv ? sV : sK;
      const int slots = kv ? C::kNV : C::kNK;
      Walk w = walk;
      Seg q;
      int i = 0;
      bool stop = false;
      uint32_t used = 0;                 // parity of each slot's v_raw
      int tail_b = -1, tail_page = 0, tail_live = 0;  // the slot to zero in; its last page, rows to keep there
      auto mend = [&] {                  // waits for it; false: gave up
        if (tail_b < 0) return true;
        if (!__all_sync(0xffffffffu, wait_ab(&c.v_raw[tail_b], (used >> tail_b) & 1, flags))) return false;
        uint4* v = reinterpret_cast<uint4*>(sV + tail_b * C::kSlot + tail_page * C::kTile);
        for (int e = lane; e < HD * 2; e += 32) {  // 16 bytes: 8 keys of one dim, (d / 8, key / 8, d % 8)
          const int j0 = (e >> 3 & 1) * 8;
          if (j0 >= tail_live) {
            v[e] = make_uint4(0, 0, 0, 0);
          } else if (j0 + 8 > tail_live) {
            __nv_bfloat16* x = reinterpret_cast<__nv_bfloat16*>(v + e);
            for (int k = tail_live - j0; k < 8; ++k) x[k] = __float2bfloat16(0.f);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.v_full[tail_b]);
        used ^= 1u << tail_b;
        tail_b = -1;
        return true;
      };
      while (!stop && w.next(p, h, q)) {
        const int pages = (q.kv + kPage - 1) / kPage;
        auto fetch = [&](int ch) {
          const int lp = (q.k0 + ch * kKeys) / kPage + lane;
          return lane < kPages && lp < pages && ch < q.c_hi ? __ldg(p.page_tables + (int64_t)q.s * p.mpps + lp) : 0;
        };
        int page = fetch(q.c_lo);
        for (int ch = q.c_lo; ch < q.c_hi; ++ch, ++i) {
          const int b = i % slots;
          if (i >= slots) {
            const uint32_t par = (i / slots - 1) & 1;
            // meanwhile the pending page (votes keep the warp together); the wait below is the bound
            for (long long n = 0; tail_b >= 0 && n < kSpinLimit; ++n) {
              if (__any_sync(0xffffffffu, flags[0] || mbar_test_wait(&empty[b], par))) break;
              if (__any_sync(0xffffffffu, mbar_test_wait(&c.v_raw[tail_b], (used >> tail_b) & 1))) mend();
            }
            if (!wait_ab(&empty[b], par, flags)) {
              stop = true;
              break;
            }
          }
          const int key = q.k0 + ch * kKeys;
          const int np = max(0, min(kPages, pages - key / kPage));
          const bool tail = kv && (np == 0 || key + np * kPage > q.kv);
          if (tail && !mend()) {  // one at a time
            stop = true;
            break;
          }
          uint64_t* bar = tail ? &c.v_raw[b] : &full[b];
          if (lane == 0) mbar_arrive_expect_tx(bar, np * C::kTile);
          __syncwarp();
          if (lane < np) {
            if (page < 0 || page >= p.num_pages) {
              if (p.status) atomicOr(p.status, DFLASH_DEV_BAD_PAGE);
              page = 0;
            }
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.pool) + page * p.page_stride +
                                       ((int64_t)q.g * 2 + kv) * (kPage * HD);
            bulk_load(ring + b * C::kSlot + lane * C::kTile, src, C::kTile, bar);
          }
          if (tail) {
            tail_b = b;
            tail_page = max(0, np - 1);
            tail_live = np == 0 ? 0 : q.kv - key - tail_page * kPage;
          }
          page = fetch(ch + 1);
        }
      }
      if (!stop) mend();
    } else if (lane == 0) {
      // ---- MMA issue
      constexpr uint32_t id_s = idesc_bf16(128, kKeys), id_o = idesc_bf16(128, HD);
      // operand descriptors of the first tiles; the others are further on (16-byte units)
      const uint64_t dQ = desc_sw128(sQ), dK = desc_noswz(sK, 128, HD * 16), dV = desc_noswz(sV, 128, 256);
      auto issue_s = [&](int x, int qb, int kb) {  // queries in tile qb
        const uint64_t q = dQ + (uint64_t)(qb * (C::kQ / 16)), k = dK + (uint64_t)(kb * (C::kSlot / 16));
#pragma unroll
        for (int d = 0; d < HD / 16; ++d)  // (queries: 32 bytes on in a 64-dim half of 16 KB)
          mma_bf16(tmem + x * 128, q + (d & 3) * 2 + (d >> 2) * 1024, k + d * 16, id_s, d > 0 ? 1u : 0u);
      };
      auto issue_pv = [&](int x, int vb, int k0, int k1, bool more) {  // pages k0 .. k1 - 1: 16 keys = 8 TMEM columns of P each
        const uint64_t v = dV + (uint64_t)(vb * (C::kSlot / 16));
        const uint32_t tS = tmem + x * 128, tO = tmem + 256 + x * 128;
        if (k1 - k0 == kPages / 2) {
#pragma unroll
          for (int k = 0; k < kPages / 2; ++k)
            mma_bf16_tmem_a(tO, tS + (k0 + k) * 8, v + (k0 + k) * (C::kTile / 16), id_o, k0 + k > 0 || more ? 1u : 0u);
        } else {
          for (int k = k0; k < k1; ++k) mma_bf16_tmem_a(tO, tS + k * 8, v + k * (C::kTile / 16), id_o, k > 0 || more ? 1u : 0u);
        }
      };
      if (NT == 2) {
        // one stream: S of a chunk, then its P V and the next S as soon as the softmax has written P
        const int x = warp == 9 ? 0 : 1;
        Walk w = walk;
        Seg q;
        int kc = 0, it = 0, act = 0;
        auto wait = [&](uint64_t* bar, int phase) {
          if (!wait_ab(bar, phase & 1, flags)) flags[0] = 1;  // after a timeout: commits only, no MMAs
        };
        auto s_of = [&](int kc) {  // (its K has been waited for)
          const int kb = kc % C::kNK;
          tc_fence_after();
          if (!flags[0]) issue_s(x, x, kb);
          mma_commit(&c.s_full[x]);
          mma_commit(&c.k_empty[kb]);
        };
        while (w.next(p, h, q)) {
          const int n = q.c_hi - q.c_lo;
          if (!It<NT>::active(h, q, x)) {
            // no row of this stream: it still follows every slot, so that its waits stay exact
            for (int j = 0; j < n; ++j, ++kc) {
              wait(&c.k_full[kc % C::kNK], kc / C::kNK);
              mbar_arrive(&c.k_empty[kc % C::kNK]);
              wait(&c.v_full[kc % C::kNV], kc / C::kNV);
              mbar_arrive(&c.v_empty[kc % C::kNV]);
            }
            continue;
          }
          wait(&c.k_full[kc % C::kNK], kc / C::kNK);
          wait(&c.q_full[x], act);
          s_of(kc);
          for (int j = 0; j < n; ++j, ++kc, ++it) {
            const int vb = kc % C::kNV;
            const int np = max(1, min(kPages, (q.kv - q.k0 - (q.c_lo + j) * kKeys + kPage - 1) / kPage));
            // what the softmax does not decide is waited for while it runs
            if (j + 1 < n) wait(&c.k_full[(kc + 1) % C::kNK], (kc + 1) / C::kNK);
            wait(&c.v_full[vb], kc / C::kNV);
            if (j == 0 && act > 0) wait(&c.o_free[x], act - 1);
            wait(&c.p_half[x], it);  // P of the first 64 keys, while the exponentials of the others run
            tc_fence_after();
            if (!flags[0]) issue_pv(x, vb, 0, min(np, kPages / 2), j > 0);
            wait(&c.p_full[x], it);
            tc_fence_after();
            if (!flags[0]) issue_pv(x, vb, kPages / 2, np, true);
            mma_commit(&c.o_done[x]);
            mma_commit(&c.v_empty[vb]);
            if (j + 1 < n) s_of(kc + 1);
          }
          ++act;
        }
      } else if (warp == 9) {
        // both streams: each alternates S and P V; whichever is ready goes out
        It<NT> its[2];
        bool pv[2] = {false, false};
        its[0].start(p, h, walk, 0);
        its[1].start(p, h, walk, 1);
        long long idle = 0;
        // A wait by parity is exact only while the phase before the awaited one is known complete, so
        // no stream may run ahead of the other by a ring: S and P V go out in chunk order over both.
        int s_next = 0, pv_next = 0;  // chunks whose S / P V is out
        while (its[0].valid || its[1].valid) {
          bool did = false;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            It<NT>& a = its[x];
            const bool give_up = flags[0];  // after a timeout: commits only, no MMAs
            if (a.valid && pv[x]) {
              const int kc = a.kc0 + a.j, vb = kc % C::kNV;
              if (give_up || (kc == pv_next && mbar_test_wait(&c.p_full[x], a.it & 1) &&
                              mbar_test_wait(&c.v_full[vb], (kc / C::kNV) & 1) &&
                              (!a.first(x) || a.seg == 0 || mbar_test_wait(&c.o_free[0], (a.seg - 1) & 1)))) {
                tc_fence_after();
                if (!give_up) {
                  const int np = max(1, a.pages());
                  issue_pv(x, vb, 0, min(np, kPages / 2), !a.first(x));
                  issue_pv(x, vb, kPages / 2, np, true);
                }
                mma_commit(&c.o_done[x]);
                mma_commit(&c.v_empty[vb]);
                ++pv_next;
                pv[x] = false;
                a.step(p, h, x);
                did = true;
              }
            }
            if (a.valid && !pv[x]) {
              const int kc = a.kc0 + a.j, kb = kc % C::kNK;
              if (give_up || (kc == s_next && mbar_test_wait(&c.k_full[kb], (kc / C::kNK) & 1) &&
                              (!a.first(x) || mbar_test_wait(&c.q_full[a.seg & 1], a.seg >> 1 & 1)))) {
                tc_fence_after();
                if (!give_up) issue_s(x, a.seg & 1, kb);
                mma_commit(&c.s_full[x]);
                mma_commit(&c.k_empty[kb]);
                ++s_next;
                pv[x] = true;
                did = true;
              }
            }
          }
          idle = did ? 0 : idle + 1;
          if (idle > kSpinLimit) flags[0] = 1;
        }
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---- softmax streams: thread = query row `row` of its tile
    const int x = warp >> 2, row = t & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lane_off;
    const int tok = row / h.group, head = row - tok * h.group;  // (by p.inv the loop's registers fall worse: 519 us for 499)
    const bool loads = (t & 127) == 0 && (NT == 2 || x == 0);  // (one tile: stream 0's, a segment ahead)
    Walk w = walk;
    Seg q, nq;
    bool have = w.next(p, h, q);
    while (NT == 2 && have && !It<NT>::active(h, q, x)) have = w.next(p, h, q);
    if (have && loads) load_q(q, x);
    int it = 0, seg = 0;  // chunks and segments done by this stream
    while (have) {
      bool more = w.next(p, h, nq);
      while (NT == 2 && more && !It<NT>::active(h, nq, x)) more = w.next(p, h, nq);
      const int n = q.c_hi - q.c_lo;
      const int tk = q.t0 + (NT == 2 ? x * h.T : 0) + tok;
      const bool valid = tok < h.T && tk < q.n;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      // keys [lo, hi) are seen by this row (rows without a token: anything, they are not written)
      const int pos = q.kv - q.n + tk;
      const int hi = !valid ? INT_MAX : p.causal ? min(q.kv, pos + 1) : q.kv;
      const int lo = valid && p.window > 0 ? max(0, pos - p.window + 1) : 0;
      float m = -INFINITY, l = 0.f;
      int done = 0;
#pragma unroll 1
      for (int j = NT == 2 ? 0 : x; j < n; j += NT == 2 ? 1 : 2, ++it, ++done) {
        if (!wait_ab(&c.s_full[x], it & 1, flags)) flags[0] = 1;
        tc_fence_after();
        // the next queries: two tiles, into the same tile once this segment's last S is done; one,
        // into the other tile once this segment's first is (so every S of the segment before is)
        if (loads && more && j == (NT == 2 ? n - 1 : 0)) load_q(nq, NT == 2 ? x : (seg + 1) & 1);
        if (warp_valid) {
          const int kb = q.k0 + (q.c_lo + j) * kKeys;
          float a[64], b[64];
          ld64(tS, a);
          ld64(tS + 64, b);
          ld_wait(a, b);
          if (__any_sync(0xffffffffu, kb < lo || kb + kKeys > hi)) {
            const unsigned span = hi > lo ? (unsigned)(hi - lo) : 0u;
#pragma unroll
            for (int e = 0; e < 64; ++e) {
              if ((unsigned)(kb + e - lo) >= span) a[e] = -INFINITY;
              if ((unsigned)(kb + 64 + e - lo) >= span) b[e] = -INFINITY;
            }
          }
          float m0 = a[0], m1 = b[0], m2 = a[1], m3 = b[1];
#pragma unroll
          for (int e = 2; e < 62; e += 4) {
            m0 = fmaxf(m0, fmaxf(a[e], a[e + 1])), m1 = fmaxf(m1, fmaxf(b[e], b[e + 1]));
            m2 = fmaxf(m2, fmaxf(a[e + 2], a[e + 3])), m3 = fmaxf(m3, fmaxf(b[e + 2], b[e + 3]));
          }
          m0 = fmaxf(m0, fmaxf(a[62], a[63])), m1 = fmaxf(m1, fmaxf(b[62], b[63]));
          const float top = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * p.scale_log2;
          const bool grow = top > m + 8.f;  // (m = -inf: any finite score)
          const float m_new = grow ? top : m;
          const float alpha = grow && m != -INFINITY ? ex2(m - m_new) : 1.f;
          if (done > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            if (!wait_ab(&c.o_done[x], (it - 1) & 1, flags)) flags[0] = 1;
            tc_fence_after();
#pragma unroll 1
            for (int d = 0; d < HD; d += 32) {
              float v[32];
              tmem_ld32(tmem + 256 + x * 128 + lane_off + d, v);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] *= alpha;
              tmem_st32(tmem + 256 + x * 128 + lane_off + d, v);
            }
          }
          const float off = m_new == -INFINITY ? 0.f : -m_new;
          const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), off2 = pair(off, off);
          uint64_t l0 = 0, l1 = 0;  // two sums of pairs
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float u, v;
            unpair(fma2(pair(a[2 * e], a[2 * e + 1]), scale2, off2), u, v);
            u = ex2(u), v = ex2(v);
            if (e & 1) l0 = add2(l0, pair(u, v)); else l1 = add2(l1, pair(u, v));
            pk[e] = pack_bf16(u, v);
          }
          st32(tS, pk);
          if (NT == 2) {
            st_wait();
            tc_fence_before();
            mbar_arrive(&c.p_half[x]);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float u, v;
            unpair(fma2(pair(b[2 * e], b[2 * e + 1]), scale2, off2), u, v);
            u = ex2(u), v = ex2(v);
            if (e & 1) l0 = add2(l0, pair(u, v)); else l1 = add2(l1, pair(u, v));
            pk[e] = pack_bf16(u, v);
          }
          st32(tS + 32, pk);
          st_wait();
          float lu, lv;
          unpair(add2(l0, l1), lu, lv);
          l = l * alpha + (lu + lv);
          m = m_new;
        }
        tc_fence_before();
        if (NT == 2 && !warp_valid) mbar_arrive(&c.p_half[x]);
        mbar_arrive(&c.p_full[x]);
      }
      // ---- the segment's rows
      const bool whole = q.c_lo == 0 && q.c_hi == q.nch;
      const int slot = 2 * blockIdx.x + (q.c_lo == 0 ? 1 : 0);  // partials: the unit's start, or a later part
      float w0 = 1.f, w1 = 0.f;  // weights of O 0 and O 1 in this row
      bool use1 = false;
      // this stream's O: its last P V done, hence every earlier one
      if (done > 0 && !wait_ab(&c.o_done[x], (it - 1) & 1, flags)) flags[0] = 1;
      if (NT == 1) {  // and the other's, with its (m, l)
        c.ml[x][row] = make_float2(m, l);
        named_barrier(1 + (warp & 3), 64);
        const float2 o = c.ml[x ^ 1][row];
        named_barrier(1 + (warp & 3), 64);  // read before the next segment's write
        const float M = fmaxf(m, o.x), base = M == -INFINITY ? 0.f : M;
        const float f = ex2(m - base), fo = ex2(o.x - base);
        l = l * f + o.y * fo;
        m = M;
        w0 = x == 0 ? f : fo;
        w1 = x == 0 ? fo : f;
        use1 = n > 1;
      }
      tc_fence_after();
      if (__all_sync(0xffffffffu, !flags[0]) && warp_valid) {
        // one tile: stream x writes dims [x HD / 2, + HD / 2) of both; two: its own row
        constexpr int kD = NT == 2 ? HD : HD / 2;
        const int d_lo = NT == 2 ? 0 : x * kD;
        const float inv = whole ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f;
        const int64_t gr = q.r0 + tk;
        const int gh = q.g * h.group + head;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + gr * p.out_stride + (int64_t)gh * HD + d_lo;
        const int prow = (NT == 2 ? x * 128 : 0) + row;
        if (NT == 1) w0 *= inv, w1 *= inv;
#pragma unroll 1
        for (int d = 0; d < kD; d += 32) {
          float v[32];
          if (NT == 2) {
            tmem_ld32(tmem + 256 + x * 128 + lane_off + d, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= inv;
          } else {
            tmem_ld32(tmem + 256 + lane_off + d_lo + d, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] *= w0;
            if (use1) {
              float v1[32];
              tmem_ld32(tmem + 384 + lane_off + d_lo + d, v1);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = fmaf(v1[e], w1, v[e]);
            }
          }
          if (!valid) continue;
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint32_t w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) w[k] = pack_bf16(v[e + 2 * k], v[e + 2 * k + 1]);
              put32(dst + d + e, w, p.wide_out);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(v[e + k]);
              put32(part_row(wk, slot, prow, NT * 128, HD) + d_lo + d + e, w, true);
            }
          }
        }
        if (valid && (NT == 2 || x == 0)) {
          if (!whole)
            __stcg(wk.ml + (int64_t)slot * (NT * 128) + prow, make_float2(m, l));
          else if (p.lse)
            p.lse[gr * p.nh + gh] = lse_of(m, l);
        }
      }
      if (t == 0 && q.c_lo == 0 && !whole) {  // the unit starts here and goes on in the next CTAs
        const long long end = walk.hi - (q.c_hi - 1) + q.nch - 1;  // past its last slot: slot hi - 1 is chunk c_hi - 1
        const int G = (int)min((long long)gridDim.x, W);
        const int last = (int)((end * G + W - 1) / W) - 1;
        wk.meta[blockIdx.x] = make_int4(last - (int)blockIdx.x + 1, q.r0 + q.t0, min(h.TT, q.n - q.t0), q.g);
      }
      tc_fence_before();
      mbar_arrive(&c.o_free[NT == 2 ? x : 0]);
      q = nq;
      have = more;
      ++seg;
    }
    if (flags[0]) {
      if (t == 0 && p.status) atomicOr(p.status, DFLASH_DEV_TIMEOUT);
      for (int k = 0; k < 2000; ++k) __nanosleep(1000);  // copies still in flight land first
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Merges the partials of the unit that starts in CTA b = blockIdx.x and ends in a later one, in
// key order.  A warp has a row (lane: HD / 32 dims); of a unit cut into more than 8 parts (few
// sequences, long contexts) the block's 8 warps share a row's parts and meet in shared memory, so
// that no warp waits for one batch of loads after another.  Bound by issue and latency: two parts
// taken as two instead of eight with six empty, and no division or lookup of the unit, brought a prompt
// of 8192 from 516 to 499 us and 32 blocks of 16 from 67 to 64.
template <int HD, int NT>
__global__ void __launch_bounds__(256) attend_combine_kernel(const AttendParams p, const AttendWork wk) {
  constexpr int kD = HD / 32;  // dims of a lane: 4 or 2
  __shared__ float s_o[8][HD];
  __shared__ float2 s_ml[8];
  pdl_trigger();
  pdl_wait();
  const int4 meta = wk.meta[blockIdx.x];
  const int nsplit = meta.x;
  if (nsplit == 0) return;
  const Shape h = shape_of(p, NT);
  const int n = meta.z, g = meta.w;  // tokens of the unit
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = n > h.T ? 2 : 1;  // query tiles with tokens
  const bool shared = nsplit > 8;
  const int rows = shared ? 1 : 8;                      // of the block at a time
  for (int base = blockIdx.y * rows; base < tiles * 128; base += gridDim.y * rows) {
    const int row = shared ? base : base + warp;
    const int x = row >> 7, tok = (row & 127) * p.inv >> 16, head = (row & 127) - tok * h.group;
    const int tk = x * h.T + tok;
    const bool valid = tok < h.T && tk < n;
    if (!valid) continue;  // (shared: the whole block has the same row)
    float M = -INFINITY, L = 0.f, acc[kD];
#pragma unroll
    for (int d = 0; d < kD; ++d) acc[d] = 0.f;
    auto merge = [&](auto parts, int q0, int step) {  // parts q0, q0 + step, ...: all loads ahead of the sums
      constexpr int N = decltype(parts)::value;
      float2 ml[N];
      float o[N][kD];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const int q = q0 + u * step, slot = 2 * (blockIdx.x + q) + (q == 0 ? 1 : 0);
        ml[u] = make_float2(-INFINITY, 0.f);
        if (q < nsplit) {
          ml[u] = __ldcg(wk.ml + (int64_t)slot * (NT * 128) + row);
          const float* src = part_row(wk, slot, row, NT * 128, HD) + lane * kD;
          if (kD == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
            o[u][0] = v.x, o[u][1] = v.y, o[u][kD - 2] = v.z, o[u][kD - 1] = v.w;
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
            o[u][0] = v.x, o[u][1] = v.y;
          }
        } else {
#pragma unroll
          for (int d = 0; d < kD; ++d) o[u][d] = 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const float Mn = fmaxf(M, ml[u].x), z = Mn == -INFINITY ? 0.f : Mn;
        const float f = exp2f(M - z), fu = exp2f(ml[u].x - z);
#pragma unroll
        for (int d = 0; d < kD; ++d) acc[d] = acc[d] * f + o[u][d] * fu;
        L = L * f + ml[u].y * fu;
        M = Mn;
      }
    };
    if (nsplit == 2)  // most units
      merge(std::integral_constant<int, 2>{}, 0, 1);
    else
      for (int q0 = shared ? warp : 0; q0 < nsplit; q0 += shared ? 64 : 8) merge(std::integral_constant<int, 8>{}, q0, shared ? 8 : 1);
    if (shared) {
#pragma unroll
      for (int d = 0; d < kD; ++d) s_o[warp][lane * kD + d] = acc[d];
      if (lane == 0) s_ml[warp] = make_float2(M, L);
      __syncthreads();
      if (warp == 0) {
        float m2[8], z = -INFINITY;
#pragma unroll
        for (int w = 0; w < 8; ++w) z = fmaxf(z, s_ml[w].x);
        M = z;
        z = z == -INFINITY ? 0.f : z;
        L = 0.f;
#pragma unroll
        for (int d = 0; d < kD; ++d) acc[d] = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          m2[w] = exp2f(s_ml[w].x - z);
          L += s_ml[w].y * m2[w];
#pragma unroll
          for (int d = 0; d < kD; ++d) acc[d] += s_o[w][lane * kD + d] * m2[w];
        }
      }
    }
    if (!shared || warp == 0) {
      const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
      const int64_t gr = meta.y + tk;
      const int gh = g * h.group + head;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + gr * p.out_stride + (int64_t)gh * HD + lane * kD;
      if (kD == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[kD - 2] * inv, acc[kD - 1] * inv));
      else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16(acc[0] * inv, acc[1] * inv);
      if (p.lse && lane == 0) p.lse[gr * p.nh + gh] = lse_of(M, L);
    }
    if (shared) __syncthreads();
  }
}

template <int HD, int NT>
cudaError_t launch(const AttendParams& p, const AttendWork& w, int sms, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  if (cudaError_t e = smem_attr_once(attend_tc_kernel<HD, NT>, Cfg<HD, NT>::kSmem, attr); e != cudaSuccess) return e;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(sms);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = Cfg<HD, NT>::kSmem;
  c.stream = st;
  c.attrs = a;
  c.numAttrs = 1;
  CUtensorMap q_map;
  if (!make_tmap_heads_bf16(&q_map, p.q, p.n_rows, p.nh, HD, p.q_stride, p.group, p.tokens)) return cudaErrorInvalidValue;
  if (cudaError_t e = cudaLaunchKernelEx(&c, attend_tc_kernel<HD, NT>, p, w, q_map); e != cudaSuccess) return e;
  c.gridDim = dim3(sms, NT * 16);  // a unit's rows in one round
  c.blockDim = dim3(256);
  c.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&c, attend_combine_kernel<HD, NT>, p, w);
}

}  // namespace

int64_t attend_tc_workspace(int head_dim, int sms) {
  // per CTA two partial slots of 256 rows: O, (m, l); and the split unit's place
  return (int64_t)sms * (2 * 256 * (head_dim * 4 + 8) + 16);
}

cudaError_t launch_attend_tc(const AttendParams& p, int head_dim, int max_new, void* workspace, int sms, cudaStream_t st) {
  AttendWork w;
  w.o = static_cast<float*>(workspace);
  w.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + (int64_t)sms * 2 * 256 * head_dim * 4);
  w.meta = reinterpret_cast<int4*>(w.ml + (int64_t)sms * 2 * 256);
  const int T = p.tokens;
  // Chunks longer than one tile: two tiles share every K/V slot, where there are units enough for the
  // SMs.  Measured (32 query heads on 4, one tile / two): 32 sequences x 17 tokens on 4096 rows
  // 111 / 92 us, x 64 197 / 156 us, 8 x 256 on 2048 117 / 100 us, 64 x 20 on 500 66 / 51 us; with few
  // units the split finer in queries wins: 4 x 32 on 8192 43 / 66 us, 1 x 32 on 30000 55 / 61 us.  The
  // same way round with heads of 64, with 64 on 8 and under a window; 8 on 8 lose 4 of 51 us by it
  // (8 x 256 on 2048).
  const bool two = max_new > T && ((int64_t)p.n_rows + T - 1) / T * p.nkv * 2 >= sms;
  w.long_chunks = max_new > 4 * (two ? 2 * T : T);
  if (head_dim == 128) return two ? launch<128, 2>(p, w, sms, st) : launch<128, 1>(p, w, sms, st);
  return two ? launch<64, 2>(p, w, sms, st) : launch<64, 1>(p, w, sms, st);
}

}  // namespace dflash
