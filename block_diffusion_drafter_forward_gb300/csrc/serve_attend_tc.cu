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
// Trees (kTree): the sequence's own rows are seen by a mask per row, the context by the window; the units' chunks
// go to the sequence's end.  32 trees of 33-64 nodes on 0.5-8 Ki rows 155 us (34 % of the tensor pipe: part-full
// tiles, and a unit of 33-48 nodes has one stream at work); one of 32 nodes on 4096 rows 19 us, latency.
//
// Pages in 8 bits (kQuant): see below.  32 blocks of 16 as above 85 us, 4 of 32 on 8 Ki rows 48, 32 of 64 on 4 Ki rows 177,
// a prompt of 8192 600 us; before the widening looked for NaN 86, 45, 164 and 580, and as such measured: with one tile a chunk
// takes a CTA 1.87 us; without the widening 1.35, without its stores 1.51, K or V alone 1.6, with one of four
// softmax warps at work 1.77: the 64 KB that are written to shared memory, beside the 96 KB that the MMAs read of
// it, and the instruction caches hold it (its loops unrolled: 2.5 us; codes read ahead of the step before: 2.05;
// two threads a query row in loops of 32 columns: 1.82, but with two tiles 680 us for the prompt).  The search in a
// warp of its own beside the widening ones, which then waits for the stages too: 99 and 670 us.
//
// Rounding: P is bf16 (the MMA's operand type), sums and O fp32, the normaliser sums the fp32 P.
// Warp roles: 0-3 stream 0, 4-7 stream 1, 8 K pages, 10 V pages, 9 and 11 MMA issue (8 bits: 8 pages, 10 the next
// segment's queries, 12-15 widening).  The V warp
// also zeroes the key rows behind a sequence's end in its last page (never-written rows may hold
// NaN, and 0 * NaN would reach O; their scores are masked by select).  Issuing an MMA blocks its
// thread while the tensor pipe's queue is full, so with two tiles each stream has a warp of its own
// (one that issued for both left the pipe idle between the streams: 614 against 564 us for a prompt
// of 8192); with one tile a single thread keeps the chunks in order over both streams.
#include <float.h>

#include <atomic>
#include <type_traits>

#include "launch_util.cuh"
#include "serve_attend_plan.cuh"
#include "tc_common.cuh"

namespace dflash {
namespace {

using namespace tc;
using plan::PlanCtl;
using plan::Seg;
using plan::Shape;
using plan::mask_bits;
using plan::shape_of;

constexpr int kKeys = 128;                      // keys per chunk
constexpr int kPages = kKeys / kPage;           // 8
template <bool kQuant>
struct Geo {
  static constexpr int kKeys = 128, kUnitCost = 3, kTwo = kQuant ? 1 : 3, kOne = kQuant ? 1 : 2, kThreads = kQuant ? 512 : 384;
};

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

template <int HD, int NT, bool kQuant>
struct Cfg {
  static constexpr int kTiles = NT;                    // query tiles of a unit
  static constexpr int kTile = kPage * HD * 2;         // a page of one head: bytes of K (or V)
  static constexpr int kQ = 128 * HD * 2;              // a query tile
  static constexpr int kSlot = kPages * kTile;         // a chunk's K (or V)
  static constexpr int kQTiles = kQuant && NT == 1 ? 1 : 2;  // queries: two tiles, or two segments' tile (8 bits: one segment's)
  static constexpr int kNK = kQuant ? (HD == 128 ? 2 : 3) : HD == 128 ? 3 : 6;  // K and V slots in flight
  static constexpr int kNV = kQuant ? (HD == 128 ? 2 : 3) : HD == 128 ? 2 : 6;
  // 8 bits: halves of a chunk as they are in the pages
  static constexpr int kCodes = 32 * HD + 32;          // a page of one head
  static constexpr int kNS = !kQuant ? 1 : HD == 64 ? 6 : NT == 1 ? 4 : 2;
  static constexpr int kHalf = kQuant ? kPages / 2 * kCodes : 0;
  static constexpr int kCtl = kQuant && HD == 128 ? 2560 : 2944;    // barriers, plan, row exchange
  static constexpr int kSmem = kQTiles * kQ + (kNK + kNV) * kSlot + kNS * kHalf + kCtl;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};

template <class C, class G, class Walk>
struct Ctl {
  uint64_t k_full[C::kNK], k_empty[C::kNK], v_full[C::kNV], v_empty[C::kNV], v_raw[C::kNV];
  uint64_t st_full[C::kNS], st_empty[C::kNS];
  int2 half[C::kNS];  // pages of the half, rows of the sequence from its first on
  uint64_t s_full[2], p_half[2], p_full[2], o_done[2], o_free[2], q_full[2], q_empty;
  uint32_t tmem_slot;
  int flags[2];  // a wait gave up; a NaN was met in pages of 8 bits
  Walk walk;     // (8 bits: this CTA's, for those)
  PlanCtl<G> plan;
  float2 ml[2][128];  // one tile: the streams' (m, l) of every row
};

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

// The chunks of stream x, in order, as every role counts them.
template <int NT, class Walk>
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

// ---- Pages in 8 bits.  A chunk comes as two halves of four pages (K and V codes and their exponents, one copy a
// page), and four warps write its values as bf16 into the K and V slots, in the layout that pages of
// bf16 have: two for K, which is wanted first, and two for V.

// A warp's wait: its lanes go on, or give up, together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, wait_ab(bar, parity, abort));
}

// Warp 8: lane l copies page l of a half.  Every half of every chunk has its turn, those without pages too; what the
// widening warps have to know of it lies beside its barrier, so that they need no walk of their own (its
// registers would spill, and local memory has next to no L1 beside 227 KB of shared memory).
template <class C, class Walk, class Ctl>
__device__ __forceinline__ void load_codes(const AttendParams& p, const Shape& h, const Walk& walk, uint8_t* stage, Ctl& c, int lane) {
  volatile int* flags = c.flags;
  Walk w = walk;
  Seg q;
  int i = 0;  // halves so far
  while (w.next(p, h, q)) {
    const int pages = (q.kv + kPage - 1) / kPage;
    const int first = q.k0 / kPage + q.c_lo * kPages, end = q.k0 / kPage + q.c_hi * kPages;
    const int32_t* table = p.page_tables + (int64_t)q.s * p.mpps;
    auto fetch = [&](int lp) { return lane < kPages / 2 && lp < min(end, pages) ? __ldg(table + lp) : 0; };
    int page = fetch(first + lane);
    for (int lp = first; lp < end; lp += kPages / 2, ++i) {
      const int b = i % C::kNS, n = max(0, min(kPages / 2, pages - lp));
      if (i >= C::kNS && !warp_wait(&c.st_empty[b], (i / C::kNS - 1) & 1, flags)) return;
      if (lane == 0) {
        c.half[b] = make_int2(n, q.kv - lp * kPage);  // pages, rows from its first on
        mbar_arrive_expect_tx(&c.st_full[b], n * C::kCodes);
      }
      __syncwarp();
      if (lane < n) {
        if (page < 0 || page >= p.num_pages) {
          if (p.status) atomicOr(p.status, DFLASH_DEV_BAD_PAGE);
          page = 0;
        }
        bulk_load(stage + b * C::kHalf + lane * C::kCodes, static_cast<const uint8_t*>(p.pool) + page * p.page_stride + (int64_t)q.g * C::kCodes,
                  C::kCodes, &c.st_full[b]);
      }
      page = fetch(lp + kPages / 2 + lane);
    }
  }
  const int b = i % C::kNS;
  if (i >= C::kNS && !warp_wait(&c.st_empty[b], (i / C::kNS - 1) & 1, flags)) return;
  if (lane == 0) {
    c.half[b] = make_int2(-1, 0);  // no more
    mbar_arrive(&c.st_full[b]);
  }
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  return a;
}

// One warp's pages (pg and pg + 2) of a half, of whose rows `rows` are the sequence's.  K: a lane has dims 16 x .. of row j,
// for two x at a time.  V: rows 8 r .. of dims 32 g + m + 8 k; rows from `rows` on become zeros (they may hold
// anything, and zero times NaN would reach O).  Eight lanes write 128 bytes in a row, and read as many from
// different banks.  Two products a pair, by 2^120 and the row's power (their product is a bf16 number for rows below
// 2^15 alone; a second instance that took one product there was slower by its code: 97 us for 91).  A loop, not unrolled: the
// roles' code together is more than the instruction caches hold (both pages unrolled: 3.6 us a chunk for 2.3; the two
// steps of a page: 107 us for 90).  Not 0: one of the sequence's rows has a NaN in dims of this lane's.
template <int HD, class C, bool kV>
__device__ __forceinline__ uint32_t widen_pages(const uint8_t* half, uint8_t* dst, int pg, int n, int rows, int lane) {
  const int j = lane & 15, m = lane & 7, r = lane >> 3 & 1, up = lane >> 4;
  const uint8_t* src = half + pg * C::kCodes + (kV ? 16 * HD + up * 512 + m * 64 : j * 64);
  const int u0 = kV ? (2 * r) ^ (m >> 1) : up ^ (j >> 1 & 3);  // the first unit of 16 bytes; the other differs in bit 0 (V), 1 (K)
  const uint8_t* ex = half + pg * C::kCodes + 32 * HD + (kV ? 16 + 8 * r : j);
  uint32_t nan = 0;
  dst += pg * C::kTile + (kV ? m * 16 + r * 128 + up * 1024 : r * (HD * 16) + m * 16 + up * 256);
  for (; pg < n; pg += 2, src += 2 * C::kCodes, ex += 2 * C::kCodes, dst += 2 * C::kTile) {
    uint32_t e0, e1;
    if (kV) {
      const uint2 e = *reinterpret_cast<const uint2*>(ex);
      e0 = e.x, e1 = e.y;
    } else {
      e0 = e1 = *ex * 0x01010101u;
    }
    uint32_t d0 = 0, d1 = 0;
    if (kV && (pg + 1) * kPage > rows) {
      const int live = rows - pg * kPage - 8 * r;  // rows of the eight that are
      d0 = live <= 0 ? 0xffffffffu : live >= 4 ? 0u : 0xffffffffu << 8 * live;
      d1 = live <= 4 ? 0xffffffffu : live >= 8 ? 0u : 0xffffffffu << 8 * (live - 4);
      e0 = (e0 & ~d0) | (0x7f7f7f7fu & d0), e1 = (e1 & ~d1) | (0x7f7f7f7fu & d1);
    }
    uint32_t f[4];  // powers of two rows
#pragma unroll
    for (int k = 0; k < (kV ? 4 : 1); ++k) f[k] = __byte_perm(k < 2 ? e0 : e1, 0, k & 1 ? 0x4342 : 0x4140) << 7;  // (an exponent byte to a half)
    uint32_t met = 0;
    auto turn = [&](uint32_t a, int k) { return mul2(mul2(a, 0x7b807b80u), f[k]); };
    auto put_k = [&](uint8_t* d, uint32_t a, uint32_t b) {
      const uint2 x = plan::widen(a, met), y = plan::widen(b, met);
      *reinterpret_cast<uint4*>(d) = make_uint4(turn(x.x, 0), turn(x.y, 0), turn(y.x, 0), turn(y.y, 0));
    };
    if constexpr (!kV && C::kTiles == 1) {  // half a step at a time (32 blocks of 16 90 -> 85 us; with two tiles a prompt of 8192 603 -> 614)
#pragma unroll 1
      for (int e = 0; e < HD / 32; ++e) {
        const uint4 w = *reinterpret_cast<const uint4*>(src + (e >> 1) * 1024 + (u0 ^ (e & 1) * 2) * 16);
        put_k(dst + e * 512, w.x, w.y), put_k(dst + e * 512 + 128, w.z, w.w);
      }
    } else {
#pragma unroll 1
      for (int e = 0; e < HD / 64; ++e) {
        const uint8_t* s = src + e * 1024;
        uint4 lo = *reinterpret_cast<const uint4*>(s + u0 * 16), hi = *reinterpret_cast<const uint4*>(s + (u0 ^ (kV ? 1 : 2)) * 16);
        uint8_t* d = dst + e * (kV ? 2048 : 1024);
        if (kV) {
          if (d0 | d1) {
            lo = make_uint4(lo.x & ~d0, lo.y & ~d0, lo.z & ~d0, lo.w & ~d0);
            hi = make_uint4(hi.x & ~d1, hi.y & ~d1, hi.z & ~d1, hi.w & ~d1);
          }
          auto put = [&](uint32_t a, uint32_t b, int k) {
            const uint2 x = plan::widen(a, met), y = plan::widen(b, met);
            *reinterpret_cast<uint4*>(d + k * 256) = make_uint4(turn(x.x, 0), turn(x.y, 1), turn(y.x, 2), turn(y.y, 3));
          };
          put(lo.x, hi.x, 0), put(lo.y, hi.y, 1), put(lo.z, hi.z, 2), put(lo.w, hi.w, 3);
        } else {
          put_k(d, lo.x, lo.y), put_k(d + 128, lo.z, lo.w), put_k(d + 512, hi.x, hi.y), put_k(d + 640, hi.z, hi.w);
        }
      }
    }
    if (kV || pg * kPage + j < rows) nan |= plan::is_nan(met);  // (V behind the end: zeros by now)
  }
  return nan;
}

// Warps 12 and 13 (`sub` 0, 1): K of the halves, every second page each; 14 and 15 (2, 3): V.
template <int HD, class C, bool kV, class Ctl>
__device__ __forceinline__ void widen_codes(const uint8_t* stage, uint8_t* slots, Ctl& c, int sub, int lane) {
  volatile int* flags = c.flags;
  constexpr int kN = kV ? C::kNV : C::kNK;
  uint64_t *full = kV ? c.v_full : c.k_full, *empty = kV ? c.v_empty : c.k_empty;
#pragma unroll 1
  for (int i = 0;; ++i) {
    const int b = i % C::kNS, kc = i >> 1, half = i & 1, slot = kc % kN;
    if (!warp_wait(&c.st_full[b], (i / C::kNS) & 1, flags)) return;
    const int n = c.half[b].x, rows = c.half[b].y;
    if (n < 0) return;
    if (half == 0 && kc >= kN && !warp_wait(&empty[slot], (kc / kN - 1) & 1, flags)) return;
    uint8_t* dst = slots + slot * C::kSlot + half * (kPages / 2) * C::kTile;
    const uint8_t* src = stage + b * C::kHalf;
    if (widen_pages<HD, C, kV>(src, dst, sub & 1, n, rows, lane)) flags[1] = 1;
    if (kV && half == 0 && n == 0 && (sub & 1) == 0) {  // a unit without keys: a page of zeros
      for (int e = lane; e < C::kTile / 16; e += 32) reinterpret_cast<uint4*>(dst)[e] = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&full[slot]);
      mbar_arrive(&c.st_empty[b]);  // (not before what was read has been used)
    }
  }
}

// NaN in K or V, given to the rows that see one, for all of a CTA's segments when they are done (beside each segment's end its
// code cost the softmax loops: a prompt of 8192 20 us).  The softmax warps; a thread has the row and dims that it wrote.
template <int HD, int NT, bool kTree, class Walk>
__device__ __noinline__ void spread_nan_tc(const AttendParams& p, const AttendWork& wk, Walk w) {
  constexpr int kD = NT == 2 ? HD : HD / 2;
  const int x = threadIdx.x >> 7, row = threadIdx.x & 127, prow = (NT == 2 ? x * 128 : 0) + row;
  const Shape h = shape_of(p, NT);
  const int tok = row / h.group, head = row - tok * h.group;
  Seg q;
  while (w.next(p, h, q)) {
    const int tk = q.t0 + (NT == 2 ? x * h.T : 0) + tok, gh = q.g * h.group + head, slot = 2 * blockIdx.x + (q.c_lo == 0 ? 1 : 0);
    const int64_t gr = q.r0 + tk;
    const bool whole = q.c_lo == 0 && q.c_hi == q.nch, first = NT == 2 || x == 0;
    plan::spread_nan<HD, kTree>(p, q, q.k0 + q.c_lo * kKeys, min(q.kv, q.k0 + q.c_hi * kKeys), tok < h.T && tk < q.n ? tk : -1,
                                NT == 2 ? 0 : x * kD, kD, HD, whole ? static_cast<__nv_bfloat16*>(p.out) + gr * p.out_stride + (int64_t)gh * HD : nullptr,
                                part_row(wk, slot, prow, NT * 128, HD), first && whole && p.lse ? p.lse + gr * p.nh + gh : nullptr,
                                first && !whole ? wk.ml + (int64_t)slot * (NT * 128) + prow : nullptr);
  }
}

template <int HD, int NT, bool kTree, bool kQuant>
__global__ void __launch_bounds__(Geo<kQuant>::kThreads, 1) attend_tc_kernel(const AttendParams p, const AttendWork wk, const __grid_constant__ CUtensorMap q_map) {
  using C = Cfg<HD, NT, kQuant>;
  using Walk = plan::Walk<Geo<kQuant>, kTree>;
  constexpr int kThreads = Geo<kQuant>::kThreads;
  static_assert(sizeof(Ctl<C, Geo<kQuant>, Walk>) <= C::kCtl, "control block overflows its slot");
  extern __shared__ __align__(1024) uint8_t smem[];  // (the queries' swizzle counts from 1 KB boundaries)
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + C::kQTiles * C::kQ;
  uint8_t* sV = sK + C::kNK * C::kSlot;
  uint8_t* sS = sV + C::kNV * C::kSlot;  // 8 bits: halves of chunks
  auto& c = *reinterpret_cast<Ctl<C, Geo<kQuant>, Walk>*>(sS + (kQuant ? C::kNS * C::kHalf : 0));
  volatile int* flags = c.flags;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const Shape h = shape_of(p, NT);

  pdl_wait();  // everything read here may come from the kernel before
  if (t == 0) wk.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
  long long W;
  const Walk walk = plan::make<Geo<kQuant>, kTree>(p, h, c.plan, reinterpret_cast<long long*>(sK), wk.long_chunks, &W);
  if (walk.lo >= walk.hi) {  // nothing for this CTA
    pdl_trigger();
    return;
  }
  if (t == 0) {
    for (int i = 0; i < C::kNK; ++i) {
      mbar_init(&c.k_full[i], kQuant ? 4 : 1);  // (8 bits: two warps, two halves)
      mbar_init(&c.k_empty[i], NT);
    }
    for (int i = 0; i < C::kNV; ++i) {
      mbar_init(&c.v_full[i], kQuant ? 4 : 1);
      mbar_init(&c.v_empty[i], NT);
      mbar_init(&c.v_raw[i], 1);
    }
    for (int i = 0; i < C::kNS; ++i) {
      mbar_init(&c.st_full[i], 1);
      mbar_init(&c.st_empty[i], 4);
    }
    mbar_init(&c.q_empty, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.s_full[i], 1);
      mbar_init(&c.p_half[i], 128);
      mbar_init(&c.p_full[i], 128);
      mbar_init(&c.o_done[i], 1);
      mbar_init(&c.o_free[i], NT == 2 ? 128 : 256);
      mbar_init(&c.q_full[i], 1);
    }
    flags[0] = flags[1] = 0;
    if (kQuant) c.walk = walk;
    fence_barrier_init();
  }
  // rows that no query fills stay finite
  if (h.group * h.T < 128)
    for (int i = t; i < C::kQTiles * C::kQ / 16; i += kThreads) reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();  // the plan's scratch is overwritten by copies
  if (warp == 0) tmem_alloc(&c.tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem_slot;
  pdl_trigger();
  // A unit that starts here and goes on in the next CTAs; end: behind the first slot of its last chunk.
  auto goes_on = [&](const Seg& q, long long end) {
    const int G = plan::ctas_of<Geo<kQuant>, kTree>(h, W), last = (int)((end * G + W - 1) / W) - 1;
    wk.meta[blockIdx.x] = make_int4(last - (int)blockIdx.x + 1, q.r0 + q.t0, min(h.TT, q.n - q.t0), q.g);
  };
  // Queries of a segment into tile b (its second query tile's: two tiles, b = 1) by TMA: rows of 64
  // dims in the 128-byte swizzle, (head, token) in the tile's row order.  One thread.  (Copied by the
  // softmax threads, 16 bytes each, they queued for thousands of cycles behind the pages.)
  auto load_q = [&](const Seg& q, int b) {
    mbar_arrive_expect_tx(&c.q_full[b], h.group * h.T * HD * 2);
    for (int d = 0; d < HD / 64; ++d)
      tma_load_3d(sQ + b * C::kQ + d * (128 * 128), &q_map, &c.q_full[b], d * 64, q.g * h.group, q.r0 + q.t0 + (NT == 2 ? b * h.T : 0));
  };

  if (warp >= 8) {
    if (kQuant)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");  // (of 128 at launch: 8 warps with 192, 8 with 64)
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if constexpr (kQuant) {
      if (warp == 8) {
        load_codes<C>(p, h, walk, sS, c, lane);
      } else if (warp >= 12) {
        warp < 14 ? widen_codes<HD, C, false>(sS, sK, c, warp - 12, lane) : widen_codes<HD, C, true>(sS, sV, c, warp - 12, lane);
      } else if (NT == 1 && warp == 10 && lane == 0) {
        // queries of one segment at a time: once the last S of the one before is done
        Walk w = walk;
        Seg q;
        for (int i = 0; w.next(p, h, q); ++i) {
          if (i > 0 && !wait_ab(&c.q_empty, (i - 1) & 1, flags)) break;
          load_q(q, 0);
        }
      }
    }
    if (!kQuant && (warp == 8 || warp == 10)) {
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
    } else if (lane == 0 && (!kQuant || warp == 9 || warp == 11)) {
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
          // (here, where the walk is at hand: what the softmax warps keep beside their loop costs 3 % of a tree's time)
          if (kTree && x == 0 && q.c_lo == 0 && q.c_hi < q.nch) goes_on(q, w.pu - plan::chunk_slots<Geo<kQuant>, kTree>(h, q.n, q.tile) + 1);
          if (!It<NT, Walk>::active(h, q, x)) {
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
      } else if constexpr (kQuant) {
        // One tile, a warp a stream: chunks j of its parity.  A wait by parity is exact only while the phase before is
        // known complete and the next one is not.  The next one needs this warp (S, P V or q_empty).  The one
        // before: q_full of a segment says that every S before it is done, hence every K loaded (K and V come in
        // order); K of a chunk says that V kNV chunks earlier is in its slot (its half had to be free); O is
        // counted by the stream's own segments.
        static_assert(NT == 2 || C::kNS == 2 * C::kNV, "K of a chunk tells of V kNV chunks earlier");
        const int x = warp == 9 ? 0 : 1;
        Walk w = walk;
        Seg q;
        int it = 0, act = 0, kc0 = 0;  // chunks and segments of this stream; chunks of the segments before
        auto wait = [&](uint64_t* bar, int phase) {
          if (!wait_ab(bar, phase & 1, flags)) flags[0] = 1;  // after a timeout: commits only, no MMAs
        };
        for (int seg = 0; w.next(p, h, q); ++seg) {
          const int n = q.c_hi - q.c_lo;
          wait(&c.q_full[0], seg);
          auto s_of = [&](int j) {
            const int kc = kc0 + j, kb = kc % C::kNK;
            wait(&c.k_full[kb], kc / C::kNK);
            tc_fence_after();
            if (!flags[0]) issue_s(x, 0, kb);
            mma_commit(&c.s_full[x]);
            mma_commit(&c.k_empty[kb]);
            if (j + 2 >= n) mma_commit(&c.q_empty);  // this stream's last
          };
          if (x < n)
            s_of(x);
          else
            mbar_arrive(&c.q_empty);
          for (int j = x; j < n; j += 2, ++it) {
            const int kc = kc0 + j, vb = kc % C::kNV;
            const int np = max(1, min(kPages, (q.kv - q.k0 - (q.c_lo + j) * kKeys + kPage - 1) / kPage));
            wait(&c.v_full[vb], kc / C::kNV);
            if (j == x && act > 0) wait(&c.o_free[x], act - 1);
            wait(&c.p_half[x], it);
            tc_fence_after();
            if (!flags[0]) issue_pv(x, vb, 0, min(np, kPages / 2), j > x);
            wait(&c.p_full[x], it);
            tc_fence_after();
            if (!flags[0]) issue_pv(x, vb, kPages / 2, np, true);
            mma_commit(&c.o_done[x]);
            mma_commit(&c.v_empty[vb]);
            if (j + 2 < n) s_of(j + 2);
          }
          if (x < n) ++act;
          kc0 += n;
        }
      } else if (warp == 9) {
        // both streams: each alternates S and P V; whichever is ready goes out
        It<NT, Walk> its[2];
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
            It<NT, Walk>& a = its[x];
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
    if (kQuant)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---- softmax streams: thread = query row `row` of its tile
    const int x = warp >> 2, row = t & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + x * 128 + lane_off;
    const int tok = row / h.group, head = row - tok * h.group;  // (by p.inv the loop's registers fall worse: 519 us for 499)
    const bool loads = (t & 127) == 0 && (NT == 2 || (x == 0 && !kQuant));  // (one tile: stream 0's, a segment ahead)
    Walk w = walk;
    Seg q, nq;
    bool have = w.next(p, h, q);
    while (NT == 2 && have && !It<NT, Walk>::active(h, q, x)) have = w.next(p, h, q);
    if (have && loads) load_q(q, x);
    int it = 0, seg = 0;  // chunks and segments done by this stream
    while (have) {
      bool more = w.next(p, h, nq);
      while (NT == 2 && more && !It<NT, Walk>::active(h, nq, x)) more = w.next(p, h, nq);
      const int n = q.c_hi - q.c_lo;
      const int tk = q.t0 + (NT == 2 ? x * h.T : 0) + tok;
      const bool valid = tok < h.T && tk < q.n;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      // keys [lo, hi) are seen by this row (rows without a token: anything, they are not written)
      // (trees: keys [lo, hi) of the context, and those of the sequence's own rows that the mask has)
      const int pos = !kTree ? q.kv - q.n + tk : valid && p.window > 0 ? max(q.kv - q.n, __ldg(p.positions + q.r0 + tk)) : 0;
      const int hi = !valid ? INT_MAX : kTree ? q.kv - q.n : p.causal ? min(q.kv, pos + 1) : q.kv;
      const int lo = valid && p.window > 0 ? max(0, kTree ? min(q.kv - q.n, pos - p.window + 1) : pos - p.window + 1) : 0;
      const uint32_t* mask = kTree ? reinterpret_cast<const uint32_t*>(p.masks + (int64_t)(q.r0 + (valid ? tk : 0)) * p.words) : nullptr;
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
          if (kTree && __any_sync(0xffffffffu, kb < lo || kb + kKeys > hi)) {
            uint32_t mk[4];  // bit e of word w: key kb + 32 w + e is seen
#pragma unroll
            for (int w = 0; w < 4; ++w) mk[w] = valid ? mask_bits(mask, 2 * p.words, kb + 32 * w, lo, q.kv - q.n, q.kv) : 0xffffffffu;
#pragma unroll
            for (int e = 0; e < 64; ++e) {
              if (!(mk[e >> 5] >> (e & 31) & 1)) a[e] = -INFINITY;
              if (!(mk[2 + (e >> 5)] >> (e & 31) & 1)) b[e] = -INFINITY;
            }
          }
          if (!kTree && __any_sync(0xffffffffu, kb < lo || kb + kKeys > hi)) {
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
          if (NT == 2 || kQuant) {
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
        if ((NT == 2 || kQuant) && !warp_valid) mbar_arrive(&c.p_half[x]);
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
      if (!(kTree && NT == 2) && t == 0 && q.c_lo == 0 && !whole) {
        goes_on(q, walk.hi + q.nch - q.c_hi);  // (slot hi - 1: chunk c_hi - 1)
      }
      tc_fence_before();
      mbar_arrive(&c.o_free[NT == 2 ? x : 0]);
      if (NT == 1 && kQuant && n > 1) mbar_arrive(&c.o_free[1]);  // (each stream's warp counts the segments that it works in)
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
  if constexpr (kQuant) {
    if (warp < 8 && flags[1] && !flags[0]) spread_nan_tc<HD, NT, kTree>(AttendParams(p), AttendWork(wk), c.walk);
  }
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
  // (where the caller's form allows: by the rounds of loads that either way waits for)
  const int filled = min(n, h.T) * h.group;  // rows of a query tile
  const bool shared = nsplit > 8 && !(wk.spread && (filled * tiles + gridDim.y - 1) / gridDim.y * ((nsplit + 63) / 64) >= (nsplit + 7) / 8);
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
cudaError_t combine(const AttendParams& p, const AttendWork& w, int sms, cudaStream_t st) {
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(sms, NT * 16);  // a unit's rows in one round
  c.blockDim = dim3(256);
  c.stream = st;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, attend_combine_kernel<HD, NT>, p, w);
}

template <int HD, int NT, bool kTree, bool kQuant>
cudaError_t launch(const AttendParams& p, const AttendWork& w, int sms, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  if (cudaError_t e = smem_attr_once(attend_tc_kernel<HD, NT, kTree, kQuant>, Cfg<HD, NT, kQuant>::kSmem, attr); e != cudaSuccess) return e;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(sms);
  c.blockDim = dim3(Geo<kQuant>::kThreads);
  c.dynamicSmemBytes = Cfg<HD, NT, kQuant>::kSmem;
  c.stream = st;
  c.attrs = a;
  c.numAttrs = 1;
  CUtensorMap q_map;
  if (!make_tmap_heads_bf16(&q_map, p.q, p.n_rows, p.nh, HD, p.q_stride, p.group, p.tokens)) return cudaErrorInvalidValue;
  if (cudaError_t e = cudaLaunchKernelEx(&c, attend_tc_kernel<HD, NT, kTree, kQuant>, p, w, q_map); e != cudaSuccess) return e;
  return combine<HD, NT>(p, w, sms, st);
}

template <bool kTree, bool kQuant>
cudaError_t launch_form(const AttendParams& p, const AttendWork& w, int head_dim, bool two, int sms, cudaStream_t st) {
  if (head_dim == 128) return two ? launch<128, 2, kTree, kQuant>(p, w, sms, st) : launch<128, 1, kTree, kQuant>(p, w, sms, st);
  return two ? launch<64, 2, kTree, kQuant>(p, w, sms, st) : launch<64, 1, kTree, kQuant>(p, w, sms, st);
}

}  // namespace

int64_t attend_tc_workspace(int head_dim, int sms) {
  // per CTA two partial slots of 256 rows: O, (m, l); and the split unit's place
  return (int64_t)sms * (2 * 256 * (head_dim * 4 + 8) + 16);
}

AttendWork attend_work(void* workspace, int head_dim, int sms, bool long_chunks) {
  AttendWork w;
  w.o = static_cast<float*>(workspace);
  w.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + (int64_t)sms * 2 * 256 * head_dim * 4);
  w.meta = reinterpret_cast<int4*>(w.ml + (int64_t)sms * 2 * 256);
  w.long_chunks = long_chunks;
  w.spread = 0;
  return w;
}

cudaError_t launch_attend_combine(const AttendParams& p, const AttendWork& w, int head_dim, int sms, cudaStream_t st) {
  return head_dim == 128 ? combine<128, 1>(p, w, sms, st) : combine<64, 1>(p, w, sms, st);
}

cudaError_t launch_attend_tc(const AttendParams& p, int head_dim, int max_new, void* workspace, int sms, cudaStream_t st) {
  AttendWork w = attend_work(workspace, head_dim, sms, false);
  const int T = p.tokens;
  // Chunks longer than one tile: two tiles share every K/V slot, where there are units enough for the
  // SMs.  Measured (32 query heads on 4, one tile / two): 32 sequences x 17 tokens on 4096 rows
  // 111 / 92 us, x 64 197 / 156 us, 8 x 256 on 2048 117 / 100 us, 64 x 20 on 500 66 / 51 us; with few
  // units the split finer in queries wins: 4 x 32 on 8192 43 / 66 us, 1 x 32 on 30000 55 / 61 us.  The
  // same way round with heads of 64, with 64 on 8 and under a window; 8 on 8 lose 4 of 51 us by it
  // (8 x 256 on 2048).  Trees: 32 x 17 on 4096 104 / 81 us, 32 x 64 188 / 150, 8 x 256 on 2048 115 / 97, and
  // over 8-bit pages 164 / 96, 309 / 182, 193 / 115; 8-bit chunks 32 x 17 151 / 94, 32 x 64 284 / 177, 8 x 256 169 / 105.
  const bool two = max_new > T && ((int64_t)p.n_rows + T - 1) / T * p.nkv * 2 >= sms;
  w.long_chunks = max_new > 4 * (two ? 2 * T : T);
  w.spread = p.masks || p.quant;
  if (p.quant) return p.masks ? launch_form<true, true>(p, w, head_dim, two, sms, st) : launch_form<false, true>(p, w, head_dim, two, sms, st);
  return p.masks ? launch_form<true, false>(p, w, head_dim, two, sms, st) : launch_form<false, false>(p, w, head_dim, two, sms, st);
}

}  // namespace dflash
