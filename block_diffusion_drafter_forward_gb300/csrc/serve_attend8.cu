// dflash_attend over pages in 8 bits, for units of at most 16 query rows (single tokens, and two or a few
// tokens of small head groups): HBM-bound, so every byte of a page is loaded once and the work per key is
// kept below the time of its bytes.
//
// A unit is (sequence, tile of 16 / group tokens, kv head); its query rows are the 16 rows of an m16n8k16
// matrix product.  Chunks of keys are spread over the CTAs as in the other form (serve_attend_plan.cuh).
// In a CTA each of 11 warps has its own ring of pages (K, V and exponents of 16 rows: one bulk copy)
// and its own running maximum, sum and O, so that no warp waits for another before the segment ends:
//   S[16, 16 keys] = Q K^T, softmax over the lane's four keys of two rows, O += P V.
// tcgen05 has nothing to give here: its smallest tile is 128 rows, of which a single token fills 8 or 16, and
// its operands would have to go through shared memory once more as 16 bits.
//
// S takes Q and the codes of K as f16 numbers, both exact: Q is scaled by 2^(14 - e) with the row's largest
// magnitude in [2^e, 2^(e+1)) (its eight bits fit; exact down to 2^-31 of the largest, below that to
// 2^-38 of it), a code is an f16 number (one conversion for two).
// V is multiplied in bf16, since P needs more range than f16 has: a code becomes a bf16 number by moving its bits -
// sign, exponent and mantissa << 4 is the code's value times 2^-120 exactly, subnormals included, three
// instructions for two.  Nothing multiplies that factor and the rows' powers of two into the codes: the
// scores are scaled by 2^ke per key, P by 2^(ve - r + 90) per key before it is rounded to bf16 (exact but for
// that rounding), and O is kept in units of 2^(r + 30), r the largest exponent ve of the pages so far, or up to
// 20 below it.
//
// Codes of NaN: K's conversion keeps them and a row's scores tell; V's moved bits do not, so that the largest are kept
// and looked at (147 us without).
//
// Measured (GB300; 16 tokens on 16-32 Ki rows, 64 heads on 8): 152 us, 5.3 TB/s, of which copies alone take 135; a further
// 128 keys of every CTA take 0.84 us, 88 % of the copy rate, and 13 us are start, split and merge.  K in bf16 as V: 163 us.
// K in e4m3 products with Q as two e4m3 parts: 204 us.  7 warps: 163 us; two pages a step: 152 us.  One token on 4096 rows
// 12.2 us: latency.  What bounds it is issue (1.8 instructions a cycle of 4, the ALU pipe at half its rate) beside HBM.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "launch_util.cuh"
#include "serve_attend_plan.cuh"
#include "tc_common.cuh"

namespace dflash {
namespace {

using namespace tc;
using plan::PlanCtl;
using plan::Seg;
using plan::Shape;

constexpr int kW = 11;  // warps with pages of their own (12 with the producer's: 168 registers a thread)
struct Geo {
  static constexpr int kKeys = 16 * kW, kUnitCost = 2, kTwo = 1, kOne = 1, kThreads = 32 * (kW + 1);
};
template <bool kTree> using Walk = plan::Walk<Geo, kTree>;

template <int HD>
struct Cfg {
  static constexpr int kBytes = 32 * HD + 32;                       // a page of one head
  static constexpr int kStages = HD == 128 ? 4 : 8;
  static constexpr int kRing = kW * kStages * kBytes;
  static constexpr int kMerge = kW * 16 * 32 * 4;                  // 32 dims of every warp's O
};

template <int HD, bool kTree>
struct Ctl {
  uint64_t full[kW][Cfg<HD>::kStages], empty[kW][Cfg<HD>::kStages];
  int flags[2];  // a wait gave up; a NaN was met in V
  Walk<kTree> walk;
  PlanCtl<Geo> plan;
  float2 ml[kW][16];
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// codes 0, 1 and 2, 3 of a word as pairs of f16
__device__ __forceinline__ void halves(uint32_t w, uint32_t& a, uint32_t& b) {
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;}" : "=r"(a), "=r"(b) : "r"(w));
}
// (volatile: what was read of a page has been used when its slot is given back)
__device__ __forceinline__ void mma_bf16w(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// NaN in V, which the scores do not show, given to the rows that see one, for all of a CTA's segments when they are done.  The
// 11 warps (eight of them have something to do); a thread has the row and dims that it wrote.
template <int HD, bool kTree>
__device__ __noinline__ void spread_nan8(const AttendParams& p, const AttendWork& wk, Walk<kTree> w) {
  const int t = threadIdx.x, row = t >> 4, x = (t & 15) * 2;
  if (row >= 16) return;
  Shape h;
  h.group = p.group, h.T = h.TT = p.tokens;
  const int tok = row * p.inv >> 16, head = row - tok * h.group;
  Seg q;
  while (w.next(p, h, q)) {
    const int token = q.t0 + tok;
    const bool whole = q.c_lo == 0 && q.c_hi == q.nch;
    plan::spread_nan<HD, kTree>(
        p, q, q.k0 + q.c_lo * Geo::kKeys, min(q.kv, q.k0 + q.c_hi * Geo::kKeys), tok < h.T && token < q.n ? token : -1, x, 2, 32,
        whole ? static_cast<__nv_bfloat16*>(p.out) + (int64_t)(q.r0 + token) * p.out_stride + (int64_t)(q.g * h.group + head) * HD : nullptr,
        part_row(wk, 2 * blockIdx.x + (q.c_lo == 0 ? 1 : 0), row, 128, HD), nullptr, nullptr);
  }
}

template <int HD, bool kTree>
__global__ void __launch_bounds__(Geo::kThreads, 1) attend8_kernel(const AttendParams p, const AttendWork wk) {
  using C = Cfg<HD>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;
  float* merge = reinterpret_cast<float*>(smem + C::kRing);  // [warp][16][32]
  Ctl<HD, kTree>& c = *reinterpret_cast<Ctl<HD, kTree>*>(smem + C::kRing + C::kMerge);
  volatile int* flags = c.flags;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  Shape h;
  h.group = p.group, h.T = h.TT = p.tokens;

  pdl_wait();  // everything read here may come from the kernel before
  if (t == 0) wk.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
  long long W;
  const Walk<kTree> walk = plan::make<Geo, kTree>(p, h, c.plan, reinterpret_cast<long long*>(ring), wk.long_chunks, &W);
  pdl_trigger();
  if (walk.lo >= walk.hi) return;
  if (t < kW) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&c.full[t][i], 1);
      mbar_init(&c.empty[t][i], 1);
    }
    fence_barrier_init();
  }
  if (t == 0) flags[0] = flags[1] = 0, c.walk = walk;
  fence_proxy_async_smem();  // the plan's scratch is overwritten by copies
  __syncthreads();

  if (warp == kW) {
    // ---- producer: lane l copies the pages of warp l
    if (lane < kW) {
      Walk<kTree> w = walk;
      Seg q;
      int i = 0;  // pages of this lane's ring
      bool stop = false;
      while (!stop && w.next(p, h, q)) {
        const int pages = (q.kv + kPage - 1) / kPage;
        int lp = q.k0 / kPage + q.c_lo * kW + lane;
        const int end = min(pages, q.k0 / kPage + q.c_hi * kW);
        const int32_t* table = p.page_tables + (int64_t)q.s * p.mpps;
        int page = lp < end ? __ldg(table + lp) : 0;
        for (; lp < end; lp += kW, ++i) {
          const int next = lp + kW < end ? __ldg(table + lp + kW) : 0;
          const int b = i % C::kStages;
          if (i >= C::kStages && !mbar_wait_ab(&c.empty[lane][b], (i / C::kStages - 1) & 1, flags)) {
            stop = true;
            break;
          }
          if (page < 0 || page >= p.num_pages) {
            if (p.status) atomicOr(p.status, DFLASH_DEV_BAD_PAGE);
            page = 0;
          }
          mbar_arrive_expect_tx(&c.full[lane][b], C::kBytes);
          bulk_load(ring + (lane * C::kStages + b) * C::kBytes,
                    static_cast<const uint8_t*>(p.pool) + page * p.page_stride + (int64_t)q.g * C::kBytes, C::kBytes, &c.full[lane][b]);
          page = next;
        }
      }
      if (flags[0])
        for (int k = 0; k < 2000; ++k) __nanosleep(1000);  // copies still in flight land first
    }
    return;
  }

  // ---- warps with pages.  Lane (r, j) = (lane / 4, lane % 4): rows r and r + 8, keys 4 j .. 4 j + 3 of a page.
  const int r = lane >> 2, j = lane & 3;
  Walk<kTree> w = walk;
  Seg q;
  int i = 0;
  while (w.next(p, h, q)) {
    // ---- the segment's queries: 16 dims from 64 x + 16 j on of both rows, four at a time the k-steps (x, y)
    uint32_t a[HD / 64][4][4];
    int lo[2], hi[2], pos[2], tk[2];
    bool valid[2];
    float rowf[2];  // scale of the scores
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int row = r + 8 * y, tok = row * p.inv >> 16, head = row - tok * h.group;
      tk[y] = q.t0 + tok;
      valid[y] = tok < h.T && tk[y] < q.n;
      uint4 v[HD / 64][2];
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + (int64_t)(q.r0 + tk[y]) * p.q_stride + (q.g * h.group + head) * HD;
#pragma unroll
      for (int x = 0; x < HD / 64; ++x)
#pragma unroll
        for (int z = 0; z < 2; ++z) v[x][z] = valid[y] ? *reinterpret_cast<const uint4*>(src + 64 * x + 16 * j + 8 * z) : make_uint4(0, 0, 0, 0);
      uint32_t top = 0;
#pragma unroll
      for (int x = 0; x < HD / 64; ++x)
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int k = 0; k < 4; ++k) top = max(top, max((&v[x][z].x)[k] & 0x7fffu, (&v[x][z].x)[k] >> 16 & 0x7fffu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = top == 0 ? 0 : max((int)(top >> 7) - 127, -112);
      const float up = pow2i(14 - e);
      rowf[y] = p.scale_log2 * pow2i(e - 14);
#pragma unroll
      for (int x = 0; x < HD / 64; ++x)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t u = (&v[x][k >> 2].x)[k & 3];
          const __half2 g = __floats2half2_rn(__uint_as_float(u << 16) * up, __uint_as_float(u & 0xffff0000u) * up);
          a[x][k >> 1][(k & 1) * 2 + y] = *reinterpret_cast<const uint32_t*>(&g);
        }
      const int ctx = q.kv - q.n;
      pos[y] = !kTree ? ctx + tk[y] : valid[y] && p.window > 0 ? max(ctx, __ldg(p.positions + q.r0 + tk[y])) : 0;
      hi[y] = !valid[y] ? INT_MAX : kTree ? ctx : p.causal ? min(q.kv, pos[y] + 1) : q.kv;
      lo[y] = valid[y] && p.window > 0 ? max(0, kTree ? min(ctx, pos[y] - p.window + 1) : pos[y] - p.window + 1) : 0;
    }
    const int see_lo = __reduce_max_sync(0xffffffffu, max(lo[0], lo[1]));                       // pages within are seen whole
    const int see_hi = min(q.kv, __reduce_min_sync(0xffffffffu, min(hi[0], hi[1])));
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[HD / 8][4];
#pragma unroll
    for (int d = 0; d < HD / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
    int ref = -1000;  // r of the comment above; none yet
    uint32_t met = 0;  // V's largest magnitudes

    const int pages = (q.kv + kPage - 1) / kPage, end = min(pages, q.k0 / kPage + q.c_hi * kW);
    for (int lp = q.k0 / kPage + q.c_lo * kW + warp; lp < end; lp += kW, ++i) {
      const int b = i % C::kStages;
      if (!__all_sync(0xffffffffu, mbar_wait_ab(&c.full[warp][b], (i / C::kStages) & 1, flags))) break;  // (the lanes together)
      uint8_t* tile = ring + (warp * C::kStages + b) * C::kBytes;
      const int key0 = lp * kPage + 4 * j;
      if ((lp + 1) * kPage > q.kv) {
        // rows behind the sequence's end may hold anything: their V becomes zeros (K's scores are replaced below)
        const int live = q.kv - key0;
        const uint32_t dead = live <= 0 ? 0xffffffffu : live >= 4 ? 0u : 0xffffffffu << 8 * live;
#pragma unroll
        for (int d = 0; d < HD / 32; ++d) {
          uint4* v = reinterpret_cast<uint4*>(tile + 16 * HD + d * 512 + r * 64 + ((j ^ (r >> 1)) * 16));
          *v = make_uint4(v->x & ~dead, v->y & ~dead, v->z & ~dead, v->w & ~dead);
        }
        uint32_t* e = reinterpret_cast<uint32_t*>(tile + 32 * HD + 16 + 4 * j);
        __syncwarp();
        if (r == 0) *e = (*e & ~dead) | (0x09090909u & dead);
        fence_proxy_async_smem();  // ahead of the copy that reuses the slot
        __syncwarp();
      }
      // ---- S: score s[x][..] of keys 4 j + 2 x, + 1 (column n of product x is key 4 (n / 2) + 2 x + n % 2)
      float s[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int key = 4 * (r >> 1) + 2 * x + (r & 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) s[x][k] = 0.f;
#pragma unroll
        for (int y = 0; y < HD / 64; ++y) {
          const uint4 k = *reinterpret_cast<const uint4*>(tile + y * 1024 + key * 64 + ((j ^ (key >> 1 & 3)) * 16));
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            uint32_t b0, b1;
            halves((&k.x)[z], b0, b1);
            mma_f16(s[x], a[y][z], b0, b1);
          }
        }
      }
      const uint32_t ek = *reinterpret_cast<const uint32_t*>(tile + 32 * HD + 4 * j), ev = *reinterpret_cast<const uint32_t*>(tile + 32 * HD + 16 + 4 * j);
      float sc[2][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = __uint_as_float(k < 3 ? ek << (23 - 8 * k) & 0x7f800000u : ek >> 1 & 0x7f800000u);  // 2^ke
#pragma unroll
        for (int y = 0; y < 2; ++y) sc[y][k] = s[k >> 1][2 * y + (k & 1)] * (f * rowf[y]);
      }
      if (lp * kPage < see_lo || (lp + 1) * kPage > see_hi) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint32_t bits = 0;
          if (kTree) {
            const uint32_t* mask = reinterpret_cast<const uint32_t*>(p.masks + (int64_t)(q.r0 + (valid[y] ? tk[y] : 0)) * p.words);
            if (valid[y]) bits = plan::mask_bits(mask, 2 * p.words, key0, lo[y], q.kv - q.n, q.kv);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) bits |= key0 + k >= lo[y] && key0 + k < min(hi[y], q.kv) ? 1u << k : 0u;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (!(bits >> k & 1)) sc[y][k] = -INFINITY;
        }
      }
      // ---- softmax: the references move only when a maximum grew by more than 2^8, or an exponent of V by 20
      bool grow = false;
      float alpha[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float top = quad_max(fmaxf(fmaxf(sc[y][0], sc[y][1]), fmaxf(sc[y][2], sc[y][3])));
        alpha[y] = 1.f;
        if (top > m[y] + 8.f) {
          alpha[y] = ex2(m[y] - top);  // (0 from -inf)
          m[y] = top;
          grow = true;
        }
      }
      uint32_t most = __vmaxu4(ev, ev >> 16);
      most = max(most & 255, most >> 8 & 255);
      if (__any_sync(0xffffffffu, grow || (int)most - 127 > ref + 20)) {
        const int top_e = (int)__reduce_max_sync(0xffffffffu, most) - 127;
        float drop = 1.f;
        if (top_e > ref + 20) {
          drop = ref - top_e < -126 ? 0.f : pow2i(ref - top_e);
          ref = top_e;
        }
        l[0] *= alpha[0], l[1] *= alpha[1];
        const float f0 = alpha[0] * drop, f1 = alpha[1] * drop;
#pragma unroll
        for (int d = 0; d < HD / 8; ++d) o[d][0] *= f0, o[d][1] *= f0, o[d][2] *= f1, o[d][3] *= f1;
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float off = m[y] == -INFINITY ? 0.f : m[y];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sc[y][k] = ex2(sc[y][k] - off);
          l[y] += sc[y][k];
        }
      }
      uint32_t pa[4];
      {
        float f[4];  // 2^(ve - ref + 90)
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = __int_as_float(max((k < 3 ? (int)(ev << (23 - 8 * k) & 0x7f800000u) : (int)(ev >> 1 & 0x7f800000u)) + (90 - ref) * (1 << 23), 1 << 23));
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) pa[2 * x + y] = pack_bf16(sc[y][2 * x] * f[2 * x], sc[y][2 * x + 1] * f[2 * x + 1]);
      }
      // ---- O += P V
#pragma unroll
      for (int d = 0; d < HD / 32; ++d) {
        const uint4 v = *reinterpret_cast<const uint4*>(tile + 16 * HD + d * 512 + r * 64 + ((j ^ (r >> 1)) * 16));
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const uint2 w = plan::widen((&v.x)[z], met);
          mma_bf16w(o[4 * d + z], pa, w.x, w.y);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.empty[warp][b]);
    }

    // ---- the warps' states meet: M, L of every row, then O by 32 dims at a time
    if (plan::is_nan(met)) flags[1] = 1;
    const bool whole = q.c_lo == 0 && q.c_hi == q.nch;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
      l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
      if (j == 0) c.ml[warp][r + 8 * y] = make_float2(m[y], l[y]);
    }
    named_barrier(1, 32 * kW);
    float f[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int u = 0; u < kW; ++u) M = fmaxf(M, c.ml[u][r + 8 * y].x);
      const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int u = 0; u < kW; ++u) L += c.ml[u][r + 8 * y].y * ex2(c.ml[u][r + 8 * y].x - base);
      f[y] = ex2(m[y] - base) * (L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L));
      if (warp == y && j == 0 && valid[y]) {
        const int row = r + 8 * y, head = row - (row * p.inv >> 16) * h.group;
        if (!whole)  // (O is normalised: a part's weight is its L 2^M)
          __stcg(wk.ml + (int64_t)(2 * blockIdx.x + (q.c_lo == 0 ? 1 : 0)) * 128 + row, L == 0.f ? make_float2(-INFINITY, 0.f) : make_float2(M + log2f(L), 1.f));
        else if (p.lse)
          p.lse[(int64_t)(q.r0 + tk[y]) * p.nh + q.g * h.group + head] = lse_of(M, L);
      }
    }
    const float unit = ref == -1000 ? 0.f : pow2i(ref);
#pragma unroll
    for (int d = 0; d < HD / 32; ++d) {
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        float* dst = merge + warp * 512 + z * 8 + 2 * j;
        *reinterpret_cast<float2*>(dst + r * 32) = make_float2(o[4 * d + z][0] * f[0] * 0x1p30f * unit, o[4 * d + z][1] * f[0] * 0x1p30f * unit);
        *reinterpret_cast<float2*>(dst + (r + 8) * 32) = make_float2(o[4 * d + z][2] * f[1] * 0x1p30f * unit, o[4 * d + z][3] * f[1] * 0x1p30f * unit);
      }
      named_barrier(1, 32 * kW);
      for (int e = t; e < 256; e += 32 * kW) {  // row e / 16, two dims
        const int row = e >> 4, x = (e & 15) * 2, tok = row * p.inv >> 16, head = row - tok * h.group, token = q.t0 + tok;
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < kW; ++u) {
          const float2 v = *reinterpret_cast<const float2*>(merge + u * 512 + row * 32 + x);
          sum.x += v.x, sum.y += v.y;
        }
        if (tok < h.T && token < q.n && !flags[0]) {
          const int dim = 32 * d + x;
          if (whole) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (int64_t)(q.r0 + token) * p.out_stride + (int64_t)(q.g * h.group + head) * HD + dim;
            *reinterpret_cast<uint32_t*>(dst) = pack_bf16(sum.x, sum.y);
          } else {
            *reinterpret_cast<float2*>(part_row(wk, 2 * blockIdx.x + (q.c_lo == 0 ? 1 : 0), row, 128, HD) + dim) = sum;
          }
        }
      }
      named_barrier(1, 32 * kW);
    }
    if (t == 0 && q.c_lo == 0 && !whole) {  // the unit starts here and goes on in the next CTAs
      const long long last_slot = walk.hi - (q.c_hi - 1) + q.nch - 1;  // past its last slot: slot hi - 1 is chunk c_hi - 1
      const int ctas = (int)min((long long)gridDim.x, W);
      const int last = (int)((last_slot * ctas + W - 1) / W) - 1;
      wk.meta[blockIdx.x] = make_int4(last - (int)blockIdx.x + 1, q.r0 + q.t0, min(h.TT, q.n - q.t0), q.g);
    }
  }
  named_barrier(1, 32 * kW);
  if (flags[1] && !flags[0]) spread_nan8<HD, kTree>(AttendParams(p), AttendWork(wk), c.walk);
  if (t == 0 && flags[0] && p.status) atomicOr(p.status, DFLASH_DEV_TIMEOUT);
}

template <int HD, bool kTree>
cudaError_t launch(const AttendParams& p, const AttendWork& w, int sms, cudaStream_t st) {
  constexpr int kSmem = Cfg<HD>::kRing + Cfg<HD>::kMerge + (int)sizeof(Ctl<HD, kTree>);
  static_assert(kSmem <= 232448, "shared memory of a CTA");
  static_assert(Cfg<HD>::kRing >= 16384 * 8, "the plan's scratch");
  static std::atomic<unsigned long long> attr{0};
  if (cudaError_t e = smem_attr_once(attend8_kernel<HD, kTree>, kSmem, attr); e != cudaSuccess) return e;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(sms);
  c.blockDim = dim3(Geo::kThreads);
  c.dynamicSmemBytes = kSmem;
  c.stream = st;
  c.attrs = a;
  c.numAttrs = 1;
  if (cudaError_t e = cudaLaunchKernelEx(&c, attend8_kernel<HD, kTree>, p, w); e != cudaSuccess) return e;
  return launch_attend_combine(p, w, HD, sms, st);
}

}  // namespace

cudaError_t launch_attend8(const AttendParams& p0, int head_dim, void* workspace, int sms, cudaStream_t st) {
  AttendParams p = p0;
  p.tokens = 16 / p.group;
  // By the hint no sequence has a second tile.  Where by the rows some have many (a hint too low is legal) a warp looks at each
  // sequence of the plan instead of a lane; single tokens in a batch of as many idle rows lose 2 of 25 us by it.
  const AttendWork w = attend_work(workspace, head_dim, sms, p.n_rows > (int64_t)32 * p.tokens * p.nb);
  if (p.masks) return head_dim == 128 ? launch<128, true>(p, w, sms, st) : launch<64, true>(p, w, sms, st);
  return head_dim == 128 ? launch<128, false>(p, w, sms, st) : launch<64, false>(p, w, sms, st);
}

}  // namespace dflash
