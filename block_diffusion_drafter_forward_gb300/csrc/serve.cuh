// Shared by the serving operators' translation units (serve_*.cu): the message of a failed call
// without a handle, and the checks of a caller's pages.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dflash_internal.cuh"

namespace dflash {

// Records `msg` (and the CUDA error's text) for dflash_last_error(NULL); returns `code`.
int call_error(int code, const char* msg, cudaError_t e = cudaSuccess) noexcept;

#ifdef __CUDACC__
// Pages in 8 bits: byte of row j, dim d in a head's K codes, and in its V codes (from 16 hd on).  K: sixteen
// dims of a row are a 16-byte unit, V: four rows of the dims d, d + 8, d + 16, d + 24; both are what a lane
// of a matrix instruction wants at once.  The units of a 128-byte line are permuted by row (K) or dim (V), so
// that eight lanes on consecutive rows or dims meet no shared-memory bank twice, nor do lanes on all
// units of two.
__device__ __forceinline__ int k8_in_tile(int j, int d) { return (d / 64) * 1024 + j * 64 + (((d / 16) % 4) ^ ((j / 2) % 4)) * 16 + d % 16; }
__device__ __forceinline__ int v8_in_tile(int j, int d) {
  return (d / 32) * 512 + (d % 8) * 64 + ((j / 4) ^ ((d % 8) / 2)) * 16 + ((d % 32) / 8) * 4 + j % 4;
}
// 2^k for k in [-126, 127]
__device__ __forceinline__ float pow2i(int k) { return __int_as_float((k + 127) << 23); }

// 32 bytes: one store (a whole sector) where they are aligned, which the host knows (`wide`)
__device__ __forceinline__ void put32(void* d, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(d)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(d)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
#endif

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Bytes of an element of the pages.
inline int page_es(const dflash_kv_pages* kv) { return kv->dtype == DFLASH_F32 ? 4 : kv->dtype == DFLASH_BF16 ? 2 : 1; }

// 0, or the status of pages that the kernels do not take.  quant: those in 8 bits are taken too.
inline int check_pages(const dflash_kv_pages* kv, bool quant = false) {
  if (!kv || !kv->pool) return call_error(DFLASH_EINVAL, "null pages");
  const bool is_quant = quant && kv->dtype == DFLASH_FP8E4M3_ROWEXP;
  if (kv->dtype != DFLASH_BF16 && kv->dtype != DFLASH_F32 && !is_quant)
    return call_error(DFLASH_EINVAL, quant ? "pages: dtype must be bf16, f32 or e4m3 with row exponents" : "pages: dtype must be bf16 or f32");
  if (kv->head_dim != 64 && kv->head_dim != 128) return call_error(DFLASH_EUNSUPPORTED, "pages: head_dim must be 64 or 128");
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 1024) return call_error(DFLASH_EINVAL, "pages: n_kv_heads must be in [1, 1024]");
  // slots are int32: page * 16 + row must fit
  if (kv->num_pages < 1 || kv->num_pages > (1 << 27) - 1) return call_error(DFLASH_EINVAL, "pages: num_pages must be in [1, 2^27)");
  const int es = page_es(kv);
  if (kv->page_stride < (int64_t)(32 * kv->head_dim + (is_quant ? 32 : 0)) * kv->n_kv_heads || (kv->page_stride * es) % 16 ||
      kv->page_stride > INT64_MAX / 8)
    return call_error(DFLASH_EINVAL, "pages: page_stride below a page or not whole 16 bytes");
  if (!aligned16(kv->pool)) return call_error(DFLASH_EINVAL, "pages: pool must be 16-byte aligned");
  return DFLASH_OK;
}

}  // namespace dflash
