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

// 0, or the status of pages that the kernels do not take.
inline int check_pages(const dflash_kv_pages* kv) {
  if (!kv || !kv->pool) return call_error(DFLASH_EINVAL, "null pages");
  if (kv->dtype != DFLASH_BF16 && kv->dtype != DFLASH_F32) return call_error(DFLASH_EINVAL, "pages: dtype must be bf16 or f32");
  if (kv->head_dim != 64 && kv->head_dim != 128) return call_error(DFLASH_EUNSUPPORTED, "pages: head_dim must be 64 or 128");
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 1024) return call_error(DFLASH_EINVAL, "pages: n_kv_heads must be in [1, 1024]");
  // slots are int32: page * 16 + row must fit
  if (kv->num_pages < 1 || kv->num_pages > (1 << 27) - 1) return call_error(DFLASH_EINVAL, "pages: num_pages must be in [1, 2^27)");
  const int es = kv->dtype == DFLASH_F32 ? 4 : 2;
  if (kv->page_stride < (int64_t)32 * kv->n_kv_heads * kv->head_dim || (kv->page_stride * es) % 16)
    return call_error(DFLASH_EINVAL, "pages: page_stride below a page or not whole 16 bytes");
  if (!aligned16(kv->pool)) return call_error(DFLASH_EINVAL, "pages: pool must be 16-byte aligned");
  return DFLASH_OK;
}

}  // namespace dflash
