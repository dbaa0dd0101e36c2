// Small helpers of the training calls: fp32 values of 8 (or 1) consecutive columns of an fp32
// or bf16 array, the embedding's row of a position, and the host checks they share.
#pragma once

#include <cuda_bf16.h>

#include "pg_internal.cuh"

namespace pg {
namespace {

constexpr uint32_t kNoRow = 0xFFFFFFFFu;
constexpr int kMaxEmbedWidth = 1 << 20;  // columns of an embedding row

inline bool real_dtype(int dtype) { return dtype == PG_F32 || dtype == PG_BF16; }
inline size_t dtype_bytes(int dtype) { return dtype == PG_F32 ? 4 : 2; }
inline size_t vec_bytes(int dtype) { return 8 * dtype_bytes(dtype); }  // 8 columns: one access of 16 or 32 bytes
inline bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Table row of position t, or kNoRow for padding (a token outside [0, vocab), or a canonical
// ID that the table does not have).
__device__ __forceinline__ uint32_t embed_row(const int32_t* __restrict__ tokens,
                                              const uint32_t* __restrict__ canon_map, uint32_t vocab, uint32_t rows,
                                              int64_t t) {
  const uint32_t x = static_cast<uint32_t>(__ldg(tokens + t));  // negative: not below vocab <= 2^31
  if (x >= vocab || x >= 0x80000000u) return kNoRow;
  const uint32_t row = canon_map ? __ldg(canon_map + x) : x;
  return row < rows ? row : kNoRow;
}

// 32 bytes with one access (sm_100 and later), 32-byte aligned.
__device__ __forceinline__ void load32(const void* p, float (&x)[8]) {
  asm("ld.global.nc.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
      : "l"(p));
}

__device__ __forceinline__ void store32(void* p, const float (&x)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
               "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}

// 8 columns with one access (the address is aligned to it), or 1.
template <int DT, int COLS>
__device__ __forceinline__ void load_cols(const void* __restrict__ base, int64_t at, float (&x)[COLS]) {
  static_assert(COLS == 1 || COLS == 8, "");
  if constexpr (DT == PG_F32) {
    const float* p = static_cast<const float*>(base) + at;
    if constexpr (COLS == 1) {
      x[0] = __ldg(p);
    } else {
      load32(p, x);
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if constexpr (COLS == 1) {
      x[0] = __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
    } else {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
      x[0] = __uint_as_float(w.x << 16); x[1] = __uint_as_float(w.x & 0xFFFF0000u);
      x[2] = __uint_as_float(w.y << 16); x[3] = __uint_as_float(w.y & 0xFFFF0000u);
      x[4] = __uint_as_float(w.z << 16); x[5] = __uint_as_float(w.z & 0xFFFF0000u);
      x[6] = __uint_as_float(w.w << 16); x[7] = __uint_as_float(w.w & 0xFFFF0000u);
    }
  }
}

// fp32 that an earlier kernel writes while this one already runs, after the wait for its end: coherent
// loads that stay behind that wait. (The read-only path of load_cols is for what nothing writes
// during the kernel, and its loads may move.)
template <int COLS>
__device__ __forceinline__ void load_now(const float* p, float (&x)[COLS]) {
  static_assert(COLS == 1 || COLS == 8, "");
  if constexpr (COLS == 1)
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(x[0]) : "l"(p) : "memory");
  else
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "l"(p)
                 : "memory");
}

// The same as load_cols from memory that this kernel writes (no read-only cache).
template <int DT, int COLS>
__device__ __forceinline__ void read_cols(const void* base, int64_t at, float (&x)[COLS]) {
#pragma unroll
  for (int j = 0; j < COLS; ++j)
    x[j] = DT == PG_F32 ? static_cast<const float*>(base)[at + j]
                        : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at + j]);
}

__device__ __forceinline__ uint32_t two_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

template <int DT, int COLS>
__device__ __forceinline__ void store_cols(void* base, int64_t at, const float (&x)[COLS]) {
  if constexpr (DT == PG_F32) {
    float* p = static_cast<float*>(base) + at;
    if constexpr (COLS == 1) {
      *p = x[0];
    } else {
      store32(p, x);
    }
  } else {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + at;
    if constexpr (COLS == 1)
      *p = __float2bfloat16_rn(x[0]);
    else
      *reinterpret_cast<uint4*>(p) = make_uint4(two_bf16(x[0], x[1]), two_bf16(x[2], x[3]), two_bf16(x[4], x[5]),
                                                two_bf16(x[6], x[7]));
  }
}

}  // namespace
}  // namespace pg
