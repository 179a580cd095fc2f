// The storage types of the 16-bit (and 32-bit) MoE operators: conversion to
// float, rounding back (nearest even), and one 8-wide matrix-core operand; and
// what the host code of these operators shares.  (Not in milo_internal.hpp: the
// committed traffic measurement of the int3 decode kernel holds for one state
// of the files which that kernel is built from.)
#pragma once

#include "milo_internal.hpp"

namespace milo {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

struct F16 {
  typedef uint16_t store;
  static __device__ __forceinline__ float up(uint16_t b) { return half_bits_to_float(b); }
  static __device__ __forceinline__ uint16_t down(float v) { return float_to_half_bits(v); }
  static __device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                  0, 0);
  }
};

struct BF16 {
  typedef uint16_t store;
  static __device__ __forceinline__ float up(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }
  static __device__ __forceinline__ uint16_t down(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
  static __device__ __forceinline__ f32x4 mfma(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
  }
};

struct F32 {
  typedef float store;
  static __device__ __forceinline__ float up(float v) { return v; }
  static __device__ __forceinline__ float down(float v) { return v; }
};

// V consecutive elements, loaded and stored as one access (V sizeof(store)
// bytes, aligned to that).  LOOSE: aligned to one element only; the memory
// system takes such accesses whole too, at a lower rate.
template <class T, int V, bool LOOSE = false>
struct alignas(LOOSE ? sizeof(typename T::store) : V * sizeof(typename T::store)) Pack {
  typename T::store v[V];
};

// Largest access width in bytes, at most 16, that row lengths of `row_bytes`
// and all the given addresses allow.
inline int access_bytes(size_t row_bytes, const void* a, const void* b = nullptr, const void* c = nullptr,
                        const void* d = nullptr) {
  const uintptr_t bits = (uintptr_t)row_bytes | (uintptr_t)a | (uintptr_t)b | (uintptr_t)c | (uintptr_t)d;
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
}

int device_cu_count();   // compute units of the current device (abi.cpp)

// rows to the experts and back (dispatch.hip)
int32_t launch_permute(const void* x, const int32_t* pos, int64_t tokens, int slots, int H, int64_t rows, int dtype,
                       bool zero, void* y, hipStream_t st);   // zero: rows that no pair names become zeros
int32_t launch_unpermute(const void* y, const int32_t* pos, const float* w, int64_t tokens, int slots, int H,
                         int64_t rows, int dtype, void* out, hipStream_t st);
int32_t launch_unpermute_grad(const void* dout, const void* y, const int32_t* pos, const float* w, int64_t tokens,
                              int slots, int H, int64_t rows, int dtype, bool zero, void* dy, float* dw,
                              hipStream_t st);
int32_t launch_route_grad(const float* dslot_w, const float* logits, const int32_t* ids, int64_t tokens, int E, int k,
                          int S, int renorm, float* dlogits, hipStream_t st);

}  // namespace milo
