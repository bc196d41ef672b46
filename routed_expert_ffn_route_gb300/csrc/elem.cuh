// elem.cuh -- element types of the token operators: packs of eight elements read and written
// as fp32, with 16-byte (8-byte for 8-bit types) accesses where addresses allow it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace moe {

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};

// a pack: eight consecutive elements of a row
template <typename T>
struct alignas(16) Pack {
  T v[8];
};

// The pack at element `i` of a row of `n` elements (elements past the end read as zero).
// VEC: the row starts on a 16-byte boundary and n is a multiple of 8.
template <typename T, bool VEC>
__device__ __forceinline__ Pack<T> load_pack(const T *__restrict__ row, int i, int n) {
  Pack<T> p;
  if (VEC) {
    constexpr int W = sizeof(Pack<T>) / 16;
#pragma unroll
    for (int k = 0; k < W; k++) ((uint4 *)&p)[k] = ((const uint4 *)(row + i))[k];
  } else {
#pragma unroll
    for (int k = 0; k < 8; k++) p.v[k] = i + k < n ? row[i + k] : T(0.f);
  }
  return p;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_pack(T *__restrict__ row, int i, int n, const Pack<T> &p) {
  if (VEC) {
    constexpr int W = sizeof(Pack<T>) / 16;
#pragma unroll
    for (int k = 0; k < W; k++) ((uint4 *)(row + i))[k] = ((const uint4 *)&p)[k];
  } else {
#pragma unroll
    for (int k = 0; k < 8; k++)
      if (i + k < n) row[i + k] = p.v[k];
  }
}

}  // namespace moe
