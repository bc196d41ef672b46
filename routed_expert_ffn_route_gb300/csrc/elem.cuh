// elem.cuh -- element types of the token operators: packs of eight elements, held as 32-bit
// words and read and written as fp32, with 16-byte accesses where addresses allow them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace moe {

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};

// eight consecutive elements of a row
template <typename T>
struct Pack {
  static constexpr int W = 8 * sizeof(T) / 4;
  uint32_t w[W];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < W; k++) w[k] = 0;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const;
  __device__ __forceinline__ void put(const float (&f)[8]);
};

template <>
__device__ __forceinline__ void Pack<float>::get(float (&f)[8]) const {
#pragma unroll
  for (int k = 0; k < 8; k++) f[k] = __uint_as_float(w[k]);
}
template <>
__device__ __forceinline__ void Pack<float>::put(const float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 8; k++) w[k] = __float_as_uint(f[k]);
}
template <>
__device__ __forceinline__ void Pack<__nv_bfloat16>::get(float (&f)[8]) const {
#pragma unroll
  for (int k = 0; k < 4; k++) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void Pack<__nv_bfloat16>::put(const float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
    w[k] = *(const uint32_t *)&v;
  }
}
template <>
__device__ __forceinline__ void Pack<__half>::get(float (&f)[8]) const {
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const float2 v = __half22float2(*(const __half2 *)&w[k]);
    f[2 * k] = v.x;
    f[2 * k + 1] = v.y;
  }
}
template <>
__device__ __forceinline__ void Pack<__half>::put(const float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const __half2 v = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
    w[k] = *(const uint32_t *)&v;
  }
}

// The pack at element `i` of a row of `n` elements (elements past the end read as zero).
// VEC: the row starts on a 16-byte boundary and n is a multiple of 8.
template <typename T, bool VEC>
__device__ __forceinline__ Pack<T> load_pack(const T *__restrict__ row, int i, int n) {
  Pack<T> p;
  if (VEC) {
#pragma unroll
    for (int k = 0; k < Pack<T>::W / 4; k++) {
      const uint4 v = ((const uint4 *)(row + i))[k];
      p.w[4 * k] = v.x, p.w[4 * k + 1] = v.y, p.w[4 * k + 2] = v.z, p.w[4 * k + 3] = v.w;
    }
  } else if (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++) p.w[k] = i + k < n ? ((const uint32_t *)row)[i + k] : 0u;
  } else {
    const uint16_t *r = (const uint16_t *)row;
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++) {
      const int e = i + 2 * k;
      p.w[k] = (e < n ? (uint32_t)r[e] : 0u) | (e + 1 < n ? (uint32_t)r[e + 1] << 16 : 0u);
    }
  }
  return p;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_pack(T *__restrict__ row, int i, int n, const Pack<T> &p) {
  if (VEC) {
#pragma unroll
    for (int k = 0; k < Pack<T>::W / 4; k++)
      ((uint4 *)(row + i))[k] =
          make_uint4(p.w[4 * k], p.w[4 * k + 1], p.w[4 * k + 2], p.w[4 * k + 3]);
  } else if (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++)
      if (i + k < n) ((uint32_t *)row)[i + k] = p.w[k];
  } else {
    uint16_t *r = (uint16_t *)row;
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++) {
      const int e = i + 2 * k;
      if (e < n) r[e] = (uint16_t)p.w[k];
      if (e + 1 < n) r[e + 1] = (uint16_t)(p.w[k] >> 16);
    }
  }
}

}  // namespace moe
