// elem.cuh -- element types of the token operators: packs of eight elements, held as 32-bit
// words and read and written as fp32, with 16-byte accesses where addresses allow them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace moe {

// eight elements of a row
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

// How the rows of a call may be read and written.  Threads of a warp hold neighbouring packs
// i = 8 (first + lane).
//   kVec    rows start on 16-byte boundaries, their length n is a multiple of 8: pack i is the
//           elements i .. i + 7, in 16-byte accesses.
//   kWord   4-byte boundaries, whole words: a warp's 256 elements are dealt out a word a lane at
//           a time, so that its accesses stay neighbours (2050-wide fp32 rows, norm: 20 us, where
//           eight neighbours a lane one at a time take 40).
//   kAny    16-bit elements at odd places, or rows of two element sizes: pack i is the elements i .. i + 7, one at a time, of
//           which the first brings the others into L1 (dealt out 2 bytes a lane, the combination
//           of 2051-wide bf16 rows takes 90 us, so 54; cut out of aligned words 87).
enum Access { kAny = 0, kWord = 1, kVec = 2 };

template <typename T, int A>
struct Place {
  static constexpr int PER = 4 / sizeof(T);  // elements of a word
  static constexpr int SPAN = 32 * PER;      // elements of one word of every lane
  // the first element of pack i; kWord: the next word's is SPAN further
  static __device__ __forceinline__ int first(int i) {
    return A == kWord ? (i & ~255) + ((i >> 3) & 31) * PER : i;
  }
};

// the pack at `i` of a row of `n` elements (elements past the end read as zero)
template <typename T, int A>
__device__ __forceinline__ Pack<T> load_pack(const T *__restrict__ row, int i, int n) {
  Pack<T> p;
  const int e = Place<T, A>::first(i);
  if (A == kVec) {
#pragma unroll
    for (int k = 0; k < Pack<T>::W / 4; k++) {
      const uint4 v = ((const uint4 *)(row + i))[k];
      p.w[4 * k] = v.x, p.w[4 * k + 1] = v.y, p.w[4 * k + 2] = v.z, p.w[4 * k + 3] = v.w;
    }
  } else if (A == kWord) {
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++) {
      const int at = e + k * Place<T, A>::SPAN;
      p.w[k] = at < n ? *(const uint32_t *)(row + at) : 0u;
    }
  } else if (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++) p.w[k] = e + k < n ? ((const uint32_t *)row)[e + k] : 0u;
  } else {
    const uint16_t *r = (const uint16_t *)row;
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++)
      p.w[k] = (e + 2 * k < n ? (uint32_t)r[e + 2 * k] : 0u) |
               (e + 2 * k + 1 < n ? (uint32_t)r[e + 2 * k + 1] << 16 : 0u);
  }
  return p;
}

template <typename T, int A>
__device__ __forceinline__ void store_pack(T *__restrict__ row, int i, int n, const Pack<T> &p) {
  const int e = Place<T, A>::first(i);
  if (A == kVec) {
#pragma unroll
    for (int k = 0; k < Pack<T>::W / 4; k++)
      ((uint4 *)(row + i))[k] =
          make_uint4(p.w[4 * k], p.w[4 * k + 1], p.w[4 * k + 2], p.w[4 * k + 3]);
  } else if (A == kWord) {
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++) {
      const int at = e + k * Place<T, A>::SPAN;
      if (at < n) *(uint32_t *)(row + at) = p.w[k];
    }
  } else if (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++)
      if (e + k < n) ((uint32_t *)row)[e + k] = p.w[k];
  } else {
    uint16_t *r = (uint16_t *)row;
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++) {
      if (e + 2 * k < n) r[e + 2 * k] = (uint16_t)p.w[k];
      if (e + 2 * k + 1 < n) r[e + 2 * k + 1] = (uint16_t)(p.w[k] >> 16);
    }
  }
}

// the widest access that addresses and row distances in bytes (or-ed into `bits`) and rows of
// H elements of `size` bytes allow
static inline int access_of(uintptr_t bits, int H, int size) {
  if (bits % 16 == 0 && H % 8 == 0) return kVec;
  return bits % 4 == 0 && (size == 4 || H % 2 == 0) ? kWord : kAny;
}

// eight neighbouring elements of one lane, the first `n` of them, one at a time
template <typename T>
__device__ __forceinline__ Pack<T> load_run(const T *r, int n) {
  Pack<T> p;
  if (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++) p.w[k] = k < n ? ((const uint32_t *)r)[k] : 0u;
  } else {
    const uint16_t *h = (const uint16_t *)r;
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++)
      p.w[k] = (2 * k < n ? (uint32_t)h[2 * k] : 0u) |
               (2 * k + 1 < n ? (uint32_t)h[2 * k + 1] << 16 : 0u);
  }
  return p;
}
template <typename T>
__device__ __forceinline__ void store_run(T *r, int n, const Pack<T> &p) {
  if (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++)
      if (k < n) ((uint32_t *)r)[k] = p.w[k];
  } else {
    uint16_t *h = (uint16_t *)r;
#pragma unroll
    for (int k = 0; k < Pack<T>::W; k++) {
      if (2 * k < n) h[2 * k] = (uint16_t)p.w[k];
      if (2 * k + 1 < n) h[2 * k + 1] = (uint16_t)(p.w[k] >> 16);
    }
  }
}

}  // namespace moe
