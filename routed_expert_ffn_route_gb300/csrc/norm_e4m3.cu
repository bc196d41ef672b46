// norm_e4m3.cu -- residual addition, RMS norm and 8-bit rows with scales in one pass.
//
// For each token: r = round(x + add) (the residual stream, in x's type), m = mean(r^2),
// y = r w / sqrt(m + eps); then for each group of G elements (or the whole row)
// a = max |y|, scale = a / 448 and q = e4m3(y * 448 / a), 448 being the largest e4m3 value.
// The statistics are fp32.  The largest |y| of a group is the largest |r w| times the row's
// factor, so the sum of squares and the maxima come out of the same single reduction and
// every element is read from memory once: the row stays in registers between the reduction
// and the encoding.  (r w is formed before the row's factor is known, so that it has to lie in
// fp32's range itself.)  Bound by memory: 8192 x 6144 bf16 with a residual moves 352 MB in 55 us,
// 6.4 TB/s of the 6.8 that a copy reaches.
// Rows past 16384 elements are held in eight packs a thread, which do not fit its registers beside
// the next row's: 16-bit types spill 144 to 324 bytes a thread, fp32 some 700 to 1050, and it
// shows: 4096 x 28672 bf16 212 us with a residual (3.9 TB/s), 132 us quantised alone (2.7 TB/s).
#include <cuda_fp8.h>

#include <algorithm>

#include "dev.cuh"
#include "elem.cuh"
#include "moe_internal.cuh"

namespace moe {

constexpr float kE4m3Max = 448.0f;
constexpr float kE4m3Tiny = 0x1p-100f;  // smaller maxima give scale 0 and codes 0: 448 / a is finite

struct NormArgs {
  const void *x, *add, *w;
  void *resid;
  uint8_t *q;
  float *scale;
  long ldx, ldadd, ldr, ldq;
  int T, H, group, gshift, normalize;  // group = 1 << gshift, or 0
  float eps;
};

// scale and factor of a group whose largest |y| is `a`; NaN and infinity pass into the scale
__device__ __forceinline__ float e4m3_factor(float a, float &scale) {
  if (a < kE4m3Tiny) {
    scale = 0.f;
    return 0.f;
  }
  scale = a * (1.0f / kE4m3Max);
  return kE4m3Max * __frcp_rn(a);
}

// most threads of a CTA with `packs` packs a thread (three such CTAs of 16-bit rows fit an SM)
constexpr int norm_threads(int packs, int size) {
  return packs == 1 ? 1024 : packs == 2 ? (size == 2 ? 384 : 1024) : 512;
}

// blockDim.x threads (whole warps) share a row; blockDim.y rows a CTA only with one warp a row.
// Thread t holds the packs t, t + blockDim.x, ... (at most PACKS of them).  A CTA takes rows at a
// stride, and loads the next one while it joins and encodes this one.  Maxima are taken on the
// bit patterns of |v|, where NaN is largest, so a NaN shows in the scale.
// GROUPED: scales by group (a scale a row needs fewer registers, which wide rows want).
template <typename T, int PACKS, int A, bool GROUPED>
__global__ void __launch_bounds__(norm_threads(PACKS, sizeof(T)),
                                  PACKS == 2 && sizeof(T) == 2 ? 3 : 1)
    rmsnorm_e4m3_kernel(const NormArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float ps[2][32];
  __shared__ uint32_t pm[2][32];
  const int tpr = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int H = a.H, G = GROUPED ? a.group : 0, ng = GROUPED ? (H + G - 1) / G : 1;
  const T *w = (const T *)a.w;
  Pack<T> px[PACKS], pa[PACKS];
  auto load = [&](int t) {
    const T *x = (const T *)a.x + (size_t)t * a.ldx;
    const T *add = (const T *)a.add + (size_t)t * a.ldadd;
#pragma unroll
    for (int j = 0; j < PACKS; j++) {
      const int i = 8 * (tid + j * tpr);
      if (Place<T, A>::first(i) >= H) continue;
      px[j] = load_pack<T, A>(x, i, H);
      if (a.add) pa[j] = load_pack<T, A>(add, i, H);
    }
  };
  const int stride = gridDim.x * blockDim.y;
  int t = blockIdx.x * blockDim.y + threadIdx.y;
  if (t < a.T) load(t);
  for (int par = 0; t < a.T; t += stride, par ^= 1) {
    float v[PACKS][8];
    uint32_t mx[PACKS], m = 0;
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < PACKS; j++) {
      const int i = 8 * (tid + j * tpr);
      mx[j] = 0;
      if (A == kWord) {  // every lane's words take part in the groups' maxima
#pragma unroll
        for (int k = 0; k < 8; k++) v[j][k] = 0.f;
      }
      if (Place<T, A>::first(i) >= H) continue;
      px[j].get(v[j]);
      if (a.add) {  // the sum is rounded to the row's type, and read as rounded
        float av[8];
        pa[j].get(av);
#pragma unroll
        for (int k = 0; k < 8; k++) v[j][k] += av[k];
        px[j].put(v[j]);
        px[j].get(v[j]);
      }
      if (a.resid) store_pack<T, A>((T *)a.resid + (size_t)t * a.ldr, i, H, px[j]);
#pragma unroll
      for (int k = 0; k < 8; k++) ss += v[j][k] * v[j][k];
      if (w) {
        float wv[8];
        load_pack<T, A>(w, i, H).get(wv);
#pragma unroll
        for (int k = 0; k < 8; k++) v[j][k] *= wv[k];
      }
#pragma unroll
      for (int k = 0; k < 8; k++) mx[j] = max(mx[j], __float_as_uint(fabsf(v[j][k])));
      m = max(m, mx[j]);
    }
    if (t + stride < a.T) load(t + stride);
    ss = warp_sum(ss);
    m = __reduce_max_sync(0xffffffffu, m);
    if (tpr > 32) {  // two sets of sums in turn: one barrier a row keeps them apart
      if (lane == 0) ps[par][warp] = ss, pm[par][warp] = m;
      __syncthreads();
      const int nw = tpr >> 5;
      ss = warp_sum(lane < nw ? ps[par][lane] : 0.f);
      m = __reduce_max_sync(0xffffffffu, lane < nw ? pm[par][lane] : 0u);
    }
    const float inv = a.normalize ? 1.0f / sqrtf(ss / (float)H + a.eps) : 1.0f;
    float *scale = a.scale + (size_t)t * ng;
    float f, s;
    if (!GROUPED) {
      f = e4m3_factor(__uint_as_float(m) * inv, s);
      if (tid == 0) scale[0] = s;
    }
    if (A != kWord && GROUPED) {  // a group is G / 8 neighbouring lanes; lanes past the row hold zero
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        if (8 * o >= G) break;
#pragma unroll
        for (int j = 0; j < PACKS; j++)
          mx[j] = max(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], o));
      }
    }
    uint8_t *q = a.q + (size_t)t * a.ldq;
#pragma unroll
    for (int j = 0; j < PACKS; j++) {
      const int i = 8 * (tid + j * tpr);
      const int e = Place<T, A>::first(i);
      if (A != kWord) {
        if (GROUPED) {
          f = e4m3_factor(__uint_as_float(mx[j]) * inv, s);
          if (i < H && (i & (G - 1)) == 0) scale[i >> a.gshift] = s;
        }
        if (i >= H) continue;
        uint16_t c[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const float2 y = make_float2(v[j][2 * k] * inv * f, v[j][2 * k + 1] * inv * f);
          c[k] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
        }
        if (A == kVec) {
          *(uint2 *)(q + i) = make_uint2(c[0] | (uint32_t)c[1] << 16, c[2] | (uint32_t)c[3] << 16);
        } else {
#pragma unroll
          for (int k = 0; k < 8; k++)
            if (i + k < H) q[i + k] = (uint8_t)(c[k >> 1] >> (8 * (k & 1)));
        }
      } else {  // word k of every lane is SPAN elements: half a group of 64, a group of 32, ...
        constexpr int W = Pack<T>::W, PER = Place<T, A>::PER, SPAN = Place<T, A>::SPAN;
        uint32_t gm[W];
        if (GROUPED) {
#pragma unroll
          for (int k = 0; k < W; k++) {
            uint32_t b = __float_as_uint(fabsf(v[j][PER * k]));
            if (PER == 2) b = max(b, __float_as_uint(fabsf(v[j][PER * k + PER - 1])));
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {  // lanes of one group: G / PER, at most the warp
              const uint32_t other = __shfl_xor_sync(0xffffffffu, b, o);
              if (PER * o < G) b = max(b, other);
            }
            gm[k] = b;
          }
#pragma unroll
          for (int o = 1; o < W; o <<= 1)
            if (G > SPAN * o) {
#pragma unroll
              for (int k = 0; k < W; k += 2 * o) {
                const uint32_t both = max(gm[k], gm[k + o]);
#pragma unroll
                for (int d = 0; d < 2 * o; d++) gm[k + d] = both;
              }
            }
        }
#pragma unroll
        for (int k = 0; k < W; k++) {
          const int at = e + SPAN * k;
          if (GROUPED) {
            f = e4m3_factor(__uint_as_float(gm[k]) * inv, s);
            if (at < H && (at & (G - 1)) == 0) scale[at >> a.gshift] = s;
          }
          if (at >= H) continue;
          if (PER == 2) {
            const float2 y = make_float2(v[j][2 * k] * inv * f, v[j][2 * k + 1] * inv * f);
            *(uint16_t *)(q + at) = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
          } else {
            q[at] = __nv_cvt_float_to_fp8(v[j][k] * inv * f, __NV_SATFINITE, __NV_E4M3);
          }
        }
      }
    }
  }
}

template <typename T, int PACKS, int A>
static cudaError_t launch_norm_p(const NormArgs &a, dim3 block, cudaStream_t st) {
  auto *k = a.group ? rmsnorm_e4m3_kernel<T, PACKS, A, true>
                    : rmsnorm_e4m3_kernel<T, PACKS, A, false>;
  const int rows = (a.T + block.y - 1) / block.y;
  const int fit = std::max(1, cached_blocks_per_sm((const void *)k, block.x * block.y, 0));
  return launch_pdl(k, dim3(std::min(rows, fit * dev_info().sms)), block, 0, st, a);
}

template <typename T, int A>
static cudaError_t launch_norm(const NormArgs &a, cudaStream_t st) {
  const int packs = (a.H + 7) / 8;
  if (packs <= 128) {  // one warp a row, four rows a CTA: nothing to exchange between warps
    const dim3 block(32, 4);
    if (packs <= 32) return launch_norm_p<T, 1, A>(a, block, st);
    if (packs <= 64) return launch_norm_p<T, 2, A>(a, block, st);
    return launch_norm_p<T, 4, A>(a, block, st);
  }
  auto threads = [&](int p) { return ((packs + p - 1) / p + 31) / 32 * 32; };
  // Few rows: as many threads as the row has packs, the shortest path through one row.  Many
  // rows: two packs a thread (8192 x 6144 bf16 with residual: one 71 us, two 55, three 75, four
  // 63: fewer leave fewer loads in flight, more take the registers of other rows; fp32, twice
  // the bytes a pack: one 104 us, two 111).  Two packs reach 6144 elements with three CTAs an SM;
  // wider 16-bit rows take four: 8192 x 5120 46 us (6.4 TB/s), 6144 55.5 (6.35), 7168 67 (6.1),
  // 8192 72 (6.5), 12288 118 (6.0), 16384 142 (6.6).
  const bool one = a.T <= 2 * dev_info().sms || sizeof(T) == 4;
  auto fits = [&](int p) { return threads(p) <= norm_threads(p, sizeof(T)); };
  if (one && fits(1)) return launch_norm_p<T, 1, A>(a, dim3(threads(1)), st);
  if (fits(2)) return launch_norm_p<T, 2, A>(a, dim3(threads(2)), st);
  if (fits(4)) return launch_norm_p<T, 4, A>(a, dim3(threads(4)), st);
  return launch_norm_p<T, 8, A>(a, dim3(threads(8)), st);
}

template <typename T>
static cudaError_t launch_norm_t(const NormArgs &a, cudaStream_t st) {
  const uintptr_t p = (uintptr_t)a.x | (uintptr_t)a.add | (uintptr_t)a.w | (uintptr_t)a.resid |
                      (uintptr_t)(a.ldx * sizeof(T)) | (uintptr_t)(a.ldadd * sizeof(T)) |
                      (uintptr_t)(a.ldr * sizeof(T));
  int acc = access_of(p, a.H, sizeof(T));
  const uintptr_t pq = (uintptr_t)a.q | (uintptr_t)a.ldq;
  if (acc == kVec && pq % 8) acc = kWord;
  if (acc == kWord && sizeof(T) == 2 && pq % 2) acc = kAny;  // codes move two at a time
  return acc == kVec    ? launch_norm<T, kVec>(a, st)
         : acc == kWord ? launch_norm<T, kWord>(a, st)
                        : launch_norm<T, kAny>(a, st);
}

}  // namespace moe

extern "C" int moe_rmsnorm_e4m3(int T, int H, const void *x, long ldx, moe_dtype dtype,
                                const void *add, long ldadd, const void *weight, float eps,
                                int normalize, int group, void *resid, long ldr, uint8_t *q,
                                long ldq, float *scale, void *stream) {
  if (T < 0 || H <= 0 || !(eps >= 0.f) || (normalize != 0 && normalize != 1))
    return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DT_F32 && dtype != MOE_DT_BF16 && dtype != MOE_DT_F16)
    return MOE_ERR_INVALID_ARG;
  if (H > 32768) return MOE_ERR_UNSUPPORTED;
  if (group != 0 && group != 32 && group != 64 && group != 128 && group != 256)
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const uintptr_t es = dtype == MOE_DT_F32 ? 4 : 2;
  if (!x || !q || !scale || ldx < H || ldq < H || (add && ldadd < H) || (resid && ldr < H))
    return MOE_ERR_INVALID_ARG;
  if ((uintptr_t)x % es || (uintptr_t)add % es || (uintptr_t)weight % es ||
      (uintptr_t)resid % es || (uintptr_t)scale % 4)
    return MOE_ERR_INVALID_ARG;
  int gshift = 0;
  while ((1 << gshift) < group) gshift++;
  if (!add) ldadd = 0;
  if (!resid) ldr = 0;
  const long scales = group ? (H + group - 1) / group : 1;
  const cudaStream_t st = (cudaStream_t)stream;
  // at most 2^30 rows a launch: the kernel's next row number stays in 32 bits (with 64, or without
  // a sign, the registers of the two-pack form change and 8192 x 6144 takes 56.4 us for 55.5)
  for (long t = 0; t < T; t += 1 << 30) {
    auto row = [&](const void *p, long ld) {
      return p ? (uint8_t *)const_cast<void *>(p) + t * ld * (long)es : nullptr;
    };
    const moe::NormArgs a{row(x, ldx), row(add, ldadd), weight, row(resid, ldr), q + t * ldq,
                          scale + t * scales, ldx, ldadd, ldr, ldq,
                          (int)std::min(T - t, 1l << 30), H, group, gshift, normalize, eps};
    const cudaError_t e = dtype == MOE_DT_F32    ? moe::launch_norm_t<float>(a, st)
                          : dtype == MOE_DT_BF16 ? moe::launch_norm_t<__nv_bfloat16>(a, st)
                                                 : moe::launch_norm_t<__half>(a, st);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
