// linear.cu -- matrix product with scales, bias, activation and residual in its epilogue,
// dense or grouped by expert.
//
//   z[r][n]   = s_x[r] s_w[e][n] sum_k x[r][k] w[e][n][k] + b[e][n]
//   out[r][n] = act(z)[r][n] + residual[r][n]            e = the expert whose rows hold r
//   (act = SwiGLU: w has 2 N rows, out = silu(z[r][n]) * z[r][N + n])
//
// The tensor cores compute transposed tiles: weight rows are the M = 128 side of each MMA,
// token rows its N side, any multiple of 16 up to 256.  One kernel then serves one token
// (16 columns, bound by reading the weights) and a prefill (256 columns, bound by the
// MMAs), and an expert's ragged last tile costs only the columns it has.  Types differ only
// in the instruction kind: a k-block is 128 bytes of a row for 8- and 16-bit elements alike.
//
// A persistent CTA per SM walks the tiles of all experts.  Warp 0 issues TMA loads into a
// ring of stages (128-byte swizzle; rows past an expert's weights, and the end of K, read as
// zero), warp 1 issues tcgen05.mma into one of two accumulators in tensor memory, warps 2-5
// turn the other accumulator into output.  For SwiGLU the weight map interleaves 16 gate
// rows with their 16 up rows, so that a gate and its up value sit 16 lanes apart in one warp.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "dev.cuh"
#include "elem.cuh"
#include "expert_args.cuh"
#include "moe_internal.cuh"
#include "tc.cuh"

namespace moe {

constexpr int kLinM = 128;         // weight rows per tile
constexpr int kLinMaxN = 256;      // token rows per tile
constexpr int kLinStages = 12;     // ring slots at most
constexpr int kLinMaxE = 256;
constexpr int kLinThreads = 192;
constexpr int kLinRing = 208 * 1024;  // shared memory of the ring
constexpr long kLinWaitNs = 2000000000L;

struct LinArgs {
  const float *x_scale, *w_scale, *bias;
  const void *residual;
  void *out;
  const int32_t *offsets;
  int32_t *status;
  long ldres, ldout;
  int R, N, E;       // E = 0: dense
  int KB, ke;        // k-blocks, elements per k-block
  int BN, stages;    // token rows per tile, ring slots
  int FT;            // feature tiles
  int act;
  int kind8, bf16;   // operand type: e4m3, or bf16 / fp16
};

struct LinBars {
  uint64_t full[kLinStages], empty[kLinStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int abort_flag;
  alignas(16) float xs[4][kLinMaxN];  // token scales of the epilogue warps' tile
  int pre[kLinMaxE + 1];   // row tiles before each expert
  int off[kLinMaxE + 1];   // first row of each expert
};

__device__ __forceinline__ void mma_ss_f8(uint32_t d_taddr, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_taddr),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(void *dst, const void *tmap, int x, int y, int z,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(tc::smem_u32(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_5d(void *dst, const void *tmap, int x, int y, int z, int u,
                                            int v, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(tc::smem_u32(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(tc::smem_u32(bar))
      : "memory");
}

// A tile: rows [r0, r0 + n) of expert e, feature tile ft.  Row tiles run fastest, so that
// CTAs working at the same time share weight tiles in L2.
struct LinTile {
  int e, ft, r0, n;
};
__device__ __forceinline__ LinTile lin_tile(const LinArgs &a, const LinBars *b, int tile) {
  // experts lie one after another; expert e holds pre[e+1] - pre[e] row tiles x FT
  int lo = 0, hi = max(1, a.E);
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile >= b->pre[mid] * a.FT) lo = mid; else hi = mid;
  }
  const int rt_n = b->pre[lo + 1] - b->pre[lo];
  const int i = tile - b->pre[lo] * a.FT;
  LinTile t;
  t.e = lo;
  t.ft = i / rt_n;
  t.r0 = b->off[lo] + (i - t.ft * rt_n) * a.BN;
  t.n = min(a.BN, b->off[lo + 1] - t.r0);
  return t;
}

__device__ __forceinline__ float lin_act(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z < 0.f ? 0.f : z;  // a NaN stays one
    case MOE_ACT_SILU: return silu_f(z);
    case MOE_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    default: return z;
  }
}

template <typename TO, bool GATED>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                  const LinArgs a) {
  extern __shared__ uint8_t smraw[];
  uint8_t *ring = tc::align_smem_1024(smraw);
  const int stage_bytes = (kLinM + a.BN) * 128;
  LinBars *b = (LinBars *)(ring + kLinRing);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < a.stages; s++) {
      tc::mbar_init(&b->full[s], 1);
      tc::mbar_init(&b->empty[s], 1);
    }
    for (int i = 0; i < 2; i++) {
      tc::mbar_init(&b->acc_full[i], 1);
      tc::mbar_init(&b->acc_empty[i], 4);
    }
    tc::mbar_init(&b->drain, 1);
    b->abort_flag = 0;
    tc::fence_barrier_init();
  }
  // tensor memory before the trigger: a successor may start as soon as every CTA has
  // triggered, and must not take columns that this grid still has to allocate
  if (warp == 0) tc::tmem_alloc<512>(&b->tmem);
  pdl_wait();
  pdl_trigger();
  // the experts' rows, clamped to [0, R] and kept in order, so that no offset leads out of x
  if (a.E == 0) {
    if (tid == 0) {
      b->off[0] = 0;
      b->off[1] = a.R;
      b->pre[0] = 0;
      b->pre[1] = (a.R + a.BN - 1) / a.BN;
    }
  } else if (warp == 1) {
    int base = 0, last = 0;
    for (int e0 = 0; e0 <= a.E; e0 += 32) {
      const int e = e0 + lane;
      int o = e <= a.E ? min(max(a.offsets[e], 0), a.R) : 0;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) o = max(o, __shfl_up_sync(0xffffffffu, o, s));
      o = max(o, last);
      int prev = __shfl_up_sync(0xffffffffu, o, 1);
      if (lane == 0) prev = last;
      // tiles of expert e - 1: rows [prev, o)
      int c = e >= 1 && e <= a.E ? (o - prev + a.BN - 1) / a.BN : 0;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, c, s);
        if (lane >= s) c += v;
      }
      if (e <= a.E) {
        b->off[e] = o;
        b->pre[e] = base + c;
      }
      base += __shfl_sync(0xffffffffu, c, 31);
      last = __shfl_sync(0xffffffffu, o, 31);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = b->tmem;
  volatile int *abort = &b->abort_flag;
  auto give_up = [&]() {
    *abort = 1;
    if (a.status) *a.status = MOE_ERR_TIMEOUT;
  };
  const int total = b->pre[max(1, a.E)] * a.FT;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------- producer
      bool ok = true;
      uint32_t it = 0, armed = 0, last_ph = 0;
      int s = 0;
      uint32_t ph = 0;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const LinTile t = lin_tile(a, b, tile);
        for (int kb = 0; kb < a.KB; kb++, it++) {
          if (!tc::mbar_wait(&b->empty[s], ph ^ 1, abort, kLinWaitNs)) { ok = false; break; }
          uint8_t *st = ring + (size_t)s * stage_bytes;
          tc::mbar_arrive_expect_tx(&b->full[s], stage_bytes);
          if (GATED)
            tma_load_5d(st, &wmap, kb * a.ke, 0, 0, t.ft * (kLinM / 32), t.e, &b->full[s]);
          else
            tma_load_3d(st, &wmap, kb * a.ke, t.ft * kLinM, t.e, &b->full[s]);
          tc::tma_load_2d(st + kLinM * 128, &xmap, kb * a.ke, t.r0, &b->full[s]);
          armed |= 1u << s;
          last_ph = (last_ph & ~(1u << s)) | (ph << s);
          if (++s == a.stages) s = 0, ph ^= 1;
        }
      }
      // every copy started lands before the CTA exits
      if (!ok) {
        give_up();
        for (int q = 0; q < a.stages; q++)
          if ((armed >> q) & 1) wait_nofail(&b->full[q], (last_ph >> q) & 1, kLinWaitNs);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (one elected lane)
    const bool leader = tc::elect_one();
    bool ok = true, issued = false;
    int s = 0, buf = 0;
    uint32_t ph = 0, bph = 0;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const LinTile t = lin_tile(a, b, tile);
      const uint32_t idesc = tc::idesc_f16(a.bf16, round16(t.n));
      int got = 1;
      if (leader) got = tc::mbar_wait(&b->acc_empty[buf], bph ^ 1, abort, kLinWaitNs);
      ok = __all_sync(0xffffffffu, got);
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t d = tbase + buf * kLinMaxN;
      for (int kb = 0; kb < a.KB; kb++) {
        if (leader) got = tc::mbar_wait_spin(&b->full[s], ph, abort, kLinWaitNs);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) break;
        tc::fence_after_sync();
        if (leader) {
          const uint32_t sa = tc::smem_u32(ring) + (uint32_t)(s * stage_bytes);
          const uint64_t da = tc::sdesc_sw128(sa), db = tc::sdesc_sw128(sa + kLinM * 128);
          if (a.kind8) {
#pragma unroll
            for (int kk = 0; kk < 4; kk++)
              mma_ss_f8(d, da + 2 * kk, db + 2 * kk, idesc, (kb | kk) != 0);
          } else {
#pragma unroll
            for (int kk = 0; kk < 4; kk++)
              tc::mma_ss(d, da + 2 * kk, db + 2 * kk, idesc, (kb | kk) != 0);
          }
          tc::mma_commit(&b->empty[s]);
        }
        __syncwarp();
        issued = true;
        if (++s == a.stages) s = 0, ph ^= 1;
      }
      if (!ok) break;
      if (leader) tc::mma_commit(&b->acc_full[buf]);
      __syncwarp();
      if (buf) bph ^= 1;
      buf ^= 1;
    }
    if (leader && !ok) {
      give_up();
      if (issued) {  // every MMA issued completes before the tensor memory is freed
        tc::mma_commit(&b->drain);
        wait_nofail(&b->drain, 0, kLinWaitNs);
      }
    }
  } else {
    // -------------------------------------------------- epilogue: a lane per weight row
    const int quad = warp & 3;  // the warp's quarter of the tensor-memory lanes
    const int rows = GATED ? 2 * a.N : a.N;
    const TO *res = (const TO *)a.residual;
    TO *out = (TO *)a.out;
    int buf = 0;
    uint32_t bph = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const LinTile t = lin_tile(a, b, tile);
      // this lane's weight row, and the output feature that it (and its partner) give
      int wr, f;
      if (GATED) {
        f = t.ft * 64 + quad * 16 + (lane & 15);
        wr = f + (lane >= 16 ? a.N : 0);
      } else {
        wr = f = t.ft * kLinM + quad * 32 + lane;
      }
      const bool in = f < a.N;
      const float sw = a.w_scale && in ? a.w_scale[(long)t.e * rows + wr] : 1.f;
      const float bi = a.bias && in ? a.bias[(long)t.e * rows + wr] : 0.f;
      // the tile's token scales, a copy per warp (1 where there are none, 0 past the rows)
      float *xs = b->xs[quad];
      __syncwarp();
      for (int c = lane; c < a.BN; c += 32)
        xs[c] = c < t.n ? a.x_scale ? a.x_scale[t.r0 + c] : 1.f : 0.f;
      __syncwarp();
      if (!__all_sync(0xffffffffu,
                      tc::mbar_wait_backoff(&b->acc_full[buf], bph, abort, kLinWaitNs, 64)))
        break;
      tc::fence_after_sync();
      const uint32_t taddr = tbase + buf * kLinMaxN + ((uint32_t)(32 * quad) << 16);
      // of two columns, the lower lanes of a SwiGLU warp finish the first, the upper the second
      const int up = GATED && lane >= 16;
      TO *op = out + (long)(t.r0 + up) * a.ldout + f;
      const TO *rp = res ? res + (long)(t.r0 + up) * a.ldres + f : nullptr;
      for (int c0 = 0; c0 < t.n; c0 += 16) {
        constexpr int S = GATED ? 2 : 1, J = 16 / S;
        float y[J], rv[J];
        uint32_t v[16];
        __syncwarp();
        tc::tmem_ld16(taddr + c0, v);
        const int left = in ? t.n - c0 - up : 0;  // columns that this lane stores
        if (rp) {
#pragma unroll
          for (int j = 0; j < J; j++)
            rv[j] = S * j < left ? Elem<TO>::get(rp[(c0 + S * j) * a.ldres]) : 0.f;
        }
        tc::tmem_wait_ld();
        if (c0 + 16 >= t.n) {  // the accumulator is read: the next tile may use it
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&b->acc_empty[buf]);
        }
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 s4 = *(const float4 *)(xs + c0 + j);
          const float z0 = fmaf(__uint_as_float(v[j]) * s4.x, sw, bi);
          const float z1 = fmaf(__uint_as_float(v[j + 1]) * s4.y, sw, bi);
          const float z2 = fmaf(__uint_as_float(v[j + 2]) * s4.z, sw, bi);
          const float z3 = fmaf(__uint_as_float(v[j + 3]) * s4.w, sw, bi);
          if (GATED) {
            const float o0 = __shfl_xor_sync(0xffffffffu, up ? z0 : z1, 16);
            const float o1 = __shfl_xor_sync(0xffffffffu, up ? z2 : z3, 16);
            y[j / 2] = up ? silu_f(o0) * z1 : silu_f(z0) * o0;
            y[j / 2 + 1] = up ? silu_f(o1) * z3 : silu_f(z2) * o1;
          } else {
            y[j] = z0, y[j + 1] = z1, y[j + 2] = z2, y[j + 3] = z3;
          }
        }
        if (!GATED && a.act != MOE_ACT_NONE) {
#pragma unroll
          for (int j = 0; j < J; j++) y[j] = lin_act(y[j], a.act);
        }
        if (rp) {
#pragma unroll
          for (int j = 0; j < J; j++) y[j] += rv[j];
        }
#pragma unroll
        for (int j = 0; j < J; j++)
          if (S * j < left) op[(c0 + S * j) * a.ldout] = Elem<TO>::put(y[j]);
      }
      if (buf) bph ^= 1;
      buf ^= 1;
    }
    // rows of no expert are zero
    if (a.E) {
      const long live0 = b->off[a.E], lead = b->off[0];
      const long first = (long)blockIdx.x * 128 + (warp - 2) * 32 + lane;
      const long step = (long)gridDim.x * 128;
      for (long i = first; i < lead * a.N; i += step)
        out[i / a.N * a.ldout + i % a.N] = Elem<TO>::put(0.f);
      for (long i = first; i < (a.R - live0) * a.N; i += step)
        out[(live0 + i / a.N) * a.ldout + i % a.N] = Elem<TO>::put(0.f);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc<512>(tbase);
}

static PFN_cuTensorMapEncodeTiled_v12000 lin_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                     cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? (PFN_cuTensorMapEncodeTiled_v12000)p : nullptr;
  }();
  return fn;
}

// Token rows per tile: the fewest tiles of at most 256 rows, all of about the same size; by
// expert the mean number of rows decides (an expert's last tile costs only what it has).
static int lin_bn(int R, int E) {
  const int m = E ? (R + E - 1) / E : R;
  if (E) return m >= 96 ? 256 : std::min(256, std::max(16, round16(2 * m)));
  const int nt = (m + kLinMaxN - 1) / kLinMaxN;
  return std::max(16, round16((m + nt - 1) / nt));
}

template <typename TO, bool GATED>
static int launch_linear(const CUtensorMap &xm, const CUtensorMap &wm, const LinArgs &a,
                         cudaStream_t st) {
  const size_t smem = 1024 + kLinRing + sizeof(LinBars);
  set_dyn_smem((const void *)linear_kernel<TO, GATED>, (int)smem);
  const long tiles = ((long)std::min(a.R, std::max(1, a.E)) + a.R / a.BN) * a.FT;
  const int grid = (int)std::min((long)dev_info().sms, std::max(1l, tiles));
  if (launch_pdl(linear_kernel<TO, GATED>, dim3(grid), dim3(kLinThreads), smem, st, xm, wm, a) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename TO>
static int launch_linear_t(const CUtensorMap &xm, const CUtensorMap &wm, const LinArgs &a,
                           cudaStream_t st) {
  return a.act == MOE_ACT_SWIGLU ? launch_linear<TO, true>(xm, wm, a, st)
                                 : launch_linear<TO, false>(xm, wm, a, st);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_linear(int R, int N, int K, int n_experts, const void *x, long ldx,
                          moe_dtype dtype, const float *x_scale, const void *w,
                          const float *w_scale, const float *bias, moe_act act,
                          const void *residual, long ldres, const int32_t *offsets, void *out,
                          long ldout, moe_dtype out_dtype, int32_t *status, void *stream) {
  if (R < 0 || N <= 0 || K <= 0 || n_experts < 0) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DT_E4M3 && dtype != MOE_DT_BF16 && dtype != MOE_DT_F16)
    return MOE_ERR_INVALID_ARG;
  if (out_dtype != MOE_DT_F32 && out_dtype != MOE_DT_BF16 && out_dtype != MOE_DT_F16)
    return MOE_ERR_INVALID_ARG;
  if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  const bool gated = act == MOE_ACT_SWIGLU;
  const int es = dtype == MOE_DT_E4M3 ? 1 : 2;
  if (n_experts > kLinMaxE || K % 16 || (gated && N % 16)) return MOE_ERR_UNSUPPORTED;
  // sizes that the 32-bit tile and coordinate arithmetic covers
  if (R > (1 << 24) || N > (1 << 20) || K > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (!x || !w || !out || ldx < K || ldout < N || (residual && ldres < N) ||
      (n_experts && !offsets))
    return MOE_ERR_INVALID_ARG;
  const uintptr_t eo = out_dtype == MOE_DT_F32 ? 4 : 2;
  if ((uintptr_t)x % 16 || (uintptr_t)w % 16 || (uintptr_t)(ldx * es) % 16 ||
      ((uintptr_t)out | (uintptr_t)residual) % eo ||
      ((uintptr_t)x_scale | (uintptr_t)w_scale | (uintptr_t)bias | (uintptr_t)offsets |
       (uintptr_t)status) % 4)
    return MOE_ERR_INVALID_ARG;
  PFN_cuTensorMapEncodeTiled_v12000 enc = lin_encode();
  if (!enc) return MOE_ERR_CUDA;

  LinArgs a{};
  a.x_scale = x_scale;
  a.w_scale = w_scale;
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.offsets = n_experts ? offsets : nullptr;
  a.status = status;
  a.ldres = ldres;
  a.ldout = ldout;
  a.R = R;
  a.N = N;
  a.E = n_experts;
  a.ke = 128 / es;
  a.KB = (K + a.ke - 1) / a.ke;
  a.BN = lin_bn(R, n_experts);
  a.stages = std::min(kLinStages, kLinRing / ((kLinM + a.BN) * 128));
  a.FT = gated ? (N + 63) / 64 : (N + kLinM - 1) / kLinM;
  a.act = act;
  a.kind8 = es == 1;
  a.bf16 = dtype == MOE_DT_BF16;

  const CUtensorMapDataType dt = es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                         : CU_TENSOR_MAP_DATA_TYPE_UINT16;
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  CUtensorMap xm, wm;
  {
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)R};
    const cuuint64_t strides[1] = {(cuuint64_t)ldx * es};
    const cuuint32_t box[2] = {(cuuint32_t)a.ke, (cuuint32_t)a.BN};
    if (enc(&xm, dt, 2, const_cast<void *>(x), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return MOE_ERR_CUDA;
  }
  const cuuint64_t row = (cuuint64_t)K * es, ne = (cuuint64_t)std::max(1, n_experts);
  CUresult cr;
  if (gated) {  // [e][N / 16][gate, up][16][K]
    const cuuint64_t dims[5] = {(cuuint64_t)K, 16, 2, (cuuint64_t)N / 16, ne};
    const cuuint64_t strides[4] = {row, row * N, row * 16, row * N * 2};
    const cuuint32_t box[5] = {(cuuint32_t)a.ke, 16, 2, kLinM / 32, 1};
    cr = enc(&wm, dt, 5, const_cast<void *>(w), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else {
    const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, ne};
    const cuuint64_t strides[2] = {row, row * N};
    const cuuint32_t box[3] = {(cuuint32_t)a.ke, kLinM, 1};
    cr = enc(&wm, dt, 3, const_cast<void *>(w), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  if (cr != CUDA_SUCCESS) return MOE_ERR_CUDA;
  const cudaStream_t st = (cudaStream_t)stream;
  return out_dtype == MOE_DT_F32    ? launch_linear_t<float>(xm, wm, a, st)
         : out_dtype == MOE_DT_BF16 ? launch_linear_t<__nv_bfloat16>(xm, wm, a, st)
                                    : launch_linear_t<__half>(xm, wm, a, st);
}
