// linear.cuh -- what the matrix products share (linear.cu: floating-point operands, linear_i8.cu:
// 8-bit integers): tiles of experts' rows, pairs and clusters of CTAs, the MMA, the epilogue, and
// waits that give up.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "dev.cuh"
#include "elem.cuh"
#include "expert_args.cuh"
#include "host.cuh"
#include "linear_plan.cuh"
#include "moe_internal.cuh"
#include "tc.cuh"

namespace moe {

constexpr int kLinMaxN = 256;      // token rows per tile
constexpr int kLinMaxE = 256;
constexpr int kLinEpi = 8;         // epilogue warps: two per quarter of the tensor-memory lanes
constexpr int kLinThreads = 64 + 32 * kLinEpi;
constexpr int kLinPitch = 36;      // floats per column of a warp's staged chunk (32 features)
constexpr int kLinStage = kLinEpi * 16 * kLinPitch * 4;  // bytes of the staged chunks
constexpr long kLinWaitNs = 2000000000L;
constexpr long kLinLateNs = 50000000L;  // a pair's copies, after a wait gave up

// fp32 outputs: the tensor cores truncate each sum to fp32 (K = 6144 bf16 loses 6e-6 of the result
// that way, 1.4e-5 of a SwiGLU's), so they sum kLinExact k-blocks at a time and the epilogue warps
// add those sums, rounded to nearest, in registers: 3e-7 and 5e-7.  (4096^3 bf16 takes 152 us so;
// eight k-blocks 134, with twice the error; the two accumulators of a pair wait on each other
// across its CTAs and take 179.)  16-bit outputs, rounded to 2^-9 or 2^-12, are summed to the end in
// tensor memory.
constexpr int kLinExact = 4;
template <typename TO>
constexpr bool lin_exact = sizeof(TO) == 4;
// columns between the two accumulators
template <typename TO>
constexpr int kLinAcc = lin_exact<TO> ? 128 : kLinMaxN;

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
  int FT;            // feature tiles (of 128 weight rows, kPair: 256)
  int group;         // row tiles taken together
  int split;         // kSplit: CTAs per tile
  int ring;          // bytes of the ring
  int exchange;      // kSplit: bytes of the partial sums' exchange behind it
  int act;
  int kind8, bf16;   // operand type: e4m3, or bf16 / fp16
  int vec;           // out's and residual's rows start on 16-byte boundaries
  int never;         // the epilogue's waits run out (moe_debug_linear_timeout)
};

struct alignas(16) LinBars {
  uint64_t full[kLinStages], empty[kLinStages], acc_full[2], acc_empty[2], drain, never;
  uint32_t tmem;
  int abort_flag;
  uint32_t armed, phases;  // for the drain: full barriers with a copy started, and their last phase
  int issued;              // some MMA was issued
  alignas(16) float xs[kLinEpi][kLinMaxN / 2];     // token scales of the epilogue warps' columns
  int pre[kLinMaxE + 1];   // row tiles before each expert
  int off[kLinMaxE + 1];   // first row of each expert
};

// ---------------------------------------------------------------- pairs and clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ void prefetch_map(const void *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// the address of a shared-memory object in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t in_cta(const void *p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void arrive_in_cta(uint64_t *bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                   in_cta(bar, rank))
               : "memory");
}
__device__ __forceinline__ void store_in_cta(uint32_t addr, const uint32_t *v) {  // 16 bytes
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

// Tensor memory of a CTA: two accumulators of 256 columns; kSplit has one, and its number is a
// constant of the instruction, without which the driver gives such a kernel whole SMs.
template <int MODE>
__device__ __forceinline__ void lin_tmem_alloc(uint32_t *dst) {  // whole warp
  if (MODE == kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     tc::smem_u32(dst))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tc::tmem_alloc<MODE == kSplit ? kLinMaxN : 2 * kLinMaxN>(dst);
  }
}
template <int MODE>
__device__ __forceinline__ void lin_tmem_free(uint32_t t) {
  if (MODE == kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(t) : "memory");
  else
    tc::tmem_dealloc<MODE == kSplit ? kLinMaxN : 2 * kLinMaxN>(t);
}

// one MMA: 32 bytes of K (32 e4m3 or 16 16-bit elements); PAIR: over both CTAs' tiles
template <bool PAIR, bool KIND8>
__device__ __forceinline__ void lin_mma(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc,
                                        uint32_t accumulate) {
#define LIN_MMA(GROUP, KIND)                                                              \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                          \
               "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" \
               ::"r"(d), "l"(da), "l"(db), "r"(idesc), "r"(accumulate) : "memory")
  if (PAIR) {
    if (KIND8) LIN_MMA("2", "f8f6f4"); else LIN_MMA("2", "f16");
  } else {
    if (KIND8) LIN_MMA("1", "f8f6f4"); else LIN_MMA("1", "f16");
  }
#undef LIN_MMA
}

// arrive on `bar` (PAIR: in both CTAs) once the MMAs issued so far have completed
template <bool PAIR>
__device__ __forceinline__ void lin_commit(uint64_t *bar) {
  if (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(tc::smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    tc::mma_commit(bar);
}

// TMA loads into this CTA's ring; `bar` is a shared::cluster address (PAIR: the leader's)
#define LIN_TMA(DIMS, COORDS, ...)                                                             \
  if (PAIR)                                                                                    \
    asm volatile("cp.async.bulk.tensor." DIMS                                                  \
                 ".shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "     \
                 "[%0], [%1, " COORDS "], [%2];" ::"r"(tc::smem_u32(dst)), "l"(map), "r"(bar), \
                 __VA_ARGS__ : "memory");                                                      \
  else                                                                                         \
    asm volatile("cp.async.bulk.tensor." DIMS                                                  \
                 ".shared::cluster.global.tile.mbarrier::complete_tx::bytes "                  \
                 "[%0], [%1, " COORDS "], [%2];" ::"r"(tc::smem_u32(dst)), "l"(map), "r"(bar), \
                 __VA_ARGS__ : "memory")
template <bool PAIR>
__device__ __forceinline__ void lin_load_2d(void *dst, const void *map, uint32_t bar, int x, int y) {
  LIN_TMA("2d", "{%3, %4}", "r"(x), "r"(y));
}
template <bool PAIR>
__device__ __forceinline__ void lin_load_3d(void *dst, const void *map, uint32_t bar, int x, int y,
                                            int z) {
  LIN_TMA("3d", "{%3, %4, %5}", "r"(x), "r"(y), "r"(z));
}
template <bool PAIR>
__device__ __forceinline__ void lin_load_5d(void *dst, const void *map, uint32_t bar, int x, int u,
                                            int v) {
  LIN_TMA("5d", "{%3, %4, %4, %5, %6}", "r"(x), "r"(0), "r"(u), "r"(v));
}
#undef LIN_TMA

// A tile: rows [r0, r0 + n) of expert e, feature tile ft.  Tiles run over `group` row tiles, then
// over the features, then over the groups: the CTAs working at one time then cover about as many
// token rows as weight rows, and both stay in L2 (32768 x 6144 tokens, larger than L2, by 4096
// features e4m3: 608 us with all row tiles first).
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
  const int g = i / (a.group * a.FT);
  const int gn = min(a.group, rt_n - g * a.group), j = i - g * a.group * a.FT;
  LinTile t;
  t.e = lo;
  t.ft = j / gn;
  t.r0 = b->off[lo] + (g * a.group + j - t.ft * gn) * a.BN;
  t.n = min(a.BN, b->off[lo + 1] - t.r0);
  return t;
}

// silu for an output of type TO: the fast form (relative error near 1e-6) where the result is
// rounded to 16 bits, the library's exponential and division where it stays fp32
template <typename TO>
__device__ __forceinline__ float lin_silu(float z) {
  return sizeof(TO) == 2 ? silu_fast(z) : silu_f(z);
}

template <typename TO>
__device__ __forceinline__ float lin_act(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z < 0.f ? 0.f : z;  // a NaN stays one
    case MOE_ACT_SILU: return lin_silu<TO>(z);
    case MOE_ACT_GELU: return 0.5f * z * erfcf(z * -0.70710678118654752f);  // z Phi(z)
    default: return z;
  }
}

// The epilogue of one warp: 32 weight rows (a lane each) of a tile.  Sixteen columns at a time
// are scaled, biased and activated in registers, staged as fp32 in shared memory, and read back
// so that a lane holds eight neighbouring features of one token: residual and output move as
// 16-byte accesses.  (Two-byte stores straight from the registers, 64 bytes a column, took 25
// instructions a column with their address arithmetic; the staged form takes about 7.)
template <typename TO, bool GATED>
struct LinOut {
  static constexpr int F = GATED ? 16 : 32;              // output features of the warp
  static constexpr int PITCH = GATED ? 16 : kLinPitch;   // floats per staged column
  static constexpr int LPR = F / 8;                      // lanes that hold one token's features
  static constexpr int RPI = 32 / LPR, IT = 16 / RPI;    // tokens per step, steps per chunk
  float sw, bi;      // weight row's scale and bias
  float *stage;
  TO *op;            // this lane's features of the tile's first token
  const TO *rp;
  long ldout, ldres;
  int nf, vec;       // features that this lane stores (0..8); all 8, 16-byte aligned
  int up, act;       // of two columns, the lower lanes of a SwiGLU warp finish the first,
                     // the upper lanes the second

  __device__ __forceinline__ LinOut(const LinArgs &a, const LinTile &t, int ft128, int quad,
                                    int lane, float *stage_)
      : stage(stage_), ldout(a.ldout), ldres(a.ldres), act(a.act) {
    up = GATED && lane >= 16;
    const int f0 = ft128 * (GATED ? 64 : kLinM) + quad * F;  // the warp's first feature
    const int f = f0 + (GATED ? lane & 15 : lane);
    const bool in = f < a.N;
    const long wi = (long)t.e * (GATED ? 2 * a.N : a.N) + f + (up ? a.N : 0);
    sw = a.w_scale && in ? a.w_scale[wi] : 1.f;
    bi = a.bias && in ? a.bias[wi] : 0.f;
    const int fo = f0 + 8 * (lane % LPR);
    nf = min(max(a.N - fo, 0), 8);
    vec = a.vec && nf == 8;
    op = (TO *)a.out + (long)(t.r0 + lane / LPR) * ldout + fo;
    rp = a.residual ? (const TO *)a.residual + (long)(t.r0 + lane / LPR) * ldres + fo : nullptr;
  }

  // the residual of columns c0 .. c0 + 15 (those below `end`), loaded ahead of the
  // accumulator's wait
  __device__ __forceinline__ void prefetch(int c0, int end, int lane, Pack<TO> (&rv)[IT]) const {
    if (!rp) return;
#pragma unroll
    for (int i = 0; i < IT; i++) {
      if (c0 + i * RPI + lane / LPR >= end) continue;
      const TO *r = rp + (long)(c0 + i * RPI) * ldres;
      rv[i] = vec ? load_pack<TO, kVec>(r, 0, 8) : load_run<TO>(r, nf);
    }
  }

  // accumulator values v of columns c0 .. c0 + 15, whose token scales are xs[0 .. 15]; columns
  // at `end` and beyond are left out
  __device__ __forceinline__ void finish(int c0, int end, int lane, const float *xs,
                                         const float (&v)[16], const Pack<TO> (&rv)[IT]) const {
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const float4 s4 = *(const float4 *)(xs + j);
      float z[4] = {fmaf(v[j] * s4.x, sw, bi), fmaf(v[j + 1] * s4.y, sw, bi),
                    fmaf(v[j + 2] * s4.z, sw, bi), fmaf(v[j + 3] * s4.w, sw, bi)};
      if (GATED) {
#pragma unroll
        for (int p = 0; p < 4; p += 2) {
          const float o = __shfl_xor_sync(0xffffffffu, up ? z[p] : z[p + 1], 16);
          const float g = up ? o : z[p], u = up ? z[p + 1] : o;
          stage[(j + p + up) * PITCH + (lane & 15)] = lin_silu<TO>(g) * u;
        }
      } else {
        if (act != MOE_ACT_NONE) {
#pragma unroll
          for (int p = 0; p < 4; p++) z[p] = lin_act<TO>(z[p], act);
        }
#pragma unroll
        for (int p = 0; p < 4; p++) stage[(j + p) * PITCH + lane] = z[p];
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < IT; i++) {
      const int c = i * RPI + lane / LPR;
      if (c0 + c < end) {
        alignas(16) float y[8];
        *(float4 *)y = *(const float4 *)(stage + c * PITCH + 8 * (lane % LPR));
        *(float4 *)(y + 4) = *(const float4 *)(stage + c * PITCH + 8 * (lane % LPR) + 4);
        if (rp) {
          float r[8];
          rv[i].get(r);
#pragma unroll
          for (int m = 0; m < 8; m++) y[m] += r[m];
        }
        Pack<TO> o;
        o.put(y);
        TO *d = op + (long)(c0 + i * RPI) * ldout;
        if (vec) store_pack<TO, kVec>(d, 0, 8, o);
        else store_run<TO>(d, nf, o);
      }
    }
    __syncwarp();
  }

  // the same of sums that are in registers
  template <int NI>
  __device__ __forceinline__ void tile_sums(const float (&sum)[NI][16], int n, int half, int lane,
                                            const float *xs) const {
#pragma unroll
    for (int i = 0; i < NI; i++) {
      const int c0 = 16 * half + 32 * i;
      if (c0 < n) {
        Pack<TO> rv[IT];
        prefetch(c0, n, lane, rv);
        finish(c0, n, lane, xs + 16 * i, sum[i], rv);
      }
    }
  }

  // the warp's chunks of a tile of n columns: the even (half = 0) or the odd ones
  __device__ __forceinline__ void tile(uint32_t taddr, int n, int half, int lane,
                                       const float *xs) const {
    for (int c0 = 16 * half; c0 < n; c0 += 32) {
      uint32_t v[16];
      float f[16];
      Pack<TO> rv[IT];
      __syncwarp();
      tc::tmem_ld16(taddr + c0, v);
      prefetch(c0, n, lane, rv);
      tc::tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; j++) f[j] = __uint_as_float(v[j]);
      finish(c0, n, lane, xs + (c0 >> 1) - 8 * half, f, rv);
    }
  }
};

// ---------------------------------------------------------------- epilogue, 16-bit outputs
// 16 tensor-memory lanes x 16 columns in the layout of an MMA's result: register 4 g + 2 h + i of
// lane l is row l / 4 + 8 h, column 8 g + 2 (l % 4) + i
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
// four 8 x 8 matrices of 16-bit values (word i of lane l: row l / 4, columns 2 (l % 4), + 1 of
// matrix i), stored transposed: lane 8 i + j gives the address of matrix i's column j
__device__ __forceinline__ void stmatrix_trans(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}
// v * s * w + b for two neighbouring columns
__device__ __forceinline__ float2 scale2(uint32_t v0, uint32_t v1, float2 s, float w, float b) {
  float2 r;
  asm("{\n\t.reg .b64 v, s, w, b;\n\tmov.b64 v, {%2, %3};\n\tmov.b64 s, {%4, %5};\n\t"
      "mov.b64 w, {%6, %6};\n\tmov.b64 b, {%7, %7};\n\tmul.rn.f32x2 v, v, s;\n\t"
      "fma.rn.f32x2 v, v, w, b;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(v0), "r"(v1), "f"(s.x), "f"(s.y), "f"(w), "f"(b));
  return r;
}
template <typename TO>
__device__ __forceinline__ uint32_t pack2(float2 y);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float2 y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(y.x, y.y);
  return *(const uint32_t *)&v;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float2 y) {
  const __half2 v = __floats2half2_rn(y.x, y.y);
  return *(const uint32_t *)&v;
}

// lin_act of N values with one look at `act` (32768 x 2048 features of K = 128 e4m3, bound by the
// epilogue: ReLU 53 us, with a look at each value 100; SiLU 69 and 130)
template <typename TO, int N>
__device__ __forceinline__ void lin_act_all(float (&z)[N], int act) {
  if (act == MOE_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; i++) z[i] = lin_act<TO>(z[i], MOE_ACT_RELU);
  } else if (act == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; i++) z[i] = lin_act<TO>(z[i], MOE_ACT_SILU);
  } else if (act == MOE_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; i++) z[i] = lin_act<TO>(z[i], MOE_ACT_GELU);
  }
}

// The same for a 16-bit output without a residual, which is rounded before it is staged: the
// accumulator is read in the layout of an MMA's result and transposed by stmatrix, gate and up
// values of a feature lie in one lane, and a chunk takes half the instructions of LinOut's (K =
// 1024, 32768 x 6144 e4m3, bound by the epilogue: 226 us with LinOut, 190 with this).
template <typename TO, bool GATED>
struct LinOut16 {
  static constexpr int F = GATED ? 16 : 32, LPR = F / 8, RPI = 32 / LPR, IT = 16 / RPI;
  static constexpr int PITCH = 2 * F + 16;  // bytes of a staged token
  float sw[4], bi[4];  // of the rows l / 4 + 8 r
  uint32_t put;        // where this lane's stmatrix column goes
  const uint8_t *get;
  TO *op;
  long ldout;
  int nf, vec, act;

  __device__ __forceinline__ LinOut16(const LinArgs &a, const LinTile &t, int ft128, int quad,
                                      int lane, float *stage)
      : ldout(a.ldout), act(a.act) {
    const int f0 = ft128 * (GATED ? 64 : kLinM) + quad * F;  // the warp's first feature
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const int f = f0 + (lane >> 2) + 8 * (GATED ? r & 1 : r);
      const bool in = f < a.N;
      const long wi = (long)t.e * (GATED ? 2 * a.N : a.N) + f + (GATED && r >= 2 ? a.N : 0);
      sw[r] = a.w_scale && in ? a.w_scale[wi] : 1.f;
      bi[r] = a.bias && in ? a.bias[wi] : 0.f;
    }
    // GATED: matrices (features 0-7, 8-15) x (tokens 0-7, 8-15); else features 0-31 x 8 tokens
    const int token = GATED ? 8 * (lane >> 4) + (lane & 7) : lane & 7;
    const int block = GATED ? (lane >> 3) & 1 : lane >> 3;
    put = tc::smem_u32(stage) + token * PITCH + block * 16;
    get = (const uint8_t *)stage + (lane / LPR) * PITCH + (lane % LPR) * 16;
    const int fo = f0 + 8 * (lane % LPR);
    nf = min(max(a.N - fo, 0), 8);
    vec = a.vec && nf == 8;
    op = (TO *)a.out + (long)(t.r0 + lane / LPR) * ldout + fo;
  }

  // columns c0 .. c0 + 15 of the accumulator at `taddr` (the warp's lanes, column c0), whose
  // token scales are xs[0 .. 15]; columns at `end` and beyond are left out
  __device__ __forceinline__ void finish(uint32_t taddr, int c0, int end, int lane,
                                         const float *xs) const {
    uint32_t v[2][8];
    tmem_ld_frag(taddr, v[0]);
    tmem_ld_frag(taddr + (16u << 16), v[1]);
    float2 s[2];
#pragma unroll
    for (int g = 0; g < 2; g++) s[g] = *(const float2 *)(xs + 8 * g + 2 * (lane & 3));
    tc::tmem_wait_ld();
    uint32_t w[2][4];
#pragma unroll
    for (int g = 0; g < 2; g++) {
      float2 z[4];
#pragma unroll
      for (int r = 0; r < 4; r++)
        z[r] = scale2(v[r >> 1][4 * g + 2 * (r & 1)], v[r >> 1][4 * g + 2 * (r & 1) + 1], s[g],
                      sw[r], bi[r]);
      if (GATED) {
#pragma unroll
        for (int r = 0; r < 2; r++)
          w[0][2 * g + r] = pack2<TO>(make_float2(lin_silu<TO>(z[r].x) * z[r + 2].x,
                                                  lin_silu<TO>(z[r].y) * z[r + 2].y));
      } else {
        float y[8] = {z[0].x, z[0].y, z[1].x, z[1].y, z[2].x, z[2].y, z[3].x, z[3].y};
        lin_act_all<TO>(y, act);
#pragma unroll
        for (int r = 0; r < 4; r++) w[g][r] = pack2<TO>(make_float2(y[2 * r], y[2 * r + 1]));
      }
    }
    stmatrix_trans(put, w[0]);
    if (!GATED) stmatrix_trans(put + 8 * PITCH, w[1]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < IT; i++) {
      if (c0 + i * RPI + lane / LPR < end) {
        const uint4 q = *(const uint4 *)(get + i * RPI * PITCH);
        TO *d = op + (long)(c0 + i * RPI) * ldout;
        if (vec) {
          *(uint4 *)d = q;
        } else {
          Pack<TO> o;
          o.w[0] = q.x, o.w[1] = q.y, o.w[2] = q.z, o.w[3] = q.w;
          store_run<TO>(d, nf, o);
        }
      }
    }
    __syncwarp();
  }

  // the warp's chunks of a tile of n columns: the even (half = 0) or the odd ones
  __device__ __forceinline__ void tile(uint32_t taddr, int n, int half, int lane,
                                       const float *xs) const {
    for (int c0 = 16 * half; c0 < n; c0 += 32)
      finish(taddr + c0, c0, n, lane, xs + (c0 >> 1) - 8 * half);
  }
};

// ---------------------------------------------------------------- waits that give up
// A wait gave up: the CTA's (PAIR: both CTAs') other waits end too, and the caller is told.  A
// limit runs out by the clock, so this may be the only role that sees it (the others may have
// finished, or go on when the GPU comes back to this context): whichever wait it is has to say so.
template <bool PAIR>
__device__ __forceinline__ void lin_give_up(const LinArgs &a, LinBars *b, uint32_t rank) {
  *(volatile int *)&b->abort_flag = 1;
  if (PAIR)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_cta(&b->abort_flag, rank ^ 1)), "r"(1)
                 : "memory");
  if (a.status) *a.status = MOE_ERR_TIMEOUT;
}

// the epilogue's wait for accumulator `buf`: in the test hook, for what nothing completes
__device__ __forceinline__ bool lin_wait_acc(const LinArgs &a, LinBars *b, int buf, uint32_t parity,
                                             volatile int *abort, uint32_t sleep_ns) {
  uint64_t *bar = a.never ? &b->never : &b->acc_full[buf];
  return __all_sync(0xffffffffu, tc::mbar_wait_backoff(bar, parity, abort,
                                                       a.never ? 0 : kLinWaitNs, sleep_ns));
}

// After a wait gave up and every role has left: copies and MMAs that were started end before the
// CTA frees its tensor memory and exits.  (Without a failure the epilogue's waits have seen to it.)
// full: the `n` barriers of the copies; OWN: every CTA's count its own.
template <bool PAIR, bool OWN = !PAIR>
__device__ __noinline__ void lin_drain(LinBars *b, uint64_t *full, int n, uint32_t rank, int warp,
                                       int lane) {
  if (warp == 0 && lane == 0) {
    // PAIR: the leader's barriers count both CTAs' copies; one that the second CTA had not started
    // is not worth a long wait
    for (int q = 0; q < n; q++)
      if ((b->armed >> q) & 1)
        wait_nofail(&full[q], (b->phases >> q) & 1, OWN ? kLinWaitNs : kLinLateNs);
    // the second CTA of a pair has no barrier of its own to wait on: its copies are loads of
    // some microseconds
    if (!OWN && rank) for (int i = 0; i < 1000; i++) __nanosleep(1000);
  } else if (warp == 1) {
    // the lane that issued the MMAs: elect gives the same one every time
    const bool leader = tc::elect_one();
    if (leader && b->issued) {
      lin_commit<PAIR>(&b->drain);
      wait_nofail(&b->drain, 0, kLinWaitNs);
    } else if (leader && PAIR && rank) {  // the leader's MMAs read this CTA's stages too
      wait_nofail(&b->drain, 0, kLinLateNs);
    }
    __syncwarp();
  }
}

// fp32 outputs: this warp's chunks of 16 columns (every second one of a tile's, NI of them at
// most), summed over the accumulators of a tile's k-blocks (CHUNK each); false when a wait gave up
template <int NI, int ACC, int CHUNK>
__device__ __forceinline__ bool lin_sum(const LinArgs &a, LinBars *b, uint32_t taddr, int n,
                                        int half, int lane, int kblocks, int &buf, uint32_t &bph,
                                        float (&sum)[NI][16], volatile int *abort) {
#pragma unroll
  for (int i = 0; i < NI; i++)
#pragma unroll
    for (int j = 0; j < 16; j++) sum[i][j] = 0.f;
  for (int k0 = 0; k0 < kblocks; k0 += CHUNK) {
    if (!lin_wait_acc(a, b, buf, bph, abort, 32)) return false;
    tc::fence_after_sync();
#pragma unroll
    for (int i = 0; i < NI; i++) {
      const int c0 = 16 * half + 32 * i;
      if (c0 < n) {
        uint32_t v[16];
        __syncwarp();
        tc::tmem_ld16(taddr + buf * ACC + c0, v);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; j++) sum[i][j] += __uint_as_float(v[j]);
      }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&b->acc_empty[buf]);
    if (buf) bph ^= 1;
    buf ^= 1;
  }
  return true;
}

// The experts' rows, clamped to [0, R] and kept in order, so that no offset leads out of x, and
// their row tiles; dense: one expert.  Called by every warp.
__device__ __forceinline__ void lin_offsets(const LinArgs &a, LinBars *b, int warp, int lane) {
  if (a.E == 0) {
    if (warp == 0 && lane == 0) {
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
}

// LinOut16's output type (fp32 outputs take LinOut)
template <typename TO>
using H16 = std::conditional_t<sizeof(TO) == 2, TO, __half>;

// The tiles of one epilogue warp.  acc: columns between the accumulators (EXACT: kLinAcc<float>).  The
// scales and biases of the next tile are loaded while this one is worked on.
template <typename OUT, bool PAIR, bool EXACT, int CHUNK = kLinExact>
__device__ __forceinline__ void lin_epilogue(const LinArgs &a, LinBars *b, uint32_t tbase, int tile,
                                             int ctas, int total, int kblocks, int acc,
                                             uint32_t rank, int warp, int lane, float *stage,
                                             volatile int *abort) {
  if (tile >= total) return;
  const int quad = warp & 3;         // the warp's quarter of the tensor-memory lanes
  const int half = (warp - 2) >> 2;  // of its chunks of 16 columns, the even or the odd ones
  float *xs = b->xs[warp - 2];
  float xr[kLinMaxN / 64];
  auto scales = [&](const LinTile &t) {  // 1 where there are none, 0 past the rows
#pragma unroll
    for (int i = 0; i < kLinMaxN / 64; i++) {
      const int k = 32 * i + lane, c = 32 * (k >> 4) + 16 * half + (k & 15);
      xr[i] = c < t.n ? a.x_scale ? a.x_scale[t.r0 + c] : 1.f : 0.f;
    }
  };
  LinTile t = lin_tile(a, b, tile);
  OUT o(a, t, PAIR ? 2 * t.ft + rank : t.ft, quad, lane, stage);
  scales(t);
  int buf = 0;
  uint32_t bph = 0;
  for (; tile < total; tile += ctas) {
    const OUT now = o;
    const int n = t.n;
#pragma unroll
    for (int i = 0; i < kLinMaxN / 64; i++) xs[32 * i + lane] = xr[i];
    __syncwarp();
    if (tile + ctas < total) {
      t = lin_tile(a, b, tile + ctas);
      o = OUT(a, t, PAIR ? 2 * t.ft + rank : t.ft, quad, lane, stage);
      scales(t);
    }
    if constexpr (EXACT) {
      float sum[kLinExactN / 32][16];
      if (!lin_sum<kLinExactN / 32, kLinAcc<float>, CHUNK>(
              a, b, tbase + ((uint32_t)(32 * quad) << 16), n, half, lane, kblocks, buf, bph, sum,
              abort)) {
        if (lane == 0) lin_give_up<PAIR>(a, b, rank);
        break;
      }
      now.tile_sums(sum, n, half, lane, xs);
      continue;
    }
    if (!lin_wait_acc(a, b, buf, bph, abort, 64)) {
      if (lane == 0) lin_give_up<PAIR>(a, b, rank);
      break;
    }
    tc::fence_after_sync();
    now.tile(tbase + buf * acc + ((uint32_t)(32 * quad) << 16), n, half, lane, xs);
    // the accumulator is read: the next tile may use it
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) {
      if (PAIR) arrive_in_cta(&b->acc_empty[buf], 0);
      else tc::mbar_arrive(&b->acc_empty[buf]);
    }
    if (buf) bph ^= 1;
    buf ^= 1;
  }
}

// kSplit: a tile's partial sums, joined; called by every thread of the CTA.
template <typename TO, bool GATED, int CHUNK = kLinExact>
__device__ __forceinline__ void lin_join(const LinArgs &a, LinBars *b, uint8_t *ring, float *stage,
                                         uint32_t tbase, int cta, int total, int kblocks,
                                         uint32_t rank, int tid, volatile int *abort) {
  const int warp = tid >> 5, lane = tid & 31;
  // A cluster has at most one tile.  Column c belongs to CTA c / cpc, whose exchange area
  // receives the partial sums [from CTA][four own columns][weight row][4]: a lane sends four
  // columns of its row in one store (a store a column, and a division to find its owner, took
  // 14 us where this takes 3: 200 columns between four CTAs).
  const int quad = warp & 3, half = (warp - 2) >> 2, row = quad * 32 + lane;
  const bool work = cta < total, mine = work && warp >= 2 && warp < 2 + kLinEpi;
  const int cpc = ((a.BN + a.split - 1) / a.split + 3) & ~3;
  const uint32_t inv = 65536u / cpc + 1;  // exact for columns below 256
  float *xs = b->xs[0];  // of all columns
  bool ok = mine;
  LinTile t{};
  if (work) t = lin_tile(a, b, cta);
  const LinOut<TO, GATED> o(a, t, t.ft, quad, lane, stage);
  const uint32_t taddr = tbase + ((uint32_t)(32 * quad) << 16);
  float sum[kLinExactSplitN / 32][16];  // fp32 outputs
  if (mine) {
    for (int c = tid - 64; c < kLinMaxN; c += 32 * kLinEpi)
      xs[c] = c < t.n ? a.x_scale ? a.x_scale[t.r0 + c] : 1.f : 0.f;
    if constexpr (lin_exact<TO>) {
      int buf = 0;
      uint32_t bph = 0;
      ok = lin_sum<kLinExactSplitN / 32, kLinAcc<TO>, CHUNK>(a, b, taddr, t.n, half, lane, kblocks,
                                                             buf, bph, sum, abort);
    } else {
      ok = lin_wait_acc(a, b, 0, 0, abort, 32);
      tc::fence_after_sync();
    }
    if (!ok && lane == 0) lin_give_up<false>(a, b, rank);
  }
  __syncwarp();
  cluster_wait();  // every CTA of the cluster has started: its memory may be written
  auto send = [&](int c0, const uint32_t (&v)[16]) {
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const uint32_t to = ((uint32_t)(c0 + j) * inv) >> 16;  // (c0 + j) / cpc
      if (c0 + j < t.n)
        store_in_cta(in_cta(ring + a.ring, to) +
                         (rank * cpc + c0 + j - to * cpc) * (kLinM * 4) + row * 16,
                     v + j);
    }
  };
  if (ok) {
    if constexpr (lin_exact<TO>) {
#pragma unroll
      for (int i = 0; i < kLinExactSplitN / 32; i++) {
        uint32_t v[16];
#pragma unroll
        for (int j = 0; j < 16; j++) v[j] = __float_as_uint(sum[i][j]);
        send(16 * half + 32 * i, v);
      }
    } else {
      for (int c0 = 16 * half; c0 < t.n; c0 += 32) {
        uint32_t v[16];
        __syncwarp();
        tc::tmem_ld16(taddr + c0, v);
        tc::tmem_wait_ld();
        send(c0, v);
      }
    }
  }
  __syncwarp();
  cluster_sync();
  if (ok) {
    const uint8_t *part = ring + a.ring + row * 16;
    const int c1 = min(t.n, (int)(rank + 1) * cpc);
    for (int c0 = rank * cpc + 16 * half; c0 < c1; c0 += 32) {
      float f[16];
      Pack<TO> rv[LinOut<TO, GATED>::IT];
      o.prefetch(c0, c1, lane, rv);
#pragma unroll
      for (int j = 0; j < 16; j++) f[j] = 0.f;
      for (int q = 0; q < a.split; q++)
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          if (c0 + j >= c1) continue;
          const float4 p =
              *(const float4 *)(part + (q * cpc + c0 + j - (int)rank * cpc) * (kLinM * 4));
          f[j] += p.x, f[j + 1] += p.y, f[j + 2] += p.z, f[j + 3] += p.w;
        }
      o.finish(c0, c1, lane, xs + c0, f, rv);
    }
  }
}

// Rows of no expert are zero: those before the first expert's and after the last one's.  Called by
// the epilogue's warps.
template <typename TO>
__device__ __forceinline__ void lin_zero_rows(const LinArgs &a, const LinBars *b, int tid) {
  const int lead = b->off[0], rest = lead + a.R - b->off[a.E];
  Pack<TO> zero;
  zero.clear();
  for (int i = blockIdx.x; i < rest; i += gridDim.x) {
    TO *row = (TO *)a.out + (long)(i < lead ? i : b->off[a.E] + i - lead) * a.ldout;
    for (int f = 8 * (tid - 64); f < a.N; f += 8 * 32 * kLinEpi) {
      if (a.vec && f + 8 <= a.N) store_pack<TO, kVec>(row, f, a.N, zero);
      else store_run<TO>(row + f, a.N - f, zero);
    }
  }
}

static inline PFN_cuTensorMapEncodeTiled_v12000 lin_encode() {
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

// The tensor maps of x and w, k-blocks of a.ke elements (128 bytes) of `xrows` token rows or `wrows`
// weight rows (SwiGLU: 16 gate rows, their 16 up rows, ...).
static inline bool lin_maps(const LinArgs &a, int K, const void *x, long ldx, const void *w, int es,
                            int xrows, CUtensorMap &xm, CUtensorMap &wm, int wrows = kLinM) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = lin_encode();
  if (!enc) return false;
  const CUtensorMapDataType dt = es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                         : CU_TENSOR_MAP_DATA_TYPE_UINT16;
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  {
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)a.R};
    const cuuint64_t strides[1] = {(cuuint64_t)ldx * es};
    const cuuint32_t box[2] = {(cuuint32_t)a.ke, (cuuint32_t)xrows};
    if (enc(&xm, dt, 2, const_cast<void *>(x), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  const cuuint64_t row = (cuuint64_t)K * es, ne = (cuuint64_t)std::max(1, a.E);
  CUresult cr;
  if (a.act == MOE_ACT_SWIGLU) {  // [e][N / 16][gate, up][16][K]
    const cuuint64_t dims[5] = {(cuuint64_t)K, 16, 2, (cuuint64_t)a.N / 16, ne};
    const cuuint64_t strides[4] = {row, row * a.N, row * 16, row * a.N * 2};
    const cuuint32_t box[5] = {(cuuint32_t)a.ke, 16, 2, (cuuint32_t)wrows / 32, 1};
    cr = enc(&wm, dt, 5, const_cast<void *>(w), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  } else {
    const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)a.N, ne};
    const cuuint64_t strides[2] = {row, row * a.N};
    const cuuint32_t box[3] = {(cuuint32_t)a.ke, (cuuint32_t)wrows, 1};
    cr = enc(&wm, dt, 3, const_cast<void *>(w), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  return cr == CUDA_SUCCESS;
}

// the product of 8-bit integers (linear_i8.cu); `a`: what does not depend on how it is cut
int linear_i8(LinArgs a, int K, const void *x, long ldx, const void *w, moe_dtype out_dtype,
              cudaStream_t st);
// the same for few token rows (linear_i8_few.cu); K < 131072, so that sums fit int32
int linear_i8_few(const LinArgs &a, int K, const void *x, long ldx, const void *w,
                  moe_dtype out_dtype, cudaStream_t st);

}  // namespace moe
