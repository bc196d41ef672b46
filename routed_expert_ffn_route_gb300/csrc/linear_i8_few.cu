// linear_i8_few.cu -- the product of 8-bit integers for few token rows, which reads weights and does
// little else: mma.sync on the codes themselves, summed in int32, exact.
//
// A tcgen05 MMA takes at least 112 cycles for its 128 weight rows, however few columns it has, and
// the codes go through it as fp16: 128 rows of 128 codes are eight of them, 18 bytes of weights a
// cycle and SM where memory brings 23.  mma.sync m16n8k32 takes int8 as it is.
//
// A persistent CTA per SM walks the tiles of all experts: 16 MR weight rows by 8 NT token rows of one
// expert.  Warp 0 loads stages of 16 KB of weights (8 / MR k-blocks of 128 codes by 16 MR rows) and
// their part of the token rows into a ring by TMA; of warps 2-9 each takes 16 weight rows of one
// k-block of every stage.  The order of K within a k-block is free as long as weights and tokens
// have the same: lane l takes the 16-byte chunks 2 (l % 4) + h of the rows l / 4 and l / 4 + 8, which
// are its operands of two MMAs as they lie, and touch every bank once.  With SwiGLU the second of
// these rows is the up row of the first one's feature.  Narrow tiles (MR below 8: there are few) join
// the sums of the warps that share K in shared memory.
//
// Measured: one row of 6144 x 2048 5.2 us (clusters that split K, linear_i8.cu: 10.9); 8 rows of
// 4096 x 155648 96 us, weights at 6.6 TB/s (16 rows: 163, linear_i8.cu 113); 128 rows of 64 experts
// (6144 x 2 x 2048) 197 to 220 us (250 to 270).
#include "linear.cuh"

namespace moe {

constexpr int kFewWarps = 8;
constexpr int kFewThreads = 64 + 32 * kFewWarps;
constexpr int kFewW = 16 * 1024;  // bytes of weights a stage
constexpr int kFewPart = 8 * 32;  // sums of a warp on their way to another

struct FewBars : LinBars {
  int part[2][kFewWarps][kFewPart];
};

__device__ __forceinline__ void few_mma(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct FewArgs : LinArgs {
  int wide;  // a stage's k-blocks come in one load
};

// the loads of a stage: weights [e][k-block][row][128], or [gate, up of e][k-block][group][16][128]
__device__ __forceinline__ void few_load_4d(void *dst, const void *map, uint32_t bar, int row,
                                            int kb, int e) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(tc::smem_u32(dst)),
      "l"(map), "r"(bar), "r"(0), "r"(row), "r"(kb), "r"(e)
      : "memory");
}
__device__ __forceinline__ void few_load_5d(void *dst, const void *map, uint32_t bar, int group,
                                            int kb, int half) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %3, %4, %5, %6}], [%2];" ::"r"(tc::smem_u32(dst)),
      "l"(map), "r"(bar), "r"(0), "r"(group), "r"(kb), "r"(half)
      : "memory");
}

// Tensor maps that see K as k-blocks of 128 codes, which it has to be whole ones of: a box holds
// `kj` k-blocks.
static bool few_maps(const LinArgs &a, int K, const void *x, long ldx, const void *w, int kj,
                     int wrows, CUtensorMap &xm, CUtensorMap &wm) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = lin_encode();
  if (!enc) return false;
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  const cuuint64_t row = (cuuint64_t)K, kb = (cuuint64_t)K / 128;
  const cuuint64_t ne = (cuuint64_t)std::max(1, a.E);
  auto make = [&](CUtensorMap &m, const void *p, int n, const cuuint64_t *dims,
                  const cuuint64_t *strides, const cuuint32_t *box) {
    return enc(&m, CU_TENSOR_MAP_DATA_TYPE_UINT8, n, const_cast<void *>(p), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t xd[3] = {128, (cuuint64_t)a.R, kb}, xs[2] = {(cuuint64_t)ldx, 128};
  const cuuint32_t xb[3] = {128, (cuuint32_t)a.BN, (cuuint32_t)kj};
  if (!make(xm, x, 3, xd, xs, xb)) return false;
  if (a.act == MOE_ACT_SWIGLU) {
    const cuuint64_t d[5] = {128, 16, (cuuint64_t)a.N / 16, kb, 2 * ne};
    const cuuint64_t s[4] = {row, row * 16, 128, row * a.N};
    const cuuint32_t box[5] = {128, 16, (cuuint32_t)wrows / 32, (cuuint32_t)kj, 2};
    return make(wm, w, 5, d, s, box);
  }
  const cuuint64_t d[4] = {128, (cuuint64_t)a.N, kb, ne}, s[3] = {row, 128, row * a.N};
  const cuuint32_t box[4] = {128, (cuuint32_t)wrows, (cuuint32_t)kj, 1};
  return make(wm, w, 4, d, s, box);
}

template <typename TO, bool GATED, int MR, int NT>
__global__ void __launch_bounds__(kFewThreads, 1)
    linear_i8_few_kernel(const __grid_constant__ CUtensorMap xmap,
                         const __grid_constant__ CUtensorMap wmap, const FewArgs a) {
  constexpr int KJ = kFewWarps / MR;             // k-blocks a stage
  constexpr int F = GATED ? 8 * MR : 16 * MR;    // features a tile
  constexpr int kWB = 16 * MR * 128, kXB = 8 * NT * 128, kStage = kFewW + KJ * kXB;
  extern __shared__ uint8_t smraw[];
  uint8_t *ring = tc::align_smem_1024(smraw);
  FewBars *b = (FewBars *)(ring + a.ring);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 32) {
    prefetch_map(&xmap);
    prefetch_map(&wmap);
  }
  if (tid == 0) {
    for (int s = 0; s < a.stages; s++) {
      tc::mbar_init(&b->full[s], 1);
      tc::mbar_init(&b->empty[s], kFewWarps);
    }
    tc::mbar_init(&b->never, 1);
    b->abort_flag = 0;
    b->armed = b->phases = 0;
    b->issued = 0;
    tc::fence_barrier_init();
  }
  __syncwarp();
  pdl_wait();
  pdl_trigger();
  lin_offsets(a, b, warp, lane);
  __syncthreads();
  volatile int *abort = &b->abort_flag;
  const int total = b->pre[max(1, a.E)] * a.FT;
  const int steps = (a.KB + KJ - 1) / KJ;  // stages a tile

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------- producer
      bool ok = true;
      uint32_t armed = 0, last_ph = 0;
      int s = 0;
      uint32_t ph = 0;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const LinTile t = lin_tile(a, b, tile);
        for (int i = 0; i < steps; i++) {
          if (!tc::mbar_wait(&b->empty[s], ph ^ 1, abort, kLinWaitNs)) { ok = false; break; }
          uint8_t *st = ring + s * kStage;
          const uint32_t bar = tc::smem_u32(&b->full[s]);
          tc::mbar_arrive_expect_tx(&b->full[s], kStage);
          armed |= 1u << s;
          last_ph = (last_ph & ~(1u << s)) | (ph << s);
          if (KJ > 1 && a.wide) {  // k-blocks past K read as zero
            if (GATED) few_load_5d(st, &wmap, bar, t.ft * (F / 16), i * KJ, 2 * t.e);
            else few_load_4d(st, &wmap, bar, t.ft * F, i * KJ, t.e);
            lin_load_3d<false>(st + kFewW, &xmap, bar, 0, t.r0, i * KJ);
          } else {
#pragma unroll
            for (int j = 0; j < KJ; j++) {
              const int k = (i * KJ + j) * 128;
              if (GATED)
                lin_load_5d<false>(st + j * kWB, &wmap, bar, k, t.ft * (F / 16), t.e);
              else
                lin_load_3d<false>(st + j * kWB, &wmap, bar, k, t.ft * F, t.e);
              lin_load_2d<false>(st + kFewW + j * kXB, &xmap, bar, k, t.r0);
            }
          }
          if (++s == a.stages) s = 0, ph ^= 1;
        }
      }
      b->armed = armed;
      b->phases = last_ph;
      if (!ok) lin_give_up<false>(a, b, 0);
    }
  } else if (warp >= 2) {
    // ------------------------------------------------ 16 weight rows of one k-block each
    const int cw = warp - 2, rb = cw % MR, kj = cw / MR, g = lane >> 2, q = lane & 3;
    const int row0 = GATED ? 32 * (rb >> 1) + 8 * (rb & 1) + g : 16 * rb + g;
    // (GATED, wide: MR = 2, all k-blocks' gate rows come before the up rows)
    const bool apart = GATED && KJ > 1 && a.wide;
    const uint8_t *wp0 = ring + kj * (apart ? kWB / 2 : kWB) + row0 * 128;
    const uint8_t *wp1 = wp0 + (apart ? kFewW / 2 : (GATED ? 16 : 8) * 128);
    const uint8_t *xp = ring + kFewW + kj * kXB + g * 128;
    const int f0 = GATED ? 16 * (rb >> 1) + 8 * (rb & 1) + g : 16 * rb + g;  // of the tile
    bool ok = true;
    int s = 0, buf = 0;
    uint32_t ph = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x, buf ^= 1) {
      const LinTile t = lin_tile(a, b, tile);
      int acc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int i = 0; i < 4; i++) acc[j][i] = 0;
      for (int i = 0; i < steps && ok; i++) {
        uint64_t *bar = a.never ? &b->never : &b->full[s];
        if (!__all_sync(0xffffffffu, tc::mbar_test_wait(bar, a.never ? 0 : ph)))
          ok = __all_sync(0xffffffffu, tc::mbar_wait_spin(bar, a.never ? 0 : ph, abort,
                                                          a.never ? 0 : kLinWaitNs));
        if (!ok) break;
        uint4 w0[2], w1[2], x[NT][2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const int at = s * kStage + (((2 * q + h) ^ g) << 4);
          w0[h] = *(const uint4 *)(wp0 + at);
          w1[h] = *(const uint4 *)(wp1 + at);
#pragma unroll
          for (int j = 0; j < NT; j++) x[j][h] = *(const uint4 *)(xp + j * 1024 + at);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&b->empty[s]);
        if (++s == a.stages) s = 0, ph ^= 1;
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int j = 0; j < NT; j++) {
            few_mma(acc[j], w0[h].x, w1[h].x, w0[h].y, w1[h].y, x[j][h].x, x[j][h].y);
            few_mma(acc[j], w0[h].z, w1[h].z, w0[h].w, w1[h].w, x[j][h].z, x[j][h].w);
          }
      }
      if (MR < kFewWarps) {  // warps rb, rb + MR, ... share K: the first joins their sums
        if (kj) {
#pragma unroll
          for (int i = 0; i < 4 * NT; i++) b->part[buf][cw][i * 32 + lane] = acc[i / 4][i % 4];
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (kj) continue;
#pragma unroll
        for (int w = 1; w < KJ; w++)
#pragma unroll
          for (int i = 0; i < 4 * NT; i++) acc[i / 4][i % 4] += b->part[buf][rb + w * MR][i * 32 + lane];
      }
      if (!ok) continue;
      // features f0 (sums 0, 1) and, without SwiGLU, f0 + 8 (2, 3); tokens 2 q and 2 q + 1
#pragma unroll
      for (int m = 0; m < (GATED ? 1 : 2); m++) {
        const int f = t.ft * F + f0 + 8 * m;
        if (f >= a.N) continue;
        const long wi = (long)t.e * (GATED ? 2 * a.N : a.N) + f;
        const float sw = a.w_scale ? a.w_scale[wi] : 1.f, bi = a.bias ? a.bias[wi] : 0.f;
        float su = 1.f, bu = 0.f;
        if (GATED) {
          su = a.w_scale ? a.w_scale[wi + a.N] : 1.f;
          bu = a.bias ? a.bias[wi + a.N] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
          for (int i = 0; i < 2; i++) {
            const int r = 8 * j + 2 * q + i;
            if (r >= t.n) continue;
            const long row = t.r0 + r;
            const float xs = a.x_scale ? a.x_scale[row] : 1.f;
            const float z = fmaf((float)acc[j][2 * m + i] * xs, sw, bi);
            float y;
            if (GATED) y = lin_silu<TO>(z) * fmaf((float)acc[j][2 + i] * xs, su, bu);
            else y = lin_act<TO>(z, a.act);
            if (a.residual) y += (float)((const TO *)a.residual)[row * a.ldres + f];
            ((TO *)a.out)[row * a.ldout + f] = (TO)y;
          }
      }
    }
    if (!ok && lane == 0) lin_give_up<false>(a, b, 0);
  }
  if (a.E && warp >= 2) lin_zero_rows<TO>(a, b, tid);
  __syncwarp();
  __syncthreads();
  if (*abort) lin_drain<false, true>(b, b->full, a.stages, 0, warp, lane);
}

template <typename TO, bool GATED, int MR, int NT>
static int launch_few(const LinArgs &base, int K, const void *x, long ldx, const void *w,
                      cudaStream_t st) {
  FewArgs a{};
  (LinArgs &)a = base;
  auto *k = linear_i8_few_kernel<TO, GATED, MR, NT>;
  constexpr int F = GATED ? 8 * MR : 16 * MR, stage = kFewW + kFewWarps / MR * 8 * NT * 128;
  const int more = 1024 + (int)sizeof(FewBars);
  a.BN = 8 * NT;
  a.FT = (a.N + F - 1) / F;
  a.group = 1;  // an expert's features one after the other
  a.stages = std::min(kLinStages, kLinRing / stage);
  a.ring = a.stages * stage;
  CUtensorMap xm, wm;
  a.wide = MR < kFewWarps && K % 128 == 0;
  if (!(a.wide ? few_maps(a, K, x, ldx, w, kFewWarps / MR, 16 * MR, xm, wm)
               : lin_maps(a, K, x, ldx, w, 1, a.BN, xm, wm, 16 * MR)))
    return MOE_ERR_CUDA;
  // at most so many tiles exist, however the rows fall on the experts
  const long rt = a.E ? (long)std::min(a.R, a.E) + a.R / a.BN : (a.R + a.BN - 1) / a.BN;
  set_dyn_smem((const void *)k, kLinRing + more);
  const cudaError_t e = launch_pdl(k, dim3((unsigned)std::min(rt * a.FT, (long)dev_info().sms)),
                                   dim3(kFewThreads), (size_t)(a.ring + more), st, xm, wm, a);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename TO, bool GATED>
static int launch_few_g(const LinArgs &a, int K, const void *x, long ldx, const void *w, int MR,
                        int NT, cudaStream_t st) {
  if (MR == 8)
    return NT == 1 ? launch_few<TO, GATED, 8, 1>(a, K, x, ldx, w, st)
                   : launch_few<TO, GATED, 8, 2>(a, K, x, ldx, w, st);
  if (GATED || MR == 2)
    return NT == 1 ? launch_few<TO, GATED, 2, 1>(a, K, x, ldx, w, st)
                   : launch_few<TO, GATED, 2, 2>(a, K, x, ldx, w, st);
  if constexpr (!GATED)
    return NT == 1 ? launch_few<TO, GATED, 1, 1>(a, K, x, ldx, w, st)
                   : launch_few<TO, GATED, 1, 2>(a, K, x, ldx, w, st);
  return MOE_ERR_UNSUPPORTED;
}

template <typename TO>
static int launch_few_t(const LinArgs &a, int K, const void *x, long ldx, const void *w, int MR,
                        int NT, cudaStream_t st) {
  return a.act == MOE_ACT_SWIGLU ? launch_few_g<TO, true>(a, K, x, ldx, w, MR, NT, st)
                                 : launch_few_g<TO, false>(a, K, x, ldx, w, MR, NT, st);
}

int linear_i8_few(const LinArgs &a, int K, const void *x, long ldx, const void *w,
                  moe_dtype out_dtype, cudaStream_t st) {
  const int rows = a.act == MOE_ACT_SWIGLU ? 2 * a.N : a.N, sms = dev_info().sms;
  const double active = a.E > 1 ? a.E * (1.0 - std::pow(1.0 - 1.0 / a.E, a.R)) : 1.0;
  auto tiles = [&](int MR) { return active * ((rows + 16 * MR - 1) / (16 * MR)); };
  // Tiles of 128 weight rows where there are plenty (64 experts, 128 rows: 205 us, of 32 rows 251),
  // else of 32 (8 experts, 16 rows of 6144 x 2 x 2048: 35 us for 40), else of 16 (one row of 6144 x
  // 2048: 5.2 us for 6.8).
  const int MR = tiles(8) >= 6 * sms ? 8 : tiles(2) >= 0.75 * sms ? 2 : 1;
  const int NT = a.E <= 1 && a.R > 8 ? 2 : 1;
  return out_dtype == MOE_DT_F32    ? launch_few_t<float>(a, K, x, ldx, w, MR, NT, st)
         : out_dtype == MOE_DT_BF16 ? launch_few_t<__nv_bfloat16>(a, K, x, ldx, w, MR, NT, st)
                                    : launch_few_t<__half>(a, K, x, ldx, w, MR, NT, st);
}

}  // namespace moe
