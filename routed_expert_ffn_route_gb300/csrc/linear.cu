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
// zero), warp 1 issues tcgen05.mma into one of two accumulators in tensor memory, warps 2-9
// turn the other accumulator into output.  For SwiGLU the weight map interleaves 16 gate
// rows with their 16 up rows, so that a gate and its up value sit 16 lanes apart in one warp.
//
// Measured, passes in a row under the power cap: 8192^3 bf16 658 us, 1.67 PFLOP/s; 32768 x 6144
// e4m3 by 4096 features 500 us, 3.3 PFLOP/s; 128 rows of 64 experts (6144 x 2 x 2048 e4m3) 202 us,
// weights at 6.9 TB/s.
#include "linear.cuh"

namespace moe {

template <typename TO, bool GATED, int MODE>
// (registers are given out to whole sets of four warps: 12 warps' worth a CTA, so that two
// kSplit CTAs share an SM only with the registers of 384 threads each)
__global__ void __launch_bounds__(MODE == kSplit ? 384 : kLinThreads, MODE == kSplit ? 2 : 1)
    linear_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                  const LinArgs a) {
  constexpr bool PAIR = MODE == kPair, SPLIT = MODE == kSplit;
  extern __shared__ uint8_t smraw[];
  uint8_t *ring = tc::align_smem_1024(smraw);
  const int xrows = PAIR ? a.BN / 2 : a.BN;  // token rows in this CTA's stages
  const int stage_bytes = (kLinM + xrows) * 128;
  LinBars *b = (LinBars *)(ring + a.ring + a.exchange);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // 16 columns of each epilogue warp on their way out: behind the barriers, kSplit: in the
  // ring, which is idle by then
  float *stage = (float *)(SPLIT ? ring : (uint8_t *)(b + 1)) +
                 ((warp - 2) & (kLinEpi - 1)) * (16 * kLinPitch);
  const uint32_t rank = MODE == kOne ? 0 : cluster_rank();
  if (SPLIT) cluster_arrive();  // waited for before the first store into another CTA
  if (tid == 32) {
    prefetch_map(&xmap);
    prefetch_map(&wmap);
  }
  if (tid == 0) {
    for (int s = 0; s < a.stages; s++) {
      tc::mbar_init(&b->full[s], 1);
      tc::mbar_init(&b->empty[s], 1);
    }
    for (int i = 0; i < 2; i++) {
      tc::mbar_init(&b->acc_full[i], 1);
      tc::mbar_init(&b->acc_empty[i], PAIR ? 2 * kLinEpi : kLinEpi);
    }
    tc::mbar_init(&b->drain, 1);
    tc::mbar_init(&b->never, 1);
    b->abort_flag = 0;
    b->armed = b->phases = 0;
    b->issued = 0;
    tc::fence_barrier_init();
  }
  __syncwarp();
  // tensor memory before the trigger: a successor may start as soon as every CTA has
  // triggered, and must not take columns that this grid still has to allocate
  if (warp == 0) lin_tmem_alloc<MODE>(&b->tmem);
  pdl_wait();
  pdl_trigger();
  lin_offsets(a, b, warp, lane);
  tc::fence_before_sync();
  if (PAIR) cluster_sync(); else __syncthreads();  // PAIR: barriers are ready in both CTAs
  tc::fence_after_sync();
  const uint32_t tbase = b->tmem;
  volatile int *abort = &b->abort_flag;
  // the tiles of this CTA (pair, cluster), and its part of K
  const int total = b->pre[max(1, a.E)] * a.FT;
  const int cta = PAIR ? blockIdx.x / 2 : SPLIT ? blockIdx.x / a.split : blockIdx.x;
  const int ctas = PAIR ? gridDim.x / 2 : SPLIT ? gridDim.x / a.split : gridDim.x;
  const int kb0 = SPLIT ? (int)((long)a.KB * rank / a.split) : 0;
  const int kb1 = SPLIT ? (int)((long)a.KB * (rank + 1) / a.split) : a.KB;
  const int chunk = lin_exact<TO> ? kLinExact : kb1 - kb0;  // k-blocks summed in tensor memory

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------- producer
      bool ok = true;
      uint32_t armed = 0, last_ph = 0;
      int s = 0;
      uint32_t ph = 0;
      for (int tile = cta; tile < total && ok; tile += ctas) {
        const LinTile t = lin_tile(a, b, tile);
        const int ft = PAIR ? 2 * t.ft + rank : t.ft;
        // the pair's MMAs take the first half of the columns from the leader
        const int row = t.r0 + (PAIR ? (int)rank * (round16(t.n) / 2) : 0);
        for (int kb = kb0; kb < kb1; kb++) {
          if (!tc::mbar_wait(&b->empty[s], ph ^ 1, abort, kLinWaitNs)) { ok = false; break; }
          uint8_t *st = ring + (size_t)s * stage_bytes;
          const uint32_t bar = PAIR ? in_cta(&b->full[s], 0) : tc::smem_u32(&b->full[s]);
          if (rank == 0 || !PAIR) {
            tc::mbar_arrive_expect_tx(&b->full[s], PAIR ? 2 * stage_bytes : stage_bytes);
            armed |= 1u << s;
            last_ph = (last_ph & ~(1u << s)) | (ph << s);
          }
          if (GATED)
            lin_load_5d<PAIR>(st, &wmap, bar, kb * a.ke, ft * (kLinM / 32), t.e);
          else
            lin_load_3d<PAIR>(st, &wmap, bar, kb * a.ke, ft * kLinM, t.e);
          lin_load_2d<PAIR>(st + kLinM * 128, &xmap, bar, kb * a.ke, row);
          if (++s == a.stages) s = 0, ph ^= 1;
        }
      }
      b->armed = armed;
      b->phases = last_ph;
      if (!ok) lin_give_up<PAIR>(a, b, rank);
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (one elected lane)
    const bool leader = tc::elect_one();
    bool ok = true, issued = false;
    int s = 0, buf = 0;
    uint32_t ph = 0, bph = 0;
    for (int tile = cta; tile < total && ok && (!PAIR || rank == 0); tile += ctas) {
      const LinTile t = lin_tile(a, b, tile);
      const uint32_t idesc = tc::idesc_f16(a.bf16, round16(t.n)) +
                             (PAIR ? (uint32_t)(kLinM >> 4) << 24 : 0u);  // M = 256
      for (int k0 = kb0; k0 < kb1 && ok; k0 += chunk) {  // an accumulator each
        int got = 1;
        if (leader) got = tc::mbar_wait(&b->acc_empty[buf], bph ^ 1, abort, kLinWaitNs);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t d = tbase + buf * kLinAcc<TO>;
        for (int kb = k0; kb < min(k0 + chunk, kb1); kb++) {
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
                lin_mma<PAIR, true>(d, da + 2 * kk, db + 2 * kk, idesc, (kb > k0) | (kk != 0));
            } else {
#pragma unroll
              for (int kk = 0; kk < 4; kk++)
                lin_mma<PAIR, false>(d, da + 2 * kk, db + 2 * kk, idesc, (kb > k0) | (kk != 0));
            }
            lin_commit<PAIR>(&b->empty[s]);
          }
          __syncwarp();
          issued = true;
          if (++s == a.stages) s = 0, ph ^= 1;
        }
        if (!ok) break;
        if (leader) lin_commit<PAIR>(&b->acc_full[buf]);
        __syncwarp();
        if (buf) bph ^= 1;
        buf ^= 1;
      }
    }
    if (leader) {
      b->issued = issued;
      if (!ok) lin_give_up<PAIR>(a, b, rank);
    }
  } else if (!SPLIT) {
    if (sizeof(TO) == 2 && !a.residual)
      lin_epilogue<LinOut16<H16<TO>, GATED>, PAIR, false>(a, b, tbase, cta, ctas, total, a.KB,
                                                          kLinMaxN, rank, warp, lane, stage, abort);
    else
      lin_epilogue<LinOut<TO, GATED>, PAIR, lin_exact<TO>>(a, b, tbase, cta, ctas, total, a.KB,
                                                           kLinMaxN, rank, warp, lane, stage, abort);
  }
  if (SPLIT)
    lin_join<TO, GATED>(a, b, ring, stage, tbase, cta, total, kb1 - kb0, rank, tid, abort);
  if (a.E && warp >= 2) lin_zero_rows<TO>(a, b, tid);
  __syncwarp();
  tc::fence_before_sync();
  if (PAIR) cluster_sync(); else __syncthreads();  // nobody still uses a peer's barriers
  tc::fence_after_sync();
  if (*abort) {  // the same for all threads: every role has left
    lin_drain<PAIR>(b, b->full, a.stages, rank, warp, lane);
    tc::fence_before_sync();
    if (PAIR) cluster_sync(); else __syncthreads();
    tc::fence_after_sync();
  }
  if (warp == 0) lin_tmem_free<MODE>(tbase);
}

template <typename TO, bool GATED, int MODE>
static size_t lin_smem(int bytes) {  // of the ring and the exchange
  const int more = 1024 + (int)sizeof(LinBars) + (MODE == kSplit ? 0 : kLinStage);
  set_dyn_smem((const void *)linear_kernel<TO, GATED, MODE>, kLinRing + more);
  // kSplit: never a third CTA on an SM.  Two hold all of its tensor memory; a third would wait
  // for columns while its cluster's other CTAs hold those that the first two wait for elsewhere.
  return std::max(bytes + more, MODE == kSplit ? 80 * 1024 : 0);
}

// Shared memory of a kSplit CTA.  It has one tile, so no more stages than its part of K has
// k-blocks; and, where that leaves four, little enough that two CTAs fit on an SM: clusters of
// eight otherwise leave SMs of a GPC idle (15 run at a time), and the next launch's CTAs can
// start beside this one's.
struct LinSplit {
  int stages, ring, exchange;
  bool two;  // two CTAs fit on an SM
};
static LinSplit lin_split(int BN, int split, int KB) {
  const int stage = (kLinM + BN) * 128;
  const int cpc = ((BN + split - 1) / split + 3) & ~3;
  LinSplit r;
  r.exchange = split * cpc * kLinM * 4;
  const int room = 112 * 1024 - (int)sizeof(LinBars) - 1024 - r.exchange;
  const int most = std::min({kLinStages, (kLinRing - r.exchange) / stage, (KB + split - 1) / split});
  const int small = std::min(most, room / stage);
  r.two = room >= kLinStage && small >= std::min(most, 4);
  r.stages = r.two ? small : most;
  r.ring = std::max(r.stages * stage, kLinStage);  // the output is staged there
  return r;
}

// Clusters of `split` CTAs that run at the same time on the current device with one CTA on an SM
// (0 where none do, or the query fails: the plan does without them)
static int lin_clusters(int split) {
  static DeviceAnswers known;
  int dev = 0;
  cudaGetDevice(&dev);
  return known.get(dev, split, [&]() {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split * dev_info().sms);
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = lin_smem<float, false, kSplit>(kLinRing);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)split, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, linear_kernel<float, false, kSplit>, &cfg) !=
        cudaSuccess) {
      cudaGetLastError();  // not an error of the call
      n = 0;
    }
    return n;
  });
}

struct LinPlan {
  int mode, BN, split;
  long tiles;
  bool sure;  // made with every answer
};

// How to cut the product: an estimate in SM cycles of each candidate, from what was measured.
// A k-block takes as long as its MMAs (2 cycles a column: the tensor cores' rate for 256 columns
// of 128 rows), its loads (2.45 cycles a 128-byte row, 52 bytes a cycle into an SM) or 430
// cycles, whichever is longest; joining a split tile takes 2000 cycles and 12 a column and
// other CTA.  One token of 6144 x 2048 bf16: split 8 6.8 us, 4 9.4, 2 15.0, none 24.9; 200
// tokens of 4096 x 4096: 112 columns split 2 13.4 us, 208 split 4 15.0, 64 unsplit 18.8.  Over 40
// random shapes (1 to 20000 rows, 64 to 8192 features, K 128 to 14336, 0 to 64 experts) the form
// taken is 3% slower than the fastest of all candidates in the mean, 26% at worst.
static LinPlan lin_make_plan(int R, int N, int E, int KB, bool gated, bool exact) {
  const int sms = dev_info().sms;
  // experts that get rows, and rows of one of them, when rows fall on experts evenly
  const double active = E > 1 ? E * (1.0 - std::pow(1.0 - 1.0 / E, R)) : 1.0;
  const double m = R / active;
  const int rows = gated ? 2 * N : N;
  const int clusters[3] = {lin_clusters(2), lin_clusters(4), lin_clusters(8)};
  const bool sure = clusters[0] > 0 && clusters[1] > 0 && clusters[2] > 0;
  LinPlan best{};
  double cost = 1e30;
  for (int mode = 0; mode < 3; mode++)
    for (int BN = 16; BN <= kLinMaxN; BN += 16)
      for (int split = mode == kSplit ? 2 : 1; split <= (mode == kSplit ? 8 : 1); split *= 2) {
        if (mode == kPair && (BN < 64 || BN % 32 || rows <= kLinM)) continue;
        if (split > KB) continue;
        if (exact && (mode == kPair || BN > (mode == kSplit ? kLinExactSplitN : kLinExactN)))
          continue;
        const int FT = (rows + (mode == kPair ? 255 : 127)) / (mode == kPair ? 256 : 128);
        // row tiles of an expert: exact when dense; by expert the last one is about half full,
        // and experts differ in size
        const double rt = E ? std::max(1.0, m / BN + 0.5) : (double)((R + BN - 1) / BN);
        const double tiles = active * rt * FT;
        const double cols = std::min((double)BN, m);
        const double kb = std::max({2.0 * cols, 430.0,
                                    2.45 * (kLinM + (mode == kPair ? BN / 2 : BN))});
        double c;
        if (mode == kSplit) {  // one tile a cluster
          const LinSplit sp = lin_split(BN, split, KB);
          const int fit = clusters[split == 2 ? 0 : split == 4 ? 1 : 2];
          if (sp.stages < 2 || tiles > fit * (sp.two ? 2 : 1)) continue;
          const double shared = tiles * split > sms ? 1.25 : 1.0;  // some SMs have two CTAs
          c = (KB + split - 1) / split * kb * shared + 2000 + 12.0 * BN * (split - 1);
        } else {
          const double width = mode == kPair ? sms / 2 : sms;
          const double waves = E ? std::max(1.0, tiles / width + 0.3) : std::ceil(tiles / width);
          c = waves * KB * kb + 500 + 4.0 * BN;  // the last tile's epilogue
        }
        if (c < cost * 0.999) {
          cost = c;
          best = LinPlan{mode, BN, split, 0, sure};
        }
      }
  const int FT = (rows + (best.mode == kPair ? 255 : 127)) / (best.mode == kPair ? 256 : 128);
  // at most so many tiles exist, however the rows fall on the experts
  const long rt = E ? (long)std::min(R, E) + R / best.BN : (R + best.BN - 1) / best.BN;
  best.tiles = rt * FT;
  return best;
}

// the plans of the last sizes seen by this thread (the estimate costs about a launch)
static LinPlan lin_plan(int R, int N, int E, int KB, bool gated, bool exact) {
  struct Entry {
    int R, N, E, KB, form, dev;
    LinPlan plan;
  };
  static thread_local Entry seen[64];
  const int form = 2 * gated + exact;
  int dev = 0;
  cudaGetDevice(&dev);
  const uint32_t h = ((uint32_t)R * 2654435761u) ^ ((uint32_t)N * 2246822519u) ^
                     ((uint32_t)KB * 3266489917u) ^ (uint32_t)(E * 4 + form) * 668265263u;
  Entry &e = seen[(h >> 16) & 63];
  if (e.R == R && e.N == N && e.E == E && e.KB == KB && e.form == form && e.dev == dev)
    return e.plan;
  const LinPlan plan = lin_make_plan(R, N, E, KB, gated, exact);
  if (plan.sure) e = Entry{R, N, E, KB, form, dev, plan};
  return plan;
}

template <typename TO, bool GATED, int MODE>
static int launch_linear(const CUtensorMap &xm, const CUtensorMap &wm, const LinArgs &a,
                         long tiles, cudaStream_t st) {
  auto *k = linear_kernel<TO, GATED, MODE>;
  const size_t smem = lin_smem<TO, GATED, MODE>(a.ring + a.exchange);
  const int per = MODE == kPair ? 2 : MODE == kSplit ? a.split : 1;  // CTAs per tile
  const long most = MODE == kSplit ? tiles : std::min(tiles, (long)dev_info().sms / per);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(most * per));
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)per, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = MODE == kOne ? 1 : 2;
  if (cudaLaunchKernelEx(&cfg, k, xm, wm, a) != cudaSuccess) return MOE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <typename TO, bool GATED>
static int launch_linear_m(const CUtensorMap &xm, const CUtensorMap &wm, const LinArgs &a,
                           const LinPlan &p, cudaStream_t st) {
  if constexpr (!lin_exact<TO>)
    if (p.mode == kPair) return launch_linear<TO, GATED, kPair>(xm, wm, a, p.tiles, st);
  return p.mode == kSplit ? launch_linear<TO, GATED, kSplit>(xm, wm, a, p.tiles, st)
                          : launch_linear<TO, GATED, kOne>(xm, wm, a, p.tiles, st);
}

template <typename TO>
static int launch_linear_t(const CUtensorMap &xm, const CUtensorMap &wm, const LinArgs &a,
                           const LinPlan &p, cudaStream_t st) {
  return a.act == MOE_ACT_SWIGLU ? launch_linear_m<TO, true>(xm, wm, a, p, st)
                                 : launch_linear_m<TO, false>(xm, wm, a, p, st);
}

// moe_linear; `never`: whose epilogue's waits run out
static int linear_call(int R, int N, int K, int n_experts, const void *x, long ldx,
                       moe_dtype dtype, const float *x_scale, const void *w,
                       const float *w_scale, const float *bias, moe_act act,
                       const void *residual, long ldres, const int32_t *offsets, void *out,
                       long ldout, moe_dtype out_dtype, int32_t *status, int never,
                       void *stream) {
  if (R < 0 || N <= 0 || K <= 0 || n_experts < 0) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DT_E4M3 && dtype != MOE_DT_BF16 && dtype != MOE_DT_F16 && dtype != MOE_DT_I8)
    return MOE_ERR_INVALID_ARG;
  if (out_dtype != MOE_DT_F32 && out_dtype != MOE_DT_BF16 && out_dtype != MOE_DT_F16)
    return MOE_ERR_INVALID_ARG;
  if (act < MOE_ACT_NONE || act > MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  const bool gated = act == MOE_ACT_SWIGLU;
  const int es = dtype == MOE_DT_E4M3 || dtype == MOE_DT_I8 ? 1 : 2;
  if (n_experts > kLinMaxE || K % 16 || (gated && N % 16)) return MOE_ERR_UNSUPPORTED;
  // sizes that the 32-bit tile and coordinate arithmetic covers
  if (R > (1 << 24) || N > (1 << 20) || K > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (!x || !w || !out || ldx < K || ldout < N || (residual && ldres < N) ||
      (n_experts && !offsets))
    return MOE_ERR_INVALID_ARG;
  const uintptr_t eo = out_dtype == MOE_DT_F32 ? 4 : 2;
  if (R == 1) ldx = K;  // there is no next row for the distance to lead to
  if ((uintptr_t)x % 16 || (uintptr_t)w % 16 || (uintptr_t)(ldx * es) % 16 ||
      ((uintptr_t)out | (uintptr_t)residual) % eo ||
      ((uintptr_t)x_scale | (uintptr_t)w_scale | (uintptr_t)bias | (uintptr_t)offsets |
       (uintptr_t)status) % 4)
    return MOE_ERR_INVALID_ARG;

  LinArgs a{};
  a.x_scale = x_scale;
  a.w_scale = w_scale;
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.offsets = n_experts ? offsets : nullptr;
  a.status = status;
  a.never = never;
  a.ldres = ldres;
  a.ldout = ldout;
  a.R = R;
  a.N = N;
  a.E = n_experts;
  a.ke = 128 / es;
  a.KB = (K + a.ke - 1) / a.ke;
  a.act = act;
  a.vec = ((uintptr_t)out | (uintptr_t)residual | (uintptr_t)(ldout * eo) |
           (uintptr_t)(residual ? ldres * eo : 0)) % 16 == 0;
  const cudaStream_t st = (cudaStream_t)stream;
  if (dtype == MOE_DT_I8) return linear_i8(a, K, x, ldx, w, out_dtype, st);

  a.kind8 = es == 1;
  a.bf16 = dtype == MOE_DT_BF16;
  const LinPlan plan = lin_plan(R, N, n_experts, a.KB, gated, out_dtype == MOE_DT_F32);
  const int xrows = plan.mode == kPair ? plan.BN / 2 : plan.BN;
  const int ftw = (plan.mode == kPair ? 2 * kLinM : kLinM) / (gated ? 2 : 1);
  a.BN = plan.BN;
  a.split = plan.split;
  const int stage = (kLinM + xrows) * 128;
  a.stages = std::min(kLinStages, kLinRing / stage);
  a.ring = a.stages * stage;
  if (plan.mode == kSplit) {
    const LinSplit sp = lin_split(a.BN, a.split, a.KB);
    a.stages = sp.stages;
    a.ring = sp.ring;
    a.exchange = sp.exchange;
  }
  a.FT = (N + ftw - 1) / ftw;
  // as many token rows as weight rows at one time, when every SM works on a tile
  const double at_once = plan.mode == kPair ? dev_info().sms / 2 : dev_info().sms;
  a.group = std::max(1, (int)std::lround(std::sqrt(at_once * ftw * (gated ? 2 : 1) / a.BN)));

  CUtensorMap xm, wm;
  if (!lin_maps(a, K, x, ldx, w, es, xrows, xm, wm)) return MOE_ERR_CUDA;
  return out_dtype == MOE_DT_F32    ? launch_linear_t<float>(xm, wm, a, plan, st)
         : out_dtype == MOE_DT_BF16 ? launch_linear_t<__nv_bfloat16>(xm, wm, a, plan, st)
                                    : launch_linear_t<__half>(xm, wm, a, plan, st);
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_linear(int R, int N, int K, int n_experts, const void *x, long ldx, moe_dtype dtype,
               const float *x_scale, const void *w, const float *w_scale, const float *bias,
               moe_act act, const void *residual, long ldres, const int32_t *offsets, void *out,
               long ldout, moe_dtype out_dtype, int32_t *status, void *stream) {
  return linear_call(R, N, K, n_experts, x, ldx, dtype, x_scale, w, w_scale, bias, act, residual,
                     ldres, offsets, out, ldout, out_dtype, status, 0, stream);
}

int moe_debug_linear_timeout(int R, int N, int K, int n_experts, const void *x, long ldx,
                             moe_dtype dtype, const float *x_scale, const void *w,
                             const float *w_scale, const float *bias, moe_act act,
                             const void *residual, long ldres, const int32_t *offsets, void *out,
                             long ldout, moe_dtype out_dtype, int32_t *status, void *stream) {
  return linear_call(R, N, K, n_experts, x, ldx, dtype, x_scale, w, w_scale, bias, act, residual,
                     ldres, offsets, out, ldout, out_dtype, status, 1, stream);
}

}  // extern "C"
