// linear_i8.cu -- matrix product of 8-bit integers with a scale for each token and channel, dense
// or grouped by expert: linear.cu's product and epilogue for int8 codes.
//
// The chip's tensor cores have no fast 8-bit integer kind.  A code goes through them as an fp16
// number, which holds it exactly; a product of two is below 2^14 + 1 and a sum of 1024 of them at
// most 2^24, so every sum of kI8Exact k-blocks is the whole number that it stands for.
//
// On the way to the MMA there is one more step than in linear.cu: warp 0 loads k-blocks of 128
// codes a row (a ring of raw stages), warps 10-17 turn them into fp16 k-blocks of 64 elements,
// warp 1 issues the MMAs on those, warps 2-9 are the epilogue.  The weights' half goes to tensor
// memory, a row a lane, from where the MMA takes its A operand; the tokens' half goes to shared
// memory.  (Both through shared memory, whose bandwidth then bounds the product, 8192 codes of
// K by 128 + 128 rows: 720 us for 4095 x 14336 x 4096.)
//
// Code b becomes fp16 by placing b ^ 0x80 in the mantissa of 1024 and taking 1152 off: 20
// instructions for 16 codes.  Two sets of four converter warps take the k-blocks in turn.
// Sub-block h of a k-block is the 16-byte chunks 2 i + h of each row, for x and w alike, so that
// reads of the swizzled raw rows and writes of the swizzled fp16 rows touch every bank once.
//
// Measured, passes in a row under the power cap: 8192^3 640 us, 1.72 PFLOP/s (linear.cu on bf16: 658);
// 4095 x 14336 by 4096 features with bias and residual 298 to 314 us; 32768 rows of 32 experts
// (6144 x 2 x 2048) 1010 to 1067 us, 1.55 to 1.63 PFLOP/s; fp32 outputs of 4096^3 153 us.
#include "linear.cuh"

namespace moe {

constexpr int kI8Threads = kLinThreads + 256;
constexpr int kI8Set = 4;     // converter warps of a set; two sets
constexpr int kI8Exact = 16;  // sub-blocks (1024 products) summed in tensor memory: exact
// Tensor memory: two accumulators, then the weights' sub-blocks, 32 columns each.  (Eight slots, where
// the accumulators are narrow: no gain.)
constexpr int kI8A = 2 * kI8MaxN;
static_assert(kI8A + 32 * kI8Slots == 512, "all of tensor memory");
template <typename TO>
constexpr int kI8Acc = lin_exact<TO> ? kLinAcc<TO> : kI8MaxN;

struct I8Args : LinArgs {
  int conv;  // bytes of a token sub-block; kI8Slots of them behind the raw stages
};
// empty: of this CTA's raw stages.  raw_full: two barriers a stage, which its k-blocks take in turn
// (LinBars' full is not used).  A wait tests one parity bit and cannot tell a phase from the one two
// before it.  With one barrier and an odd number of stages, a set comes to stages whose last k-block
// was the other set's: where that has not landed, the wait passes at once (three stages; with five and
// more the wait for the slots holds the set back).  With two, k-block i shares its barrier with k-block
// i + 2 stages, an even number on, so that one set waits for every phase of it.
struct I8Bars : LinBars {
  uint64_t raw_full[2][kLinStages];
  uint64_t conv_full[kI8Slots], conv_empty[kI8Slots];
};
// place in a ring of raw stages: the stage, which of its barriers, and the parity of that one's phase
struct I8Place {
  int s = 0;
  uint32_t lap = 0, ph = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) s = 0, ph ^= lap, lap ^= 1;
  }
};

// A converter warp's sub-block is handed to the pair's MMAs by an arrive in CTA `rank`, without a
// release at cluster scope.  What the MMAs read of this CTA is in its own shared and tensor memory and
// is read by its own tensor core, not by a thread of the other CTA; it is there before the arrive is
// issued: fence.proxy.async in every lane has the shared-memory writes seen by the async proxy, as
// which the tensor core reads, tcgen05.wait::st has the tensor-memory writes complete, and __syncwarp
// puts every lane's before the one that arrives.  So the order is carried by those two and by the
// barrier's phase, not by what the arrive releases.  A release at cluster scope would also wait for all
// that the SM has in flight: 8192^3 1517 us instead of 641, where an otherwise idle warp issues it.
__device__ __forceinline__ void i8_arrive_in_cta(uint64_t *bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_cta(bar, rank)) : "memory");
}

// one MMA with its A operand in tensor memory: 16 of K; PAIR: over both CTAs' tiles
template <bool PAIR>
__device__ __forceinline__ void i8_mma(uint32_t d, uint32_t ta, uint64_t db, uint32_t idesc,
                                       uint32_t accumulate) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(ta), "l"(db), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    tc::mma_ts(d, ta, db, idesc, accumulate);
}

// four codes as fp16 numbers
__device__ __forceinline__ void i8_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const uint32_t x = w ^ 0x80808080u;
  const uint32_t l = __byte_perm(x, 0x64646464u, 0x4140), h = __byte_perm(x, 0x64646464u, 0x4342);
  const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 a = __hsub2(*(const __half2 *)&l, off), b = __hsub2(*(const __half2 *)&h, off);
  lo = *(const uint32_t *)&a;
  hi = *(const uint32_t *)&b;
}

// This lane's row of sub-block h of the raw weights as fp16, as it goes to 32 columns of tensor
// memory.  `rows`: the warp's 32 rows, which are its quarter of the lanes.
__device__ __forceinline__ void i8_load_row(const uint8_t *rows, int h, int lane, uint32_t (&r)[32]) {
  const uint8_t *src = rows + lane * 128;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = *(const uint4 *)(src + (((2 * i + h) ^ (lane & 7)) << 4));
#pragma unroll
  for (int i = 0; i < 4; i++) {
    i8_to_f16(v[i].x, r[8 * i], r[8 * i + 1]);
    i8_to_f16(v[i].y, r[8 * i + 2], r[8 * i + 3]);
    i8_to_f16(v[i].z, r[8 * i + 4], r[8 * i + 5]);
    i8_to_f16(v[i].w, r[8 * i + 6], r[8 * i + 7]);
  }
}

// Groups of eight token rows of sub-block h, kI8Set groups apart: N 16-byte chunks a lane of the
// raw rows, and the same as fp16 in shared memory.
template <int N>
__device__ __forceinline__ void i8_load_groups(const uint8_t *raw, int h, int lane, uint4 (&v)[N]) {
  const int r = lane >> 2, i = lane & 3;
  const uint8_t *src = raw + r * 128 + (((2 * i + h) ^ r) << 4);
#pragma unroll
  for (int g = 0; g < N; g++) v[g] = *(const uint4 *)(src + g * kI8Set * 1024);
}
template <int N>
__device__ __forceinline__ void i8_store_groups(uint8_t *conv, int lane, const uint4 (&v)[N]) {
  const int r = lane >> 2, i = lane & 3;
  uint8_t *d0 = conv + r * 128 + (((2 * i) ^ r) << 4), *d1 = conv + r * 128 + (((2 * i + 1) ^ r) << 4);
#pragma unroll
  for (int g = 0; g < N; g++) {
    uint4 a, b;
    i8_to_f16(v[g].x, a.x, a.y);
    i8_to_f16(v[g].y, a.z, a.w);
    i8_to_f16(v[g].z, b.x, b.y);
    i8_to_f16(v[g].w, b.z, b.w);
    *(uint4 *)(d0 + g * kI8Set * 1024) = a;
    *(uint4 *)(d1 + g * kI8Set * 1024) = b;
  }
}

template <typename TO, bool GATED, int MODE>
__global__ void __launch_bounds__(kI8Threads, 1)
    linear_i8_kernel(const __grid_constant__ CUtensorMap xmap,
                     const __grid_constant__ CUtensorMap wmap, const I8Args a) {
  constexpr bool PAIR = MODE == kPair, SPLIT = MODE == kSplit;
  extern __shared__ uint8_t smraw[];
  uint8_t *ring = tc::align_smem_1024(smraw);
  const int xrows = PAIR ? a.BN / 2 : a.BN;  // token rows in this CTA's stages
  const int stage_bytes = (kLinM + xrows) * 128;  // of a raw stage
  uint8_t *conv = ring + a.stages * stage_bytes;
  I8Bars *b = (I8Bars *)(ring + a.ring + a.exchange);
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
      tc::mbar_init(&b->raw_full[0][s], 1);
      tc::mbar_init(&b->raw_full[1][s], 1);
      tc::mbar_init(&b->empty[s], kI8Set);
    }
    for (int s = 0; s < kI8Slots; s++) {
      tc::mbar_init(&b->conv_full[s], PAIR ? 2 * kI8Set : kI8Set);
      tc::mbar_init(&b->conv_empty[s], 1);
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
  // tensor memory before the trigger, as in linear.cu
  if (warp == 0) lin_tmem_alloc<PAIR ? kPair : kOne>(&b->tmem);
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
  const int blocks = 2 * (kb1 - kb0);  // fp16 sub-blocks
  const int chunk = lin_exact<TO> ? kI8Exact : blocks;  // of them summed in tensor memory

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------- producer: raw stages of this CTA
      bool ok = true;
      uint32_t armed = 0, last_ph = 0;
      I8Place p;
      for (int tile = cta; tile < total && ok; tile += ctas) {
        const LinTile t = lin_tile(a, b, tile);
        const int ft = PAIR ? 2 * t.ft + rank : t.ft;
        // the pair's MMAs take the first half of the columns from the leader
        const int row = t.r0 + (PAIR ? (int)rank * (round16(t.n) / 2) : 0);
        for (int kb = kb0; kb < kb1; kb++) {
          if (!tc::mbar_wait(&b->empty[p.s], p.lap ^ 1, abort, kLinWaitNs)) { ok = false; break; }
          uint8_t *st = ring + (size_t)p.s * stage_bytes;
          const int full = (int)p.lap * kLinStages + p.s;
          const uint32_t bar = tc::smem_u32(&b->raw_full[0][full]);
          tc::mbar_arrive_expect_tx(&b->raw_full[0][full], stage_bytes);
          armed |= 1u << full;
          last_ph = (last_ph & ~(1u << full)) | (p.ph << full);
          if (GATED)
            lin_load_5d<false>(st, &wmap, bar, kb * a.ke, ft * (kLinM / 32), t.e);
          else
            lin_load_3d<false>(st, &wmap, bar, kb * a.ke, ft * kLinM, t.e);
          lin_load_2d<false>(st + kLinM * 128, &xmap, bar, kb * a.ke, row);
          p.next(a.stages);
        }
      }
      b->armed = armed;
      b->phases = last_ph;
      if (!ok) lin_give_up<PAIR>(a, b, rank);
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (one elected lane)
    const bool leader = tc::elect_one();
    bool ok = true, issued = false, ready = false;  // ready: the next sub-block is there
    int s = 0, buf = 0;
    uint32_t ph = 0, bph = 0;
    uint64_t *empty = &b->conv_empty[0];
    const uint32_t ta0 = tbase + kI8A;
    const uint64_t db0 = tc::sdesc_sw128(tc::smem_u32(conv));
    for (int tile = cta; tile < total && ok && (!PAIR || rank == 0); tile += ctas) {
      const LinTile t = lin_tile(a, b, tile);
      const uint32_t idesc =
          tc::idesc_f16(0, round16(t.n)) + (PAIR ? (uint32_t)(kLinM >> 4) << 24 : 0u);  // M = 256
      for (int k0 = 0; k0 < blocks && ok; k0 += chunk) {  // an accumulator each
        int got = 1;
        if (leader) got = tc::mbar_wait(&b->acc_empty[buf], bph ^ 1, abort, kLinWaitNs);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t d = tbase + buf * kI8Acc<TO>;
        const int n = min(chunk, blocks - k0);
        for (int kb = 0; kb < n; kb++) {
          if (!__all_sync(0xffffffffu, ready)) {
            ok = __all_sync(0xffffffffu,
                            tc::mbar_wait_spin(&b->conv_full[s], ph, abort, kLinWaitNs));
            if (!ok) break;
          }
          tc::fence_after_sync();
          const uint32_t ta = ta0 + 32 * s;
          const uint64_t db = db0 + (uint64_t)(s * (uint32_t)(a.conv >> 4));
          if (++s == kI8Slots) s = 0, ph ^= 1;
          ready = tc::mbar_test_wait(&b->conv_full[s], ph);  // while the MMAs are issued
          if (leader) {
            i8_mma<PAIR>(d, ta, db, idesc, kb != 0);
#pragma unroll
            for (int kk = 1; kk < 4; kk++) i8_mma<PAIR>(d, ta + 8 * kk, db + 2 * kk, idesc, 1);
            lin_commit<PAIR>(empty);
          }
          empty = &b->conv_empty[s];
          issued = true;
        }
        __syncwarp();
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
  } else if (warp >= 2 + kLinEpi) {
    // ------------------------------------------------ converters: each set every second k-block
    const int set = (warp - 2 - kLinEpi) / kI8Set, quad = warp & 3;  // the warp's quarter of the rows
    const uint32_t ta = tbase + ((uint32_t)(32 * quad) << 16) + kI8A;
    bool ok = true;
    I8Place p;
    uint32_t turn = 0, cph = 0;
    for (int tile = cta; tile < total && ok; tile += ctas) {
      const LinTile t = lin_tile(a, b, tile);
      // token rows that the MMAs read from here
      const int groups = (PAIR ? round16(t.n) / 2 : round16(t.n)) / 8;
      for (int kb = kb0; kb < kb1; kb++, turn ^= 1) {
        if (turn == set) {
          uint64_t *const full = &b->raw_full[p.lap][p.s];
          if (!__all_sync(0xffffffffu, tc::mbar_test_wait(full, p.ph)))
            ok = __all_sync(0xffffffffu, tc::mbar_wait_spin(full, p.ph, abort, kLinWaitNs));
          if (!ok) break;
          const uint8_t *raw = ring + (size_t)p.s * stage_bytes;
          const uint8_t *wraw = raw + quad * 32 * 128, *xraw = raw + kLinM * 128 + quad * 1024;
#pragma unroll
          for (int h = 0; h < 2; h++) {  // the block's two sub-blocks
            const int c = 2 * set + h;
            uint8_t *to = conv + (size_t)c * a.conv + quad * 1024;
            const bool free = tc::mbar_test_wait(&b->conv_empty[c], cph ^ 1);
            uint32_t wv[32];
            i8_load_row(wraw, h, lane, wv);
            if (!__all_sync(0xffffffffu, free)) {
              ok = __all_sync(0xffffffffu,
                              tc::mbar_wait_spin(&b->conv_empty[c], cph ^ 1, abort, kLinWaitNs));
              if (!ok) break;
            }
            tc::fence_after_sync();
            tc::tmem_st32(ta + 32 * c, wv);
            int g = quad;
            for (; g + 2 * kI8Set < groups; g += 3 * kI8Set) {
              uint4 v[3];
              i8_load_groups<3>(xraw + (g - quad) * 1024, h, lane, v);
              i8_store_groups<3>(to + (g - quad) * 1024, lane, v);
            }
            for (; g < groups; g += kI8Set) {
              uint4 v[1];
              i8_load_groups<1>(xraw + (g - quad) * 1024, h, lane, v);
              i8_store_groups<1>(to + (g - quad) * 1024, lane, v);
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              if (h) tc::mbar_arrive(&b->empty[p.s]);
              if (PAIR) i8_arrive_in_cta(&b->conv_full[c], 0);
              else tc::mbar_arrive(&b->conv_full[c]);
            }
          }
          if (!ok) break;
          cph ^= 1;
        }
        p.next(a.stages);
      }
    }
    if (!ok && lane == 0) lin_give_up<PAIR>(a, b, rank);
  } else if (!SPLIT) {
    if (sizeof(TO) == 2 && !a.residual)
      lin_epilogue<LinOut16<H16<TO>, GATED>, PAIR, false>(a, b, tbase, cta, ctas, total, blocks,
                                                          kI8Acc<TO>, rank, warp, lane, stage, abort);
    else
      lin_epilogue<LinOut<TO, GATED>, PAIR, lin_exact<TO>, kI8Exact>(
          a, b, tbase, cta, ctas, total, blocks, kI8Acc<TO>, rank, warp, lane, stage, abort);
  }
  if (SPLIT)
    lin_join<TO, GATED, kI8Exact>(a, b, ring, stage, tbase, cta, total, blocks, rank, tid, abort);
  if (a.E && warp >= 2 && warp < 2 + kLinEpi) lin_zero_rows<TO>(a, b, tid);
  __syncwarp();
  tc::fence_before_sync();
  if (PAIR) cluster_sync(); else __syncthreads();  // nobody still uses a peer's barriers
  tc::fence_after_sync();
  if (*abort) {  // the same for all threads: every role has left
    lin_drain<PAIR, true>(b, b->raw_full[0], 2 * kLinStages, rank, warp, lane);
    tc::fence_before_sync();
    if (PAIR) cluster_sync(); else __syncthreads();
    tc::fence_after_sync();
  }
  if (warp == 0) lin_tmem_free<PAIR ? kPair : kOne>(tbase);
}

template <typename TO, bool GATED, int MODE>
static size_t i8_smem(int bytes) {  // of the rings and the exchange
  const int more = 1024 + (int)sizeof(I8Bars) + (MODE == kSplit ? 0 : kLinStage);
  set_dyn_smem((const void *)linear_i8_kernel<TO, GATED, MODE>, kLinRing + more);
  return bytes + more;
}

static int i8_clusters(int split) {
  static DeviceAnswers known;
  int dev = 0;
  cudaGetDevice(&dev);
  return known.get(dev, split, [&]() {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split * dev_info().sms);
    cfg.blockDim = dim3(kI8Threads);
    cfg.dynamicSmemBytes = i8_smem<float, false, kSplit>(kLinRing);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)split, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, linear_i8_kernel<float, false, kSplit>, &cfg) !=
        cudaSuccess) {
      cudaGetLastError();  // not an error of the call
      n = 0;
    }
    return n;
  });
}

// the plans of the last sizes seen by this thread (the estimate costs about a launch)
static I8Plan i8_plan(int R, int N, int E, int KB, bool gated, bool exact) {
  struct Entry {
    int R, N, E, KB, form, dev;
    I8Plan plan;
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
  const int clusters[3] = {i8_clusters(2), i8_clusters(4), i8_clusters(8)};
  const I8Plan plan = i8_make_plan(R, N, E, KB, gated, exact, dev_info().sms, clusters);
  if (plan.sure) e = Entry{R, N, E, KB, form, dev, plan};
  return plan;
}

template <typename TO, bool GATED, int MODE>
static int launch_i8(const CUtensorMap &xm, const CUtensorMap &wm, const I8Args &a, long tiles,
                     cudaStream_t st) {
  auto *k = linear_i8_kernel<TO, GATED, MODE>;
  const size_t smem = i8_smem<TO, GATED, MODE>(a.ring + a.exchange);
  const int per = MODE == kPair ? 2 : MODE == kSplit ? a.split : 1;  // CTAs per tile
  const long most = MODE == kSplit ? tiles : std::min(tiles, (long)dev_info().sms / per);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(most * per));
  cfg.blockDim = dim3(kI8Threads);
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
static int launch_i8_m(const CUtensorMap &xm, const CUtensorMap &wm, const I8Args &a,
                       const I8Plan &p, cudaStream_t st) {
  if constexpr (!lin_exact<TO>)
    if (p.mode == kPair) return launch_i8<TO, GATED, kPair>(xm, wm, a, p.tiles, st);
  return p.mode == kSplit ? launch_i8<TO, GATED, kSplit>(xm, wm, a, p.tiles, st)
                          : launch_i8<TO, GATED, kOne>(xm, wm, a, p.tiles, st);
}

template <typename TO>
static int launch_i8_t(const CUtensorMap &xm, const CUtensorMap &wm, const I8Args &a,
                       const I8Plan &p, cudaStream_t st) {
  return a.act == MOE_ACT_SWIGLU ? launch_i8_m<TO, true>(xm, wm, a, p, st)
                                 : launch_i8_m<TO, false>(xm, wm, a, p, st);
}

// Whether the form for few rows (linear_i8_few.cu) takes the product.  Its MMAs keep up with memory
// for 8 token rows a tile, and take twice as long for 16.  That was measured where there are about as
// many tiles as SMs, 2048 features and more; fewer features are bound by what one SM reads of K
// (one row: 256 to 1024 features of K = 6144 4.9 to 5.0 us, of 14336 7.5 to 7.7).  With several experts:
// five rows an expert in the mean.
static bool i8_few(int R, int rows, int K, int E) {
  if (E <= 1) return R <= 8 || (R <= 16 && (long)rows * K <= 24 << 20);
  return R <= 5.0 * E * (1.0 - std::pow(1.0 - 1.0 / E, R));
}

int linear_i8(LinArgs base, int K, const void *x, long ldx, const void *w, moe_dtype out_dtype,
              cudaStream_t st) {
  if (K < 131072 && i8_few(base.R, (base.act == MOE_ACT_SWIGLU ? 2 : 1) * base.N, K, base.E))
    return linear_i8_few(base, K, x, ldx, w, out_dtype, st);
  I8Args a{};
  (LinArgs &)a = base;
  const bool gated = a.act == MOE_ACT_SWIGLU;
  const I8Plan plan = i8_plan(a.R, a.N, a.E, a.KB, gated, out_dtype == MOE_DT_F32);
  const int xrows = plan.mode == kPair ? plan.BN / 2 : plan.BN;
  const int ftw = (plan.mode == kPair ? 2 * kLinM : kLinM) / (gated ? 2 : 1);
  a.BN = plan.BN;
  a.split = plan.split;
  const int stage = (kLinM + xrows) * 128;
  if (plan.mode == kSplit) a.exchange = i8_exchange(a.BN, a.split);
  a.conv = xrows * 128;
  a.stages = i8_stages(xrows, a.exchange);
  if (a.stages < 2) return MOE_ERR_UNSUPPORTED;  // (no plan is like that)
  // kSplit: the output is staged there
  a.ring = std::max(a.stages * stage + kI8Slots * a.conv, kLinStage);
  a.FT = (a.N + ftw - 1) / ftw;
  // as many token rows as weight rows at one time, when every SM works on a tile
  const double at_once = plan.mode == kPair ? dev_info().sms / 2 : dev_info().sms;
  a.group = std::max(1, (int)std::lround(std::sqrt(at_once * ftw * (gated ? 2 : 1) / a.BN)));
  CUtensorMap xm, wm;
  if (!lin_maps(a, K, x, ldx, w, 1, xrows, xm, wm)) return MOE_ERR_CUDA;
  return out_dtype == MOE_DT_F32    ? launch_i8_t<float>(xm, wm, a, plan, st)
         : out_dtype == MOE_DT_BF16 ? launch_i8_t<__nv_bfloat16>(xm, wm, a, plan, st)
                                    : launch_i8_t<__half>(xm, wm, a, plan, st);
}

}  // namespace moe
