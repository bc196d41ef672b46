// tokens.cu -- tokens sorted by expert and back, with weights applied, and the gradients.
//
// The routed rows of T tokens with k slots each are ordered by (expert, slot):
//   sort      slot_pos[t][j] = position of slot (t, j), perm = its inverse, offsets[E+1]
//   dispatch  xs[slot_pos[t][j]] = x[t]
//   combine   out[t] = add[t] + sum_j w[t][j] y[slot_pos[t][j]]
//   gradients dy[slot_pos[t][j]] = w[t][j] dout[t],  dw[t][j] = <dout[t], y[slot_pos[t][j]]>,
//             dx[t] = sum_j dxs[slot_pos[t][j]]
// Everything but the sort is bound by memory traffic; all of it is organised by token, so a
// token's row is read (or written) once for its k slots, and every sum has one fixed order:
// no atomics touch a result.
#include <cooperative_groups.h>

#include <algorithm>

#include "dev.cuh"
#include "elem.cuh"
#include "host.cuh"
#include "moe_internal.cuh"

namespace cg = cooperative_groups;

namespace moe {

// ------------------------------------------------------------------------------- sort
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxE = 256;

// A stable counting sort in one launch: one CTA, or a cluster of eight or sixteen for long id
// arrays.  Each warp owns a contiguous run of slots and counts it into its own row of `hist`; the rows
// are scanned over the warps, the CTA totals over the cluster (distributed shared memory), the
// expert totals over the experts; then each warp walks its run again, 32 slots at a time, and
// gives a slot the position base + expert's slots so far + equal ids in lower lanes.  The lanes
// of an id come from a mask in shared memory that every lane sets its bit in (the order of those
// atomics does not matter); match_any finds them too, but slower: 65,536 slots of 256 experts
// 21 us against 10 on eight CTAs.
struct SortShared {
  int hist[kSortWarps][kSortMaxE];       // slots of the warp's run, then positions handed out
  uint32_t mask[kSortWarps][kSortMaxE];  // the lanes of each id among the warp's 32 slots
  int total[kSortMaxE];                  // this CTA's slots per expert
  int start[kSortMaxE + 1];              // first position of each expert
  int base[kSortMaxE];                   // first position of each expert in this CTA
  int warps[8];                          // slots of each 32 experts
};

constexpr int kSortBatch = 8;  // steps of 32 slots loaded at a time

__device__ __forceinline__ void load_ids(const int32_t *ids, long i0, long hi, int E, int lane,
                                         int (&e)[kSortBatch]) {
#pragma unroll
  for (int u = 0; u < kSortBatch; u++) {
    const long i = i0 + u * 32 + lane;
    e[u] = i < hi ? ids[i] : -1;
    if (e[u] >= E) e[u] = -1;
  }
}

__global__ void __launch_bounds__(kSortThreads) sort_tokens_kernel(int n, int E, const int32_t *ids,
                                                                   int32_t *offsets, int32_t *perm,
                                                                   int32_t *slot_pos) {
  extern __shared__ uint8_t sort_raw[];
  SortShared &S = *(SortShared *)sort_raw;
  cg::cluster_group cl = cg::this_cluster();
  const int ncta = cl.num_blocks(), rank = cl.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = blockDim.x >> 5;
  const unsigned below = (1u << lane) - 1u;
  pdl_wait();
  pdl_trigger();
  const int runs = ncta * nw;
  const int len = ((n + runs - 1) / runs + 31) / 32 * 32;  // slots per warp
  const long lo = min((long)n, (long)(rank * nw + warp) * len);
  const long hi = min((long)n, lo + len);
  int *hist = S.hist[warp];
  uint32_t *mask = S.mask[warp];
  int e[kSortBatch];
  load_ids(ids, lo, hi, E, lane, e);
  for (int i = lane; i < E; i += 32) hist[i] = 0, mask[i] = 0u;
  __syncwarp();
  for (long i0 = lo; i0 < hi; i0 += 32 * kSortBatch) {
    if (i0 != lo) load_ids(ids, i0, hi, E, lane, e);
#pragma unroll
    for (int u = 0; u < kSortBatch; u++)
      if (e[u] >= 0) atomicAdd(&hist[e[u]], 1);
  }
  __syncthreads();
  for (int x = tid; x < E; x += blockDim.x) {  // exclusive scan over the warps, eight at a time
    int s = 0;
    for (int w0 = 0; w0 < nw; w0 += 8) {
      int c[8];
#pragma unroll
      for (int w = 0; w < 8; w++) c[w] = S.hist[w0 + w][x];
#pragma unroll
      for (int w = 0; w < 8; w++) {
        S.hist[w0 + w][x] = s;
        s += c[w];
      }
    }
    S.total[x] = s;
  }
  if (ncta > 1) cl.sync(); else __syncthreads();
  // exclusive scan over the experts (at most 256, a thread each): within warps, then over them
  int all = 0, before = 0;
  if (tid < E) {
    for (int c = 0; c < ncta; c++) {
      const int v = ncta > 1 ? cl.map_shared_rank(S.total, c)[tid] : S.total[tid];
      if (c < rank) before += v;
      all += v;
    }
  }
  int incl = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31 && warp < 8) S.warps[warp] = incl;
  __syncthreads();
  if (tid < kSortMaxE) {
    int add = 0;
#pragma unroll
    for (int q = 0; q < 8; q++) add += q < warp ? S.warps[q] : 0;
    if (tid < E) {
      S.start[tid] = add + incl - all;
      S.base[tid] = add + incl - all + before;
    }
    if (tid == E - 1) S.start[E] = add + incl;
  }
  __syncthreads();
  const bool once = hi - lo <= 32 * kSortBatch;  // the run's ids are still in registers
  for (long i0 = lo; i0 < hi; i0 += 32 * kSortBatch) {
    if (!once) load_ids(ids, i0, hi, E, lane, e);
#pragma unroll
    for (int u = 0; u < kSortBatch; u++) {
      const long i = i0 + u * 32 + lane;
      if (i0 + u * 32 >= hi) break;
      if (e[u] >= 0) atomicOr(&mask[e[u]], 1u << lane);
      __syncwarp();
      int pos = -1;
      uint32_t m = 0;
      if (e[u] >= 0) {
        m = mask[e[u]];
        pos = S.base[e[u]] + hist[e[u]] + __popc(m & below);
      }
      __syncwarp();
      if (e[u] >= 0 && (m & below) == 0) {  // the lowest lane of the id moves its count on
        hist[e[u]] += __popc(m);
        mask[e[u]] = 0u;
      }
      __syncwarp();
      if (i < hi) slot_pos[i] = pos;
      if (pos >= 0) perm[pos] = (int32_t)i;
    }
  }
  // dropped slots leave a tail without rows
  for (long p = (long)S.start[E] + rank * blockDim.x + tid; p < n; p += (long)ncta * blockDim.x)
    perm[p] = -1;
  if (rank == 0)
    for (int x = tid; x <= E; x += blockDim.x) offsets[x] = S.start[x];
  if (ncta > 1) cl.sync();  // no CTA leaves while another may still read its totals
}

// ----------------------------------------------------------------------- row movement
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;

constexpr int kMoveThreads = 128;
constexpr int kMoveWarps = kMoveThreads / 32;

// Row copies move `U` units of W bytes a lane per step, all loads before the stores: a token's row
// is read once for its k slots.  8192 tokens x 8 of 6144 bf16: 138 us, 97% of the copy rate.
template <typename W>
__global__ void __launch_bounds__(kMoveThreads)
    dispatch_kernel(int T, int k, int E, long units, long ldx, const W *x, const int32_t *slot_pos,
                    const int32_t *offsets, W *xs, int pieces, int SC, const float *sc, long ldsc,
                    float *scs) {
  constexpr int U = 8;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long n = (long)T * k;
  const long nwarps = (long)gridDim.x * kMoveWarps;
  const long gw = (long)blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
  for (long item = gw; item < (long)T * pieces; item += nwarps) {
    const long t = item / pieces;
    const int piece = (int)(item - t * pieces);
    const int my = lane < k ? slot_pos[t * k + lane] : -1;
    const W *src = x + t * ldx;
    for (long u0 = (long)piece * 32 * U; u0 < units; u0 += (long)pieces * 32 * U) {
      W v[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const long i = u0 + u * 32 + lane;
        if (i < units) v[u] = src[i];
      }
      for (int j = 0; j < k; j++) {
        const int p = __shfl_sync(0xffffffffu, my, j);
        if (p < 0 || p >= n) continue;
        W *dst = xs + (long)p * units;
#pragma unroll
        for (int u = 0; u < U; u++) {
          const long i = u0 + u * 32 + lane;
          if (i < units) dst[i] = v[u];
        }
      }
    }
    if (piece == 0 && sc)
      for (int j = 0; j < k; j++) {
        const int p = __shfl_sync(0xffffffffu, my, j);
        if (p < 0 || p >= n) continue;
        for (int i = lane; i < SC; i += 32) scs[(long)p * SC + i] = sc[t * ldsc + i];
      }
  }
  // rows without a slot are zero
  const long live = min(n, (long)max(0, offsets[E]));
  for (long p = live + gw; p < n; p += nwarps) {
    W zero = {};
    for (long i = lane; i < units; i += 32) xs[p * units + i] = zero;
    if (sc)
      for (int i = lane; i < SC; i += 32) scs[p * SC + i] = 0.f;
  }
}

struct CombineArgs {
  const void *y, *add;
  const int32_t *slot_pos;
  const float *w;
  void *out;
  long ldadd, ldout;
  int T, k, H;
};

// A thread owns a pack of eight elements of the rows of tokens t, t + stride, ...: U slots' rows
// (and the addend) in flight at a time, the next token's slots loaded meanwhile, so that only
// the first token waits for slots before its rows; fp32 sum in slot order, one rounding.
// 8192 tokens x 8 of 6144 bf16: 151 us, 6.7 TB/s (a CTA per token and eight slots in flight:
// 184; four 169); x 2 of 4096: 45 us, 5.9 TB/s (two to four tokens or packs a thread: 48 to 61).
// Two slots of 16-bit rows are few bytes a thread: six CTAs an SM (40 registers a thread) take 45
// us where five take 49; more bytes a thread want the registers (four slots: 171 us against 151).
template <typename TY, typename TO, int A, int U>
__global__ void __launch_bounds__(kRowThreads, U <= 2 && sizeof(TY) == 2 ? 6 : 4)
    combine_rows_kernel(const CombineArgs a) {
  pdl_wait();
  pdl_trigger();
  const int i = 8 * (int)(blockIdx.x * blockDim.x + threadIdx.x);
  const int stride = gridDim.y * blockDim.y;
  int t = blockIdx.y * blockDim.y + threadIdx.y;
  if (t >= a.T || Place<TO, A>::first(i) >= a.H) return;
  const int n = a.T * a.k;
  const TY *y = (const TY *)a.y;
  int pos[U];
  float w[U];
  auto slots = [&](int token, int j0) {
#pragma unroll
    for (int j = 0; j < U; j++) {
      const bool in = token < a.T && j0 + j < a.k;
      const long s = (long)token * a.k + j0 + j;
      pos[j] = in ? a.slot_pos[s] : -1;
      w[j] = in ? a.w ? a.w[s] : 1.0f : 0.f;
    }
  };
  slots(t, 0);
  for (; t < a.T; t += stride) {
    Pack<TO> pa;
    pa.clear();
    if (a.add) pa = load_pack<TO, A>((const TO *)a.add + t * a.ldadd, i, a.H);
    float acc[8];
    for (int j0 = 0; j0 < a.k; j0 += U) {
      Pack<TY> v[U];
      float wv[U];
#pragma unroll
      for (int j = 0; j < U; j++) {
        const bool live = pos[j] >= 0 && pos[j] < n;
        wv[j] = live ? w[j] : 0.f;  // a slot without a row adds zero
        v[j].clear();
        if (live) v[j] = load_pack<TY, A>(y + (long)pos[j] * a.H, i, a.H);
      }
      if (j0 + U < a.k) slots(t, j0 + U); else slots(t + stride, 0);
      if (j0 == 0) pa.get(acc);  // waited for after the rows are on their way
#pragma unroll
      for (int j = 0; j < U; j++) {
        float f[8];
        v[j].get(f);
#pragma unroll
        for (int m = 0; m < 8; m++) acc[m] = fmaf(wv[j], f[m], acc[m]);
      }
    }
    Pack<TO> o;
    o.put(acc);
    store_pack<TO, A>((TO *)a.out + t * a.ldout, i, a.H, o);
  }
}

struct GradArgs {
  const void *dout, *y;
  const int32_t *slot_pos, *offsets;
  const float *w;
  void *dy;
  float *dw;
  long lddout;
  int T, k, E, H;
};

// A CTA per token: its dout pack stays in registers for the k slots (KC of them at a time),
// whose y rows are read for dw and whose dy rows are written.  dw is summed over lanes, then
// over warps, in a fixed order.  CTAs past the tokens write the zero rows of the tail.  4096
// tokens x 8 of 6144 bf16: 128 us, 99% of the copy rate (eight slots at a time, more registers
// and fewer warps, 7% slower).
template <typename T, int A, int KC>
__global__ void __launch_bounds__(kRowThreads) combine_grad_kernel(const GradArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float part[KC][kRowWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long n = (long)a.T * a.k;
  T *dy = (T *)a.dy;
  if ((int)blockIdx.x >= a.T) {
    const long live = min(n, (long)max(0, a.offsets[a.E]));
    Pack<T> zero;
    zero.clear();
    for (long p = live + (blockIdx.x - a.T); p < n; p += gridDim.x - a.T)
      for (int i = 8 * tid; Place<T, A>::first(i) < a.H; i += 8 * blockDim.x)
        store_pack<T, A>(dy + p * a.H, i, a.H, zero);
    return;
  }
  const long t = blockIdx.x;
  const T *dout = (const T *)a.dout + t * a.lddout;
  const T *y = (const T *)a.y;
  for (int j0 = 0; j0 < a.k; j0 += KC) {
    int pos[KC];
    float w[KC], acc[KC];
#pragma unroll
    for (int j = 0; j < KC; j++) {
      const bool in = j0 + j < a.k;
      pos[j] = in ? a.slot_pos[t * a.k + j0 + j] : -1;
      if (pos[j] >= n) pos[j] = -1;
      w[j] = in ? a.w ? a.w[t * a.k + j0 + j] : 1.0f : 0.f;
      acc[j] = 0.f;
    }
    for (int i = 8 * tid; Place<T, A>::first(i) < a.H; i += 8 * blockDim.x) {
      const Pack<T> pd = load_pack<T, A>(dout, i, a.H);
      Pack<T> py[KC];
#pragma unroll
      for (int j = 0; j < KC; j++) {
        py[j].clear();
        if (pos[j] >= 0) py[j] = load_pack<T, A>(y + (long)pos[j] * a.H, i, a.H);
      }
      float d[8];
      pd.get(d);
#pragma unroll
      for (int j = 0; j < KC; j++) {
        if (pos[j] < 0) continue;
        float f[8], g[8];
        py[j].get(f);
#pragma unroll
        for (int m = 0; m < 8; m++) {
          acc[j] = fmaf(d[m], f[m], acc[j]);
          g[m] = w[j] * d[m];
        }
        Pack<T> o;
        o.put(g);
        store_pack<T, A>(dy + (long)pos[j] * a.H, i, a.H, o);
      }
    }
    if (j0) __syncthreads();  // the last slots' sums have been read
#pragma unroll
    for (int j = 0; j < KC; j++) {
      const float s = warp_sum(acc[j]);
      if (lane == 0) part[j][warp] = s;
    }
    __syncthreads();
    if (tid < KC && j0 + tid < a.k) {
      float s = 0.f;
      for (int q = 0; q < (int)blockDim.x / 32; q++) s += part[tid][q];
      a.dw[t * a.k + j0 + tid] = s;
    }
  }
}

template <typename TY, typename TO, int A, int U>
static cudaError_t launch_combine_u(const CombineArgs &a, cudaStream_t st) {
  const int packs = (a.H + 7) / 8;
  int bx = 32;  // short rows: several tokens a CTA
  while (bx < packs && bx < kRowThreads) bx *= 2;
  const dim3 block(bx, kRowThreads / bx);
  const int gx = (packs + bx - 1) / bx, rows = (a.T + block.y - 1) / block.y;
  const int per_sm = U <= 2 ? 16 : 8;  // CTAs: enough to fill the SMs once or twice over
  const dim3 grid(gx, std::min(rows, std::max(1, per_sm * dev_info().sms / gx)));
  return launch_pdl(combine_rows_kernel<TY, TO, A, U>, grid, block, 0, st, a);
}

template <typename TY, typename TO, int A>
static cudaError_t launch_combine_v(const CombineArgs &a, cudaStream_t st) {
  return a.k <= 2 ? launch_combine_u<TY, TO, A, 2>(a, st)
                  : launch_combine_u<TY, TO, A, 4>(a, st);
}

template <typename TY, typename TO>
static cudaError_t launch_combine_rows(const CombineArgs &a, cudaStream_t st) {
  const uintptr_t p = (uintptr_t)a.y | (uintptr_t)a.add | (uintptr_t)a.out |
                      (uintptr_t)(a.ldadd * sizeof(TO)) | (uintptr_t)(a.ldout * sizeof(TO));
  const int acc = access_of(p, a.H, sizeof(TY));
  if (acc == kVec) return launch_combine_v<TY, TO, kVec>(a, st);
  // the words of a pack are the same elements only where both types have one size; of two sizes,
  // rows off 8 elements move one element at a time (16384 x 4 bf16 rows to fp32: of 2048 61 us, of
  // 2050 198; to bf16 52 and 72, of 2051 179)
  constexpr int W = sizeof(TY) == sizeof(TO) ? kWord : kAny;
  return acc == kWord ? launch_combine_v<TY, TO, W>(a, st) : launch_combine_v<TY, TO, kAny>(a, st);
}

template <typename T, int A>
static cudaError_t launch_grad(const GradArgs &a, cudaStream_t st) {
  const int packs = (a.H + 7) / 8;
  const dim3 block(std::min(kRowThreads, (packs + 31) / 32 * 32));
  const dim3 grid(a.T + std::min(a.T, 2 * dev_info().sms));
  if (a.k <= 2) return launch_pdl(combine_grad_kernel<T, A, 2>, grid, block, 0, st, a);
  return launch_pdl(combine_grad_kernel<T, A, 4>, grid, block, 0, st, a);
}

template <typename T>
static cudaError_t launch_grad_t(const GradArgs &a, cudaStream_t st) {
  const uintptr_t p = (uintptr_t)a.dout | (uintptr_t)a.y | (uintptr_t)a.dy |
                      (uintptr_t)(a.lddout * sizeof(T));
  const int acc = access_of(p, a.H, sizeof(T));
  return acc == kVec    ? launch_grad<T, kVec>(a, st)
         : acc == kWord ? launch_grad<T, kWord>(a, st)
                        : launch_grad<T, kAny>(a, st);
}

static bool float_type(int dt) {
  return dt == MOE_DT_F32 || dt == MOE_DT_BF16 || dt == MOE_DT_F16;
}
static uintptr_t type_size(int dt) {
  return dt == MOE_DT_F32 ? 4 : dt == MOE_DT_E4M3 ? 1 : 2;
}

// T and k as everywhere in the library; a row of H elements
static int check_tokens(int T, int k, int H = 1) {
  if (T < 0 || H <= 0) return MOE_ERR_INVALID_ARG;
  if (k < 1 || k > 16 || T > 65535 || H > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

template <typename W>
static cudaError_t launch_dispatch(int T, int k, int E, long row_bytes, long ldx_bytes,
                                   const void *x, const int32_t *slot_pos, const int32_t *offsets,
                                   void *xs, int SC, const float *sc, long ldsc, float *scs,
                                   cudaStream_t st) {
  const long units = row_bytes / (long)sizeof(W);
  // a warp moves a piece of 256 units of a row: the loads of eight a lane, then the stores of
  // each slot (a whole row a warp: 155 us where pieces take 147, 8192 x 8 rows of 6144 bf16)
  const int pieces = (int)std::max(1l, (units + 255) / 256);
  const long items = (long)T * pieces;
  const unsigned grid = (unsigned)std::min((items + kMoveWarps - 1) / kMoveWarps,
                                           (long)dev_info().sms * 128);
  return launch_pdl(dispatch_kernel<W>, dim3(std::max(1u, grid)), dim3(kMoveThreads), 0, st, T, k,
                    E, units, ldx_bytes / (long)sizeof(W), (const W *)x, slot_pos, offsets,
                    (W *)xs, pieces, SC, sc, ldsc, scs);
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_sort_tokens(int T, int k, int n_experts, const int32_t *ids, int32_t *offsets,
                    int32_t *perm, int32_t *slot_pos, void *stream) {
  if (int r = check_tokens(T, k)) return r;
  if (n_experts < 1 || n_experts > kSortMaxE) return MOE_ERR_UNSUPPORTED;
  if (!offsets || (T && (!ids || !perm || !slot_pos))) return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)ids | (uintptr_t)offsets | (uintptr_t)perm | (uintptr_t)slot_pos) % 4)
    return MOE_ERR_INVALID_ARG;
  const int n = T * k;
  // 65,536 slots: 10.0 us with eight CTAs, 8.4 with sixteen; 262,144: 27.9 and 17.7
  const int e = sort_launch(n, [&](int ctas) {
    const void *kernel = (const void *)sort_tokens_kernel;
    cudaError_t r = cudaSuccess;
    if (ctas == 16)
      r = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    // one CTA: a warp for every 32 slots (in eights, as the scan takes them), and the scans' threads
    cfg.blockDim = dim3(ctas > 1 ? kSortThreads
                                 : std::min(kSortThreads, std::max(256, (n + 255) / 256 * 256)));
    cfg.dynamicSmemBytes = sizeof(SortShared);
    set_dyn_smem(kernel, (int)sizeof(SortShared));
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)ctas, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (r == cudaSuccess)
      r = cudaLaunchKernelEx(&cfg, sort_tokens_kernel, n, n_experts, ids, offsets, perm, slot_pos);
    if (r != cudaSuccess) cudaGetLastError();  // not the next launch's error
    return (int)r;
  });
  return e == 0 && cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_dispatch_rows(int T, int k, int n_experts, int H, moe_dtype dtype, const void *x, long ldx,
                      const int32_t *slot_pos, const int32_t *offsets, void *xs, int n_scales,
                      const float *scale, long ldscale, float *scale_s, void *stream) {
  if (int r = check_tokens(T, k, H)) return r;
  if (!float_type(dtype) && dtype != MOE_DT_E4M3) return MOE_ERR_INVALID_ARG;
  if (n_scales < 0 || n_experts < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const uintptr_t es = type_size(dtype);
  if (!x || !xs || !slot_pos || !offsets || ldx < H) return MOE_ERR_INVALID_ARG;
  if (n_scales && (!scale || !scale_s || ldscale < n_scales)) return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)x | (uintptr_t)xs) % es || ((uintptr_t)slot_pos | (uintptr_t)offsets) % 4 ||
      ((uintptr_t)scale | (uintptr_t)scale_s) % 4)
    return MOE_ERR_INVALID_ARG;
  const long row = (long)H * es, ld = ldx * (long)es;
  const uintptr_t al = (uintptr_t)x | (uintptr_t)xs | (uintptr_t)row | (uintptr_t)ld;
  const float *sc = n_scales ? scale : nullptr;
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  // the widest unit that every row's start and length allow (16384 x 4 rows: of 2048 e4m3 26 us, of
  // 2052 29, of 2050 38, of 2051, a byte a lane, 55; of 2048 bf16 51, of 2050 52, of 2051 65)
  if (al % 16 == 0)
    e = launch_dispatch<uint4>(T, k, n_experts, row, ld, x, slot_pos, offsets, xs, n_scales, sc,
                               ldscale, scale_s, st);
  else if (al % 4 == 0)
    e = launch_dispatch<uint32_t>(T, k, n_experts, row, ld, x, slot_pos, offsets, xs, n_scales, sc,
                                  ldscale, scale_s, st);
  else if (al % 2 == 0)
    e = launch_dispatch<uint16_t>(T, k, n_experts, row, ld, x, slot_pos, offsets, xs, n_scales, sc,
                                  ldscale, scale_s, st);
  else
    e = launch_dispatch<uint8_t>(T, k, n_experts, row, ld, x, slot_pos, offsets, xs, n_scales, sc,
                                 ldscale, scale_s, st);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_combine_rows(int T, int k, int H, const void *y, moe_dtype y_dtype,
                     const int32_t *slot_pos, const float *w, const void *add, long ldadd,
                     void *out, long ldout, moe_dtype out_dtype, void *stream) {
  if (int r = check_tokens(T, k, H)) return r;
  if (!float_type(y_dtype) || !float_type(out_dtype)) return MOE_ERR_INVALID_ARG;
  if (out_dtype != y_dtype && out_dtype != MOE_DT_F32) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const uintptr_t ey = type_size(y_dtype), eo = type_size(out_dtype);
  if (!y || !slot_pos || !out || ldout < H || (add && ldadd < H)) return MOE_ERR_INVALID_ARG;
  if ((uintptr_t)y % ey || ((uintptr_t)out | (uintptr_t)add) % eo ||
      ((uintptr_t)slot_pos | (uintptr_t)w) % 4)
    return MOE_ERR_INVALID_ARG;
  const CombineArgs a{y, add, slot_pos, w, out, add ? ldadd : 0, ldout, T, k, H};
  const cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (y_dtype == MOE_DT_F32)
    e = launch_combine_rows<float, float>(a, st);
  else if (y_dtype == MOE_DT_BF16)
    e = out_dtype == MOE_DT_F32 ? launch_combine_rows<__nv_bfloat16, float>(a, st)
                                : launch_combine_rows<__nv_bfloat16, __nv_bfloat16>(a, st);
  else
    e = out_dtype == MOE_DT_F32 ? launch_combine_rows<__half, float>(a, st)
                                : launch_combine_rows<__half, __half>(a, st);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_combine_rows_grad(int T, int k, int n_experts, int H, moe_dtype dtype, const void *dout,
                          long lddout, const void *y, const int32_t *slot_pos,
                          const int32_t *offsets, const float *w, void *dy, float *dw,
                          void *stream) {
  if (int r = check_tokens(T, k, H)) return r;
  if (n_experts < 0 || !float_type(dtype)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const uintptr_t es = type_size(dtype);
  if (!dout || !y || !slot_pos || !offsets || !dy || !dw || lddout < H) return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)dout | (uintptr_t)y | (uintptr_t)dy) % es ||
      ((uintptr_t)slot_pos | (uintptr_t)offsets | (uintptr_t)w | (uintptr_t)dw) % 4)
    return MOE_ERR_INVALID_ARG;
  const GradArgs a{dout, y, slot_pos, offsets, w, dy, dw, lddout, T, k, n_experts, H};
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == MOE_DT_F32    ? launch_grad_t<float>(a, st)
                        : dtype == MOE_DT_BF16 ? launch_grad_t<__nv_bfloat16>(a, st)
                                               : launch_grad_t<__half>(a, st);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_dispatch_rows_grad(int T, int k, int H, moe_dtype dtype, const void *dxs,
                           const int32_t *slot_pos, void *dx, long lddx, moe_dtype dx_dtype,
                           void *stream) {
  return moe_combine_rows(T, k, H, dxs, dtype, slot_pos, nullptr, nullptr, 0, dx, lddx, dx_dtype,
                          stream);
}

}  // extern "C"
