// route_logits.cu -- experts chosen from a user's own router logits, and the gradient back to them.
//
//   s = softmax(l) or sigmoid(l) over the available experts of a token (l not NaN, not -inf; +inf
//       counts as the largest finite number),  c = s + bias
//   groups: the sum of a group's one or two largest c ranks it; topk_group groups are kept
//   ids = the k largest c of the kept groups, descending, ties to the lower index
//   w_j = f s_j / sum_i s_i over the chosen (norm), or f s_j
//
// One warp a token: lane i holds the V = 1, 2, 4 or 8 neighbouring experts V i .. V i + V - 1, so
// that a lower lane means a lower index and a group is a run of lanes.  Scores become integers of
// the same order whose last bits give way to the place in the lane; each lane sorts its own, and
// the k largest come out one after the other: the warp's largest by one reduction, the first lane
// that holds it gives it up.  8192 tokens of 256 experts: 6.2 us without a bias, sigmoid with one 8.4,
// with one and eight groups 10.3, of which 2.2 are a launch; bound by instructions, some 550 (no
// bias) and 850 (groups) a token.  Two forms take longer: softmax with a bias, whose near scores go
// to fp64 (23 us, 32 in eight groups; 64 experts 12), and groups that are no run of 2^n lanes, which
// one lane each walks (8192 x 160 in eight groups: sigmoid with a bias 23 us, softmax 35).
//
// What is chosen is what 64-bit scores choose.  Without a bias the logits themselves have the
// scores' order.  With one, fp32 scores are compared, and where two that follow each other lie
// nearer than their error (8192 tokens of 256 experts: some ten such pairs), the candidates are
// ranked again by scores in two floats, one candidate a lane, and where those do not tell them
// apart the token is done over in fp64.  The same for the last group kept and the first left out.
#include <cuda_fp16.h>

#include <cfloat>

#include "dev.cuh"
#include "elem.cuh"
#include "moe_internal.cuh"

namespace moe {

constexpr int kRouteWarps = 4;  // tokens a CTA
constexpr int kRouteMaxE = 256, kRouteMaxK = 16, kRouteMaxG = 32;

struct RouteArgs {
  const void *logits;
  const float *bias;
  int32_t *ids;
  float *w;
  long ld;
  int T, E, k, G, keep, best, softmax, norm;
  float f;
  int vec;          // a lane's logits (and biases) are aligned accesses
  int step, shift;  // lanes of a group, 1 << shift; 0: it is no such run of lanes
};

__device__ __forceinline__ float route_f32(float v) { return v; }
__device__ __forceinline__ float route_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float route_f32(__half v) { return __half2float(v); }

// a > b iff key(a) > key(b), for floats that are not NaN and with one zero; never 0
__device__ __forceinline__ uint32_t route_key(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);  // -0 + 0 = 0
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
constexpr uint32_t kRouteNone = 0x007FFFFFu;  // the key of -inf
__device__ __forceinline__ float route_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// V neighbouring logits of a row from `e`; experts past the last one count as unavailable
template <typename T, int V>
__device__ __forceinline__ void route_load(const T *row, int e, int E, int vec, float (&l)[V]) {
  alignas(16) T t[V];
  if (vec && e < E) {
    if constexpr (sizeof(t) % 16 == 0) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(t) / 16; i++) ((uint4 *)t)[i] = ((const uint4 *)(row + e))[i];
    } else if constexpr (sizeof(t) == 8) {
      *(uint2 *)t = *(const uint2 *)(row + e);
    } else if constexpr (sizeof(t) == 4) {
      *(uint32_t *)t = *(const uint32_t *)(row + e);
    } else {
      t[0] = row[e];
    }
#pragma unroll
    for (int v = 0; v < V; v++) l[v] = route_f32(t[v]);
  } else {
#pragma unroll
    for (int v = 0; v < V; v++) l[v] = e + v < E ? route_f32(row[e + v]) : -INFINITY;
  }
#pragma unroll
  for (int v = 0; v < V; v++) l[v] = l[v] > -INFINITY ? fminf(l[v], FLT_MAX) : -INFINITY;
}

// the score in 64 bits; top and total: softmax's largest logit and its sum
__device__ __noinline__ double route_score64(float l, int softmax, float top, double total) {
  if (!(l > -INFINITY)) return 0.0;
  return softmax ? exp((double)l - top) / total : 1.0 / (1.0 + exp(-(double)l));
}
__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// rank of this lane's group `g` among G, by the score `s` that it has in common with the other lanes
// of the group, `step` lanes each: how many groups come before it
template <typename S>
__device__ __forceinline__ int group_rank(S s, int g, int G, int step) {
  int rank = 0;
  for (int q = 0; q < G; q++) {
    const S o = __shfl_sync(0xffffffffu, s, q * step);
    rank += o > s || (o == s && q < g);
  }
  return rank;
}

// exp2 and 1 / x as the hardware has them, off by 2^-22
__device__ __forceinline__ float route_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float route_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// sums and maxima over the lanes of the slots, of which there are at most 16
__device__ __forceinline__ float slots_sum(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float slots_max(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// What the slots' scores are to each other, one a lane (0 of -inf): exp(x), or sigmoid(x), over exp(L),
// with L the largest logit (sigmoid: or 0, where that is less).  Sigmoids of logits far below 0 are
// their exponentials, and share out what no fp32 holds; rows with a deep one take this form.
__device__ __forceinline__ bool route_deep(float x) { return x > -INFINITY && x < -60.f; }
__device__ __forceinline__ float route_share(float x, int softmax) {
  const float top = fmaxf(slots_max(x), -FLT_MAX);
  if (softmax) return expf(x - top);
  return expf(fminf(x, 0.f) - fminf(top, 0.f)) / (1.f + expf(-fabsf(x)));
}

// The lane's scores with bias, unavailable ones -inf, from its logits and biases.  top, total:
// softmax's largest logit and the sum of its exponentials.
template <int V>
__device__ __forceinline__ void route_scores(const RouteArgs &a, const float (&l)[V],
                                             const float (&b)[V], float top, float total,
                                             float (&c)[V]) {
  const float inv = 1.f / total;
#pragma unroll
  for (int v = 0; v < V; v++) {
    const float s = a.softmax ? expf(l[v] - top) * inv
                              : route_rcp(1.f + route_exp2(l[v] * -1.44269504f));
    c[v] = l[v] > -INFINITY ? fmaxf(s + b[v], -INFINITY) : -INFINITY;  // (a NaN is -inf)
  }
}

// The error of a difference of two fp32 scores, beside 2^-21 of what a bias makes of them:
// exponential, sum and division; a sigmoid's slope is 1/4.
__device__ __forceinline__ float route_eps(int softmax) { return softmax ? 0x1p-18f : 0x1p-20f; }

// The largest finite |score| of all groups, from the lane's group's two best.  With a bias the scores
// round as they are large, and so do the sums of two of both signs, however small those come out; and a
// group far from the border may be off by more than the two at it.
__device__ __forceinline__ float route_largest(float m1, float m2) {
  const float x = fabsf(m1) < INFINITY ? fabsf(m1) : 0.f, y = fabsf(m2) < INFINITY ? fabsf(m2) : 0.f;
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(x, y))));
}

template <int V>
__device__ __forceinline__ void route_bias(const RouteArgs &a, int lane, float (&b)[V]) {
  if (V >= 4 && a.vec && a.bias && V * lane < a.E) {
#pragma unroll
    for (int v = 0; v < V; v += 4) *(float4 *)(b + v % V) = *(const float4 *)(a.bias + V * lane + v);
  } else {
#pragma unroll
    for (int v = 0; v < V; v++) b[v] = a.bias && V * lane + v < a.E ? a.bias[V * lane + v] : 0.f;
  }
}

// The groups kept, bit g for group g: for groups that are no runs of 2^n lanes, and for those whose
// scores lie too near to each other.  buf: one double an expert, this warp's.
template <typename T, int V>
__device__ __noinline__ uint32_t route_groups(const RouteArgs &a, const T *row, float top,
                                              float total, int lane, double *buf) {
  alignas(16) float b[V];
  float l[V], c[V];
  route_load<T, V>(row, V * lane, a.E, a.vec, l);
  route_bias<V>(a, lane, b);
  route_scores<V>(a, l, b, top, total, c);
  float *fbuf = (float *)buf;
  const int gs = a.E / a.G;
#pragma unroll
  for (int v = 0; v < V; v++)
    if (V * lane + v < a.E) fbuf[V * lane + v] = c[v];
  __syncwarp();
  float s = -INFINITY, m1 = -INFINITY, m2 = -INFINITY;  // lane g: group g
  if (lane < a.G) {
    for (int i = 0; i < gs; i++) {
      const float x = fbuf[lane * gs + i];
      m2 = fmaxf(m2, fminf(m1, x));
      m1 = fmaxf(m1, x);
    }
    // halves, so that the sum of two lowest numbers is still one
    s = a.best == 2 ? 0.5f * m1 + (m2 > -INFINITY ? 0.5f * m2 : 0.f) : m1;
  }
  int rank = group_rank(s, lane, a.G, 1);
  if (a.keep < a.G) {  // the last one kept and the first one left out
    const uint32_t in = __ballot_sync(0xffffffffu, lane < a.G && rank == a.keep - 1);
    const uint32_t out = __ballot_sync(0xffffffffu, lane < a.G && rank == a.keep);
    const float si = __shfl_sync(0xffffffffu, s, __ffs(in) - 1);
    const float so = __shfl_sync(0xffffffffu, s, __ffs(out) - 1);
    const float big = route_largest(m1, a.best == 2 ? m2 : 0.f);
    if (so > -INFINITY && si - so <= 2.f * route_eps(a.softmax) + 0x1p-21f * big) {
      double total64 = 1.0;
      if (a.softmax) {
        total64 = 0.0;
        for (int v = 0; v < V; v++) total64 += route_score64(l[v], 1, top, 1.0);
        total64 = warp_sum64(total64);
      }
      __syncwarp();
      for (int v = 0; v < V; v++)
        if (V * lane + v < a.E)
          buf[V * lane + v] = c[v] > -INFINITY
                                  ? route_score64(l[v], a.softmax, top, total64) + (double)b[v]
                                  : -INFINITY;
      __syncwarp();
      double s64 = -INFINITY;
      if (lane < a.G) {
        double m1 = -INFINITY, m2 = -INFINITY;
        for (int i = 0; i < gs; i++) {
          const double x = buf[lane * gs + i];
          m2 = fmax(m2, fmin(m1, x));
          m1 = fmax(m1, x);
        }
        s64 = a.best == 2 && m2 > -INFINITY ? m1 + m2 : m1;
      }
      rank = group_rank(s64, lane, a.G, 1);
    }
  }
  __syncwarp();
  return __ballot_sync(0xffffffffu, lane < a.G && rank < a.keep && s > -INFINITY);
}

// All scores in 64 bits, ranked in full: for rows where more candidates than a warp has lanes lie
// too near to each other.  Lane j returns the expert of slot j.
template <int V>
__device__ __noinline__ int route_all64(const RouteArgs &a, const float (&l)[V],
                                        const float (&b)[V], const uint32_t (&key)[V], float top,
                                        int lane) {
  double total = 1.0, c[V];
  if (a.softmax) {
    total = 0.0;
    for (int v = 0; v < V; v++) total += route_score64(l[v], 1, top, 1.0);
    total = warp_sum64(total);
  }
  uint32_t left = 0;
#pragma unroll
  for (int v = 0; v < V; v++) {
    c[v] = route_score64(l[v], a.softmax, top, total) + (double)b[v];
    if (key[v]) left |= 1u << v;
  }
  int id = -1;
  for (int j = 0; j < a.k; j++) {
    double m = 0.0;
    int at = kRouteMaxE;  // none
#pragma unroll
    for (int v = 0; v < V; v++)
      if (((left >> v) & 1) && (at == kRouteMaxE || c[v] > m)) m = c[v], at = V * lane + v;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double m2 = __shfl_xor_sync(0xffffffffu, m, o);
      const int at2 = __shfl_xor_sync(0xffffffffu, at, o);
      if (at2 < kRouteMaxE && (at == kRouteMaxE || m2 > m || (m2 == m && at2 < at)))
        m = m2, at = at2;
    }
    if (at == kRouteMaxE) break;  // the same for all lanes
    if (at / V == lane) left &= ~(1u << (at % V));
    if (lane == j) id = at;
  }
  return id;
}

// The choice of a token whose scores lie too near to each other for the short way.  kept: bit g for
// group g.  Lane j returns the expert of slot j.
template <typename T, int V>
__device__ __noinline__ int route_near(const RouteArgs &a, const T *row, uint32_t kept, float top,
                                       float total, int lane) {
  alignas(16) float b[V];
  float l[V], c[V];
  route_load<T, V>(row, V * lane, a.E, a.vec, l);
  route_bias<V>(a, lane, b);
  if (a.bias) route_scores<V>(a, l, b, top, total, c);
  uint32_t key[V];  // 0: not to be had
  const int gs = a.E / a.G;
#pragma unroll
  for (int v = 0; v < V; v++) {
    const int e = V * lane + v;
    const bool in = e < a.E && l[v] > -INFINITY && (!a.bias || c[v] > -INFINITY) &&
                    (a.G == 1 || ((kept >> (e / gs)) & 1));
    key[v] = in ? route_key(a.bias ? c[v] : l[v]) : 0u;
  }
  const float eps = route_eps(a.softmax);
  // the k largest, one after the other; with a bias, on through those that lie too near to the
  // last one (`near`: two different ones do; `all`: more of them than this finds)
  int id = -1, n = 0, near = 0, all = 0;
  {
    uint32_t left[V], last = 0;
    int prev = 0, skipped = 0;
#pragma unroll
    for (int v = 0; v < V; v++) left[v] = key[v];
    while (true) {
      uint32_t m = left[0];
#pragma unroll
      for (int v = 1; v < V; v++) m = max(m, left[v]);
      const uint32_t best = __reduce_max_sync(0xffffffffu, m);
      if (best == 0) break;
      const int from = __ffs(__ballot_sync(0xffffffffu, m == best)) - 1;
      int at = 0;
#pragma unroll
      for (int v = V - 1; v >= 0; v--)
        if (left[v] == best) at = v;
      const int e = V * from + __shfl_sync(0xffffffffu, at, from);
      const float x = route_value(last), y = route_value(best);
      if (a.bias && n > 0 && x - y <= eps + 0x1p-21f * fabsf(x)) {
        if (n >= a.k && !near) {
          // Equal logits with equal biases stay behind the one that was found first, and without a
          // different one near it that one stays where it is.  (With one it may move up past the last
          // slot, and others with it: they are ranked too.)
          const float lp = fminf(route_f32(row[prev]), FLT_MAX), bp = a.bias[prev];
          bool same = best == last;
#pragma unroll
          for (int v = 0; v < V; v++)
            if (left[v] == best && !(l[v] == lp && b[v] == bp)) same = false;
          if (__all_sync(0xffffffffu, same)) {
#pragma unroll
            for (int v = 0; v < V; v++)
              if (left[v] == best) left[v] = 0u;
            skipped = 1;
            continue;
          }
        }
        // near, unless logit and bias are the same ones
        if (!(route_f32(row[prev]) == route_f32(row[e]) && a.bias[prev] == a.bias[e])) near = 1;
        if (n >= 32 || (near && skipped)) {
          all = 1;
          break;
        }
      } else if (n >= a.k) {
        break;
      }
      if (lane == n) id = e;
      n++;
      last = best;
      prev = e;
      if (lane == from) {
#pragma unroll
        for (int v = 0; v < V; v++)
          if (v == at) left[v] = 0u;
      }
    }
  }
  if (all) return route_all64<V>(a, l, b, key, top, lane);
  if (!near) return lane < a.k ? id : -1;
  double total64 = 1.0;
  if (a.softmax) {
    total64 = 0.0;
    for (int v = 0; v < V; v++) total64 += route_score64(l[v], 1, top, 1.0);
    total64 = warp_sum64(total64);
  }
  double x = -INFINITY;
  if (lane < n)
    x = route_score64(fminf(route_f32(row[id]), FLT_MAX), a.softmax, top, total64) +
        (double)a.bias[id];
  int rank = 0, got = -1;
  for (int q = 0; q < n; q++) {
    const double o = __shfl_sync(0xffffffffu, x, q);
    const int oid = __shfl_sync(0xffffffffu, id, q);
    rank += o > x || (o == x && oid < id);
  }
  for (int q = 0; q < n; q++) {
    const int r = __shfl_sync(0xffffffffu, rank, q), oid = __shfl_sync(0xffffffffu, id, q);
    if (r == lane) got = oid;
  }
  return lane < a.k ? got : -1;
}

// ------------------------------------------------------------------ scores in two floats
// A number as the sum of two floats, some 46 bits (sums and products without error after Knuth and
// Dekker): fp64 would tell near scores apart too, but takes over 10,000 cycles for one on this chip.
struct Two {
  float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fadd_rn(s, -a);
  return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t))};
}
__device__ __forceinline__ Two two_fast(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fadd_rn(b, -__fadd_rn(s, -a))};
}
__device__ __forceinline__ Two two_mul(Two a, Two b) {
  const float p = __fmul_rn(a.h, b.h);
  float e = __fmaf_rn(a.h, b.h, -p);
  e = __fmaf_rn(a.h, b.l, e);
  return two_fast(p, __fmaf_rn(a.l, b.h, e));
}
__device__ __forceinline__ Two two_add(Two a, Two b) {
  const Two s = two_sum(a.h, b.h);
  return two_fast(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Two two_of(double v) {  // of a constant
  return {(float)v, (float)(v - (double)(float)v)};
}

// sigmoid(l) + b, off by at most 2^-38 + 2^-46 |b|, or (softmax, without a bias) exp(l - top), by
// 2^-38 of it where l lies within kTwoDepth of top, and else that of the depth.  exp(x) = 2^n exp(r) with
// |r| <= 0.35, whose Taylor series is summed in fp32 from the fifth power on (which is below 2^-14, so
// that its rounding is below 2^-38) and in two floats before.
constexpr float kTwoDepth = 80.f;
__device__ __noinline__ Two route_two(float l, float b, int softmax, float top) {
  constexpr double kLn2 = 0.693147180559945309417;
  constexpr float kL1 = (float)((int)(kLn2 * 32768.0)) / 32768.0f;  // times n: exact
  constexpr float kL2 = (float)(kLn2 - kL1), kL3 = (float)(kLn2 - kL1 - kL2);
  const Two x = !softmax               ? Two{-fminf(fabsf(l), kTwoDepth), 0.f}
                : l - top < -kTwoDepth ? Two{-kTwoDepth, 0.f}
                                       : two_sum(l, -top);
  const float n = rintf(x.h * 1.44269504f);
  const float t = __fmaf_rn(-n, kL1, x.h);  // exact
  const float p = __fmul_rn(n, kL2), pe = __fmaf_rn(n, kL2, -p);
  const Two u = two_sum(t, -p);
  const Two r = two_fast(u.h, __fadd_rn(u.l, __fadd_rn(x.l, -__fmaf_rn(n, kL3, pe))));
  float q = 2.7557319e-7f;  // 1 / 10!
  q = fmaf(q, r.h, 2.7557319e-6f);
  q = fmaf(q, r.h, 2.4801587e-5f);
  q = fmaf(q, r.h, 1.9841270e-4f);
  q = fmaf(q, r.h, 1.3888889e-3f);
  q = fmaf(q, r.h, 8.3333333e-3f);  // 1 / 5!
  Two e = two_mul(Two{q, 0.f}, r);
  e = two_add(e, two_of(1.0 / 24));
  e = two_add(two_mul(e, r), two_of(1.0 / 6));
  e = two_add(two_mul(e, r), Two{0.5f, 0.f});
  e = two_add(two_mul(e, r), Two{1.f, 0.f});
  e = two_add(two_mul(e, r), Two{1.f, 0.f});
  const float scale = __uint_as_float((uint32_t)(127 + (int)n) << 23);  // 2^n, n >= -116
  e.h *= scale;
  e.l *= scale;
  if (softmax) return e;
  // 1 / (1 + e), or e / (1 + e): a quotient, and what it leaves
  const Two d = two_add(Two{1.f, 0.f}, e), num = l >= 0.f ? Two{1.f, 0.f} : e;
  const float inv = route_rcp(d.h), s0 = num.h * inv;
  const Two back = two_mul(d, Two{s0, 0.f});
  const float rest = __fadd_rn(__fadd_rn(num.h, -back.h), __fadd_rn(num.l, -back.l));
  return two_add(two_fast(s0, rest * inv), Two{b, 0.f});
}

__device__ __forceinline__ bool two_less(Two a, Two b) { return a.h < b.h || (a.h == b.h && a.l < b.l); }

// The rank of the lane's group where the last one kept (score si) and the first one left out (so)
// lie within `tol`: those groups' scores in two floats, from the experts that may be among their
// two best, one a lane.  big: the largest score that a sum is made of, 0 without a bias.  near: that
// does not tell them apart either.  mem: 96 words of this warp.
template <int V>
__device__ __noinline__ int route_groups_two(const RouteArgs &a, const float (&l)[V],
                                             const float (&b)[V], const float (&c)[V], float top,
                                             float s, float m1, float m2, float si, float so,
                                             float tol, float big, int rank, int lane, float *mem,
                                             bool &near) {
  const bool close = s >= so - tol && s <= si + tol;
  const float least = (a.best == 2 && m2 > -INFINITY ? m2 : m1) - 2.f * tol;
  const int g = lane >> a.shift;
  int n = 0;
#pragma unroll
  for (int v = 0; v < V; v++) {
    const bool may = close && c[v] > -INFINITY && c[v] >= least;
    const uint32_t all = __ballot_sync(0xffffffffu, may);
    const int at = n + __popc(all & ((1u << lane) - 1));
    if (may && at < 32) mem[at] = l[v], mem[32 + at] = b[v], mem[64 + at] = (float)g;
    n += __popc(all);
  }
  near = n > 32;
  if (near) return rank;
  __syncwarp();
  const bool have = lane < n;
  // a softmax's scores below the depth would all count as one size, and their number decide
  near = a.softmax && __any_sync(0xffffffffu, have && mem[lane] - top < -kTwoDepth);
  if (near) return rank;
  const Two x = route_two(have ? mem[lane] : top, have ? mem[32 + lane] : 0.f, a.softmax, top);
  const int of = have ? (int)mem[64 + lane] : -1;
  __syncwarp();
  Two t1{-INFINITY, 0.f}, t2 = t1;  // the two best of the lane's group
  for (int q = 0; q < n; q++) {
    const Two o{__shfl_sync(0xffffffffu, x.h, q), __shfl_sync(0xffffffffu, x.l, q)};
    const bool mine = __shfl_sync(0xffffffffu, of, q) == g;
    if (mine && two_less(t1, o)) t2 = t1, t1 = o;
    else if (mine && two_less(t2, o)) t2 = o;
  }
  const Two sum = a.best == 2 && t2.h > -INFINITY ? two_add(t1, t2) : t1;
  int r = 0;
  for (int q = 0; q < a.G; q++) {
    const float os = __shfl_sync(0xffffffffu, s, q * a.step);
    const float oh = __shfl_sync(0xffffffffu, sum.h, q * a.step);
    const float ol = __shfl_sync(0xffffffffu, sum.l, q * a.step);
    const bool both = close && os >= so - tol && os <= si + tol;
    if (both) {
      const float d = (oh - sum.h) + (ol - sum.l);
      r += d > 0.f;
      near |= q != g && !(fabsf(d) > (a.softmax ? 0.f : 0x1p-35f) + 0x1p-35f * fabsf(sum.h) +
                                        0x1p-42f * big);
    } else {
      r += os > s || (os == s && q < g);
    }
  }
  near = __any_sync(0xffffffffu, near);
  return near ? rank : r;
}

// v[0] the largest: networks of 0, 1, 5 and 19 comparisons
template <int V>
__device__ __forceinline__ void route_sort(uint32_t (&v)[V]) {
  constexpr int n8[19][2] = {{0, 2}, {1, 3}, {4, 6}, {5, 7}, {0, 4}, {1, 5}, {2, 6},
                             {3, 7}, {0, 1}, {2, 3}, {4, 5}, {6, 7}, {2, 4}, {3, 5},
                             {1, 4}, {3, 6}, {1, 2}, {3, 4}, {5, 6}};
  constexpr int n4[5][2] = {{0, 2}, {1, 3}, {0, 1}, {2, 3}, {1, 2}};
  auto swap = [&](int i, int j) {
    const uint32_t x = v[i], y = v[j];
    v[i] = max(x, y);
    v[j] = min(x, y);
  };
  if constexpr (V == 8) {
#pragma unroll
    for (int q = 0; q < 19; q++) swap(n8[q][0], n8[q][1]);
  } else if constexpr (V == 4) {
#pragma unroll
    for (int q = 0; q < 5; q++) swap(n4[q][0], n4[q][1]);
  } else if constexpr (V == 2) {
    swap(0, 1);
  }
}

// BIAS: the choice goes by scores with a bias, else by the logits.  (The arguments stay in constant
// memory: calls take their address, for which every thread otherwise copies them to its stack.)
template <typename T, int V, bool BIAS>
__global__ void __launch_bounds__(32 * kRouteWarps, 8)
    route_logits_kernel(const __grid_constant__ RouteArgs a) {
  __shared__ double buf[kRouteWarps][kRouteMaxE];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kRouteWarps + warp;
  if (t >= a.T) return;
  const T *row = (const T *)a.logits + (size_t)t * a.ld;
  alignas(16) float b[V];
  float l[V], c[V];
  route_load<T, V>(row, V * lane, a.E, a.vec, l);
  if (BIAS) route_bias<V>(a, lane, b);
  else
#pragma unroll
    for (int v = 0; v < V; v++) b[v] = 0.f;
  float top = -INFINITY, total = 1.f;
  if (a.softmax && (BIAS || a.G > 1 || !a.norm)) {
#pragma unroll
    for (int v = 0; v < V; v++) top = fmaxf(top, l[v]);
    top = warp_max(top);
    total = 0.f;
#pragma unroll
    for (int v = 0; v < V; v++) total += l[v] > -INFINITY ? expf(l[v] - top) : 0.f;
    total = warp_sum(total);
  }
  if (BIAS || a.G > 1) route_scores<V>(a, l, b, top, total, c);
  const float eps = route_eps(a.softmax);
  uint32_t kept = 0xffffffffu;  // lanes (a group is `step` of them) or bits g of groups
  // the order goes by c; an expert that is not to be had is -inf, below all others
  if (!BIAS && a.G == 1) {
#pragma unroll
    for (int v = 0; v < V; v++) c[v] = l[v];
  }
  bool by_lane = false;
  if (a.G > 1) {
    bool near = a.step == 0;
    if (!near) {  // a group is `step` lanes, a power of two
      float m1 = c[0], m2 = -INFINITY;
#pragma unroll
      for (int v = 1; v < V; v++) {
        m2 = fmaxf(m2, fminf(m1, c[v]));
        m1 = fmaxf(m1, c[v]);
      }
      for (int o = 1; o < a.step; o <<= 1) {
        const float o1 = __shfl_xor_sync(0xffffffffu, m1, o);
        const float o2 = __shfl_xor_sync(0xffffffffu, m2, o);
        m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
        m1 = fmaxf(m1, o1);
      }
      const float s = a.best == 2 ? 0.5f * m1 + (m2 > -INFINITY ? 0.5f * m2 : 0.f) : m1;
      const int g = lane >> a.shift;  // lanes past the last group have ranks of G and more
      int rank = group_rank(s, g, a.G, a.step);
      if (a.keep < a.G) {
        const uint32_t last = __ballot_sync(0xffffffffu, g < a.G && rank == a.keep - 1);
        const uint32_t out = __ballot_sync(0xffffffffu, g < a.G && rank == a.keep);
        const float si = __shfl_sync(0xffffffffu, s, __ffs(last) - 1);
        const float so = __shfl_sync(0xffffffffu, s, __ffs(out) - 1);
        // without a bias a softmax's errors go with its size: the exponential's argument is off by
        // up to 88 u, and its smallest results by their last bits
        const float big = BIAS ? route_largest(m1, a.best == 2 ? m2 : 0.f) : 0.f;
        const float tol = a.softmax && !BIAS ? 0x1p-16f * si + 0x1p-120f
                                             : eps + 0x1p-21f * (BIAS ? big : si);
        if (so > -INFINITY && si - so <= tol) {
          near = BIAS && a.softmax;
          if (!near) {
            float l2[V], b2[V], c2[V];  // copies: what a call takes the address of is in memory
#pragma unroll
            for (int v = 0; v < V; v++) l2[v] = l[v], b2[v] = b[v], c2[v] = c[v];
            bool near2 = false;
            rank = route_groups_two<V>(a, l2, b2, c2, top, s, m1, m2, si, so, tol, big, rank,
                                       lane, (float *)buf[warp], near2);
            near = near2;
          }
        }
      }
#pragma unroll
      for (int v = 0; v < V; v++) c[v] = rank < a.keep ? BIAS ? c[v] : l[v] : -INFINITY;
      kept = __ballot_sync(0xffffffffu, rank < a.keep);
    }
    by_lane = !near;
    if (near) {
      kept = route_groups<T, V>(a, row, top, total, lane, buf[warp]);
      if (BIAS) route_scores<V>(a, l, b, top, total, c);
      const int gs = a.E / a.G;
#pragma unroll
      for (int v = 0; v < V; v++)
        c[v] = (kept >> min((V * lane + v) / gs, 31)) & 1 ? BIAS ? c[v] : l[v] : -INFINITY;
    }
  }
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; v++) key[v] = (route_key(c[v]) & ~(V - 1u)) | (V - 1 - v);
  route_sort<V>(key);
  constexpr uint32_t kPlace = V - 1u;  // the bits that give the place in the lane
  // The lane's keys by size in shared memory, and after them one of -inf; slots: keys and their
  // lanes as they come out
  uint32_t *const mem = (uint32_t *)buf[warp], *head = mem + lane;
  int2 *const slot = (int2 *)(mem + 32 * (V + 1));
  __syncwarp();
#pragma unroll
  for (int v = 1; v < V; v++) mem[32 * v + lane] = key[v];
  mem[32 * V + lane] = kRouteNone;
  const float rel = V > 1 ? 0x1p-19f : 0x1p-21f;
  const uint32_t before = (1u << lane) - 1;
  uint32_t mine = key[0];
  int n = 0;
  auto next_best = [&]() {  // the warp's best one leaves its lane
    const uint32_t hi = mine & ~kPlace;
    const uint32_t best = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t hold = __ballot_sync(0xffffffffu, hi == best);
    if (hi == best && (hold & before) == 0) {
      slot[n] = make_int2((int)mine, lane);
      head += 32;
      mine = *head;
    }
    return best;
  };
  // Whether two that follow each other lie too near: scores with a bias nearer than their error, and
  // fp32 logits that differ in the bits that gave way to the place at most.
  constexpr bool kNear = BIAS || (V > 1 && sizeof(T) == 4);
  auto near_keys = [&](uint32_t x, uint32_t y) {
    if (!BIAS) return x == y;
    const float p = route_value(x);
    return p - route_value(y) <= eps + rel * fabsf(p);
  };
  // the k largest and the one after them, and on through those that lie near to the last
  uint32_t last = 0, best = 0xffffffffu;
  for (; n <= a.k; n++) {
    last = best;
    best = next_best();
    if (best <= kRouteNone) break;
  }
  if (kNear)
    while (best > kRouteNone && n < 32 && near_keys(last, best)) {
      last = best;
      best = next_best();
      if (best > kRouteNone) n++;
    }
  __syncwarp();
  int id = -1;
  uint32_t key_of = 0;
  if (lane < n) {
    const int2 got = slot[lane];
    key_of = (uint32_t)got.x & ~kPlace;
    id = V * got.y + (int)(kPlace - ((uint32_t)got.x & kPlace));
  }
  float x = id >= 0 ? fminf(route_f32(row[id]), FLT_MAX) : -INFINITY;
  if (kNear) {
    // near, unless logit and bias are the same ones, which stand in their order
    const float bj = BIAS && id >= 0 ? a.bias[id] : 0.f;
    const uint32_t next = __shfl_down_sync(0xffffffffu, key_of, 1);
    const float lx = __shfl_down_sync(0xffffffffu, x, 1);
    const float bx = __shfl_down_sync(0xffffffffu, bj, 1);
    const bool near = lane < n - 1 && near_keys(key_of, next) && !(x == lx && bj == bx);
    if (__any_sync(0xffffffffu, near) || n == 32) {
      bool hard = n == 32 || (BIAS && a.softmax);
      if (!hard) {  // ranked again by the logits, or by scores in two floats
        const Two c2 = BIAS ? route_two(lane < n ? x : 0.f, bj, 0, 0.f) : Two{x, 0.f};
        int rank = 0;
        for (int q = 0; q < n; q++) {
          const float oh = __shfl_sync(0xffffffffu, c2.h, q), ol = __shfl_sync(0xffffffffu, c2.l, q);
          const float ox = __shfl_sync(0xffffffffu, x, q), ob = __shfl_sync(0xffffffffu, bj, q);
          const int oid = __shfl_sync(0xffffffffu, id, q);
          const float d = (oh - c2.h) + (ol - c2.l);
          if (ox == x && ob == bj) rank += oid < id;
          else if (!BIAS) rank += ox > x;
          else rank += d > 0.f, hard |= !(fabsf(d) > 0x1p-36f + 0x1p-44f * fabsf(c2.h));
        }
        hard = __any_sync(0xffffffffu, hard && lane < n);
        if (lane < n) slot[rank & 31].y = id;  // (a rank that is hard to tell is not used)
        __syncwarp();
        if (!hard) {
          id = lane < n ? slot[lane].y : -1;
          x = id >= 0 ? fminf(route_f32(row[id]), FLT_MAX) : -INFINITY;
        }
      }
      if (hard) {
        if (by_lane)  // lane 2^shift g has bit g
          kept = __ballot_sync(0xffffffffu, lane < a.G && ((kept >> ((lane << a.shift) & 31)) & 1));
        id = route_near<T, V>(a, row, kept, top, total, lane);
        x = id >= 0 ? fminf(route_f32(row[id]), FLT_MAX) : -INFINITY;
      }
    }
  }
  // weights: one slot a lane
  if (lane >= a.k) id = -1, x = -INFINITY;
  float s;
  if (a.norm) {
    if (a.softmax || __any_sync(0xffffffffu, route_deep(x)))
      s = route_share(x, a.softmax);
    else
      s = 1.f / (1.f + expf(-x));  // 0 of -inf
    s /= fmaxf(slots_sum(s), FLT_MIN);  // (none is chosen: 0)
  } else {
    s = a.softmax ? expf(x - top) / total : 1.f / (1.f + expf(-x));
  }
  if (lane < a.k) {
    a.ids[(size_t)t * a.k + lane] = id;
    a.w[(size_t)t * a.k + lane] = id >= 0 ? a.f * s : 0.f;
  }
}

// ------------------------------------------------------------------------------ gradient
// The choice is constant.  With v_j = w_j / f and D = sum_i v_i dw_i:
//   norm, softmax: dl_j = f v_j (dw_j - D)       norm, sigmoid: the same times 1 - s_j
//   sigmoid:       dl_j = f s_j (1 - s_j) dw_j
//   softmax:       dl_e = f s_e (dw_e - sum_i s_i dw_i), for every expert, dw_e = 0 if not chosen
// One warp a token writes the whole row (zeros, or the last line's terms), then the chosen ones'.
struct RouteGradArgs {
  const float *dw;
  const void *logits;
  const int32_t *ids;
  void *dlogits;
  long ld, ldd;
  int T, E, k, softmax, norm;
  float f;
  int vec;
};

template <typename T>
__device__ __forceinline__ T route_round(float v);
template <>
__device__ __forceinline__ float route_round<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 route_round<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half route_round<__half>(float v) { return __float2half_rn(v); }

// V neighbouring elements of a row from `e`, those before E
template <typename T, int V>
__device__ __forceinline__ void route_store(T *row, int e, int E, int vec, const T (&v)[V]) {
  alignas(16) T r[V];
#pragma unroll
  for (int i = 0; i < V; i++) r[i] = v[i];
  if (vec) {
    if (e >= E) return;
    if constexpr (sizeof(r) % 16 == 0) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(r) / 16; i++) ((uint4 *)(row + e))[i] = ((uint4 *)r)[i];
    } else if constexpr (sizeof(r) == 8) {
      *(uint2 *)(row + e) = *(uint2 *)r;
    } else if constexpr (sizeof(r) == 4) {
      *(uint32_t *)(row + e) = *(uint32_t *)r;
    } else {
      row[e] = r[0];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i++)
      if (e + i < E) row[e + i] = r[i];
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(32 * kRouteWarps) route_grad_kernel(const RouteGradArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kRouteWarps + warp;
  if (t >= a.T) return;
  const T *row = (const T *)a.logits + (size_t)t * a.ld;
  T *out = (T *)a.dlogits + (size_t)t * a.ldd;
  const bool whole = a.softmax && !a.norm;
  if (!whole) {  // while the loads are on their way
    if (sizeof(T) * V == 32 && a.vec) {  // (a lane's own 32 bytes are two halves of a sector)
#pragma unroll
      for (int i = 0; i < 2; i++)
        if ((32 * i + lane) * (V / 2) < a.E)
          *(uint4 *)(out + (32 * i + lane) * (V / 2)) = make_uint4(0, 0, 0, 0);
    } else {
      T zero[V];
#pragma unroll
      for (int v = 0; v < V; v++) zero[v] = route_round<T>(0.f);
      route_store<T, V>(out, V * lane, a.E, a.vec, zero);
    }
  }
  int id = lane < a.k ? a.ids[(size_t)t * a.k + lane] : -1;
  float x = -INFINITY, dw = 0.f;
  if (id >= 0 && id < a.E) {
    x = fminf(route_f32(row[id]), FLT_MAX);  // (a NaN gives FLT_MAX: told apart below)
    if (!(route_f32(row[id]) > -INFINITY)) x = -INFINITY;
  }
  if (!(x > -INFINITY)) id = -1;
  if (id >= 0) dw = a.dw[(size_t)t * a.k + lane];
  float l[V], top = -INFINITY, total = 1.f;
  if (whole) {
    route_load<T, V>(row, V * lane, a.E, a.vec, l);
#pragma unroll
    for (int v = 0; v < V; v++) top = fmaxf(top, l[v]);
    top = warp_max(top);
    total = 0.f;
#pragma unroll
    for (int v = 0; v < V; v++) {
      l[v] = l[v] > -INFINITY ? expf(l[v] - top) : 0.f;
      total += l[v];
    }
    total = warp_sum(total);
    if (total == 0.f) total = 1.f;  // no expert is available: every term is 0
  }
  float s, rest = 1.f;  // the score (0 of -inf), and 1 - a sigmoid
  if (a.norm && (a.softmax || __any_sync(0xffffffffu, route_deep(x))))
    s = route_share(x, a.softmax);
  else
    s = a.softmax ? expf(x - top) / total : 1.f / (1.f + expf(-x));
  if (!a.softmax) rest = 1.f / (1.f + expf(x));
  if (id < 0) s = 0.f;
  if (a.norm) s /= fmaxf(slots_sum(s), FLT_MIN);
  float D = a.norm || a.softmax ? slots_sum(s * dw) : 0.f;
  if (whole) D = __shfl_sync(0xffffffffu, D, 0);  // every lane's elements have it
  float g = a.f * s * rest * (dw - D);
  // an expert that stands in several slots gets them all
  bool first = id >= 0;
  const uint32_t same = __match_any_sync(0xffffffffu, id);
  if (__any_sync(0xffffffffu, id >= 0 && (same & (same - 1)))) {
    float sum = 0.f;
    // (whole: the row's own term belongs to one of them alone)
    const float mine = whole && id >= 0 ? a.f * s * dw : g;
    for (int q = 0; q < a.k; q++) {
      const float o = __shfl_sync(0xffffffffu, mine, q);
      if ((same >> q) & 1) sum += o;
    }
    if (id >= 0) {
      g = whole ? sum - a.f * s * D : sum;
      first = (same & ((1u << lane) - 1)) == 0;
    }
  }
  if (whole) {
    T r[V];
#pragma unroll
    for (int v = 0; v < V; v++) r[v] = route_round<T>(-a.f * (l[v] / total) * D);
    route_store<T, V>(out, V * lane, a.E, a.vec, r);
  }
  __syncwarp();  // the row before the chosen ones
  if (first) out[id] = route_round<T>(g);
}

// whether a lane's V elements of every row are one aligned access (16 bytes, or all of them)
static int route_vec(uintptr_t bits, int E, int V, int es) {
  const int n = V * es;
  return E % V == 0 && bits % (n < 16 ? n : 16) == 0;
}
static int route_v(int E) { return E <= 32 ? 1 : E <= 64 ? 2 : E <= 128 ? 4 : 8; }

template <typename T>
static cudaError_t launch_route(const RouteArgs &a, cudaStream_t st) {
  const dim3 grid((a.T + kRouteWarps - 1) / kRouteWarps), block(32 * kRouteWarps);
  auto go = [&](void (*biased)(const RouteArgs), void (*plain)(const RouteArgs)) {
    return launch_pdl(a.bias ? biased : plain, grid, block, 0, st, a);
  };
  switch (route_v(a.E)) {
    case 1: return go(route_logits_kernel<T, 1, true>, route_logits_kernel<T, 1, false>);
    case 2: return go(route_logits_kernel<T, 2, true>, route_logits_kernel<T, 2, false>);
    case 4: return go(route_logits_kernel<T, 4, true>, route_logits_kernel<T, 4, false>);
    default: return go(route_logits_kernel<T, 8, true>, route_logits_kernel<T, 8, false>);
  }
}
template <typename T>
static cudaError_t launch_route_grad(const RouteGradArgs &a, cudaStream_t st) {
  const dim3 grid((a.T + kRouteWarps - 1) / kRouteWarps), block(32 * kRouteWarps);
  switch (route_v(a.E)) {
    case 1: return launch_pdl(route_grad_kernel<T, 1>, grid, block, 0, st, a);
    case 2: return launch_pdl(route_grad_kernel<T, 2>, grid, block, 0, st, a);
    case 4: return launch_pdl(route_grad_kernel<T, 4>, grid, block, 0, st, a);
    default: return launch_pdl(route_grad_kernel<T, 8>, grid, block, 0, st, a);
  }
}

// what both calls check of their sizes and options
static int route_check(int T, int E, int k, moe_dtype dtype, int router, int norm, float f) {
  if (T < 0 || E < 0 || k < 0) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DT_F32 && dtype != MOE_DT_BF16 && dtype != MOE_DT_F16)
    return MOE_ERR_INVALID_ARG;
  if (router != MOE_ROUTER_SOFTMAX && router != MOE_ROUTER_SIGMOID_GROUPED)
    return MOE_ERR_INVALID_ARG;
  if ((norm != 0 && norm != 1) || !(f > -INFINITY && f < INFINITY)) return MOE_ERR_INVALID_ARG;
  if (E < 1 || E > kRouteMaxE || k < 1 || k > kRouteMaxK || k > E) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_route_logits(int T, int n_experts, int k, const void *logits, long ldl, moe_dtype dtype,
                     const float *bias, moe_router_kind router, int n_group, int topk_group,
                     int group_best, int norm_topk, float routed_scaling_factor, int32_t *ids,
                     float *w, void *stream) {
  if (int r = route_check(T, n_experts, k, dtype, router, norm_topk, routed_scaling_factor))
    return r;
  if (n_group < 1 || n_group > kRouteMaxG || n_experts % n_group || topk_group < 1 ||
      topk_group > n_group || group_best < 1 || group_best > 2)
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  const uintptr_t es = dtype == MOE_DT_F32 ? 4 : 2;
  if (!logits || !ids || !w || ldl < n_experts) return MOE_ERR_INVALID_ARG;
  if ((uintptr_t)logits % es || ((uintptr_t)bias | (uintptr_t)ids | (uintptr_t)w) % 4)
    return MOE_ERR_INVALID_ARG;
  const uintptr_t bits = (uintptr_t)logits | (T > 1 ? (uintptr_t)(ldl * (long)es) : 0);
  const int V = route_v(n_experts), gs = n_experts / n_group, lanes = gs / V;
  const bool run = gs % V == 0 && (lanes & (lanes - 1)) == 0;
  const int vec = route_vec(bits, n_experts, V, (int)es) && (uintptr_t)bias % 16 == 0;
  const RouteArgs a{logits, bias, ids, w, ldl, T, n_experts, k, n_group, topk_group, group_best,
                    router == MOE_ROUTER_SOFTMAX, norm_topk, routed_scaling_factor, vec,
                    run ? lanes : 0, run ? __builtin_ctz(lanes) : 0};
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == MOE_DT_F32    ? launch_route<float>(a, st)
                        : dtype == MOE_DT_BF16 ? launch_route<__nv_bfloat16>(a, st)
                                               : launch_route<__half>(a, st);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_route_logits_grad(int T, int n_experts, int k, const float *dw, const void *logits,
                          long ldl, moe_dtype dtype, const int32_t *ids, moe_router_kind router,
                          int norm_topk, float routed_scaling_factor, void *dlogits, long lddl,
                          void *stream) {
  if (int r = route_check(T, n_experts, k, dtype, router, norm_topk, routed_scaling_factor))
    return r;
  if (T == 0) return MOE_OK;
  const uintptr_t es = dtype == MOE_DT_F32 ? 4 : 2;
  if (!dw || !logits || !ids || !dlogits || ldl < n_experts || lddl < n_experts)
    return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)logits | (uintptr_t)dlogits) % es || ((uintptr_t)dw | (uintptr_t)ids) % 4)
    return MOE_ERR_INVALID_ARG;
  const uintptr_t bits = (uintptr_t)logits | (uintptr_t)dlogits |
                         (T > 1 ? (uintptr_t)(ldl * (long)es) | (uintptr_t)(lddl * (long)es) : 0);
  const RouteGradArgs a{dw, logits, ids, dlogits, ldl, lddl, T, n_experts, k,
                        router == MOE_ROUTER_SOFTMAX, norm_topk, routed_scaling_factor,
                        route_vec(bits, n_experts, route_v(n_experts), (int)es)};
  const cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == MOE_DT_F32    ? launch_route_grad<float>(a, st)
                        : dtype == MOE_DT_BF16 ? launch_route_grad<__nv_bfloat16>(a, st)
                                               : launch_route_grad<__half>(a, st);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
