// linear_plan.cuh -- sizes and rules of the matrix products' launches that need no GPU: plain C++, so
// that they are tested without one.
#pragma once

#include <algorithm>
#include <cmath>

namespace moe {

constexpr int kLinM = 128;            // weight rows per CTA and tile
constexpr int kLinStages = 12;        // ring slots at most
constexpr int kLinRing = 192 * 1024;  // shared memory of the ring and the exchange, at most
// fp32 outputs: the largest tiles whose sums fit the registers
constexpr int kLinExactN = 128, kLinExactSplitN = 64;

// How CTAs share a tile:
//   kOne    one CTA a tile, persistent.
//   kPair   two CTAs (the two SMs of a TPC) a tile of 256 weight rows: each loads its own 128
//           weight rows and half of the token rows, and the leader issues MMAs of M = 256 that
//           read both halves, so token rows cross from L2 once for 256 weight rows.
//   kSplit  a cluster of up to eight CTAs a tile, each over a part of K, not persistent: the
//           partial sums are exchanged through distributed shared memory and added in rank
//           order, each CTA finishing a share of the columns.
enum LinMode { kOne = 0, kPair = 1, kSplit = 2 };

// ---------------------------------------------------------------- 8-bit integers
constexpr int kI8Slots = 4;   // fp16 sub-blocks on their way to the MMA
constexpr int kI8MaxN = 192;  // token rows per tile

// columns of a split tile that one CTA finishes, and the bytes of the partial sums' exchange
inline int i8_exchange(int BN, int split) {
  const int cpc = ((BN + split - 1) / split + 3) & ~3;
  return split * cpc * kLinM * 4;
}

// raw stages beside the exchange and the token sub-blocks of xrows rows
inline int i8_stages(int xrows, int exchange) {
  return std::min(kLinStages,
                  (kLinRing - exchange - kI8Slots * xrows * 128) / ((kLinM + xrows) * 128));
}

struct I8Plan {
  int mode, BN, split;
  long tiles;
  bool sure;  // made with every answer
};

// How to cut the product: an estimate in SM cycles of each candidate.  A k-block of 128 takes as long as
// its MMAs (4 cycles a column), 800 cycles (a hand-over and eight MMAs take no less), or the rows that
// are turned into fp16 (3.5 cycles each), whichever is longest; joining a split tile takes 2000 cycles and
// 12 a column and other CTA.  Over 16 shapes (64 to 32768 rows, 1024 to 8192 features, K 1024 to 14336,
// 0 to 64 experts) the form taken is 2% slower than the fastest of six widths in every mode in the
// mean, 11% at worst (4096 rows of 64 experts: one CTA a tile 348 us, a pair 313).  sms: of the device;
// clusters: of 2, 4 and 8 CTAs that run on it at a time (0: not known).
inline I8Plan i8_make_plan(int R, int N, int E, int KB, bool gated, bool exact, int sms,
                           const int (&clusters)[3]) {
  // experts that get rows, and rows of one of them, when rows fall on experts evenly
  const double active = E > 1 ? E * (1.0 - std::pow(1.0 - 1.0 / E, R)) : 1.0;
  const double m = R / active;
  const int rows = gated ? 2 * N : N;
  I8Plan best{};
  best.sure = clusters[0] > 0 && clusters[1] > 0 && clusters[2] > 0;
  double cost = 1e30;
  for (int mode = 0; mode < 3; mode++)
    for (int BN = 16; BN <= kI8MaxN; BN += 16)
      for (int split = mode == kSplit ? 2 : 1; split <= (mode == kSplit ? 8 : 1); split *= 2) {
        if (mode == kPair && (BN < 64 || BN % 32 || rows <= kLinM)) continue;
        if (split > KB) continue;
        if (exact && (mode == kPair || BN > (mode == kSplit ? kLinExactSplitN : kLinExactN)))
          continue;
        const int FT = (rows + (mode == kPair ? 255 : 127)) / (mode == kPair ? 256 : 128);
        const double rt = E ? std::max(1.0, m / BN + 0.5) : (double)((R + BN - 1) / BN);
        const double tiles = active * rt * FT;
        const double cols = std::min((double)BN, m);
        const double x = mode == kPair ? cols / 2 : cols;
        const double kb = std::max({4.0 * cols, 800.0, 3.5 * (kLinM + x)});
        double c;
        if (mode == kSplit) {  // one tile a cluster
          if (tiles > clusters[split == 2 ? 0 : split == 4 ? 1 : 2]) continue;
          if (i8_stages(BN, i8_exchange(BN, split)) < 2) continue;
          c = (KB + split - 1) / split * kb + 2000 + 12.0 * BN * (split - 1);
        } else {
          const double width = mode == kPair ? sms / 2 : sms;
          const double waves = E ? std::max(1.0, tiles / width + 0.3) : std::ceil(tiles / width);
          c = waves * KB * kb + 500 + 4.0 * BN;  // the last tile's epilogue
        }
        if (c < cost * 0.999) {
          cost = c;
          best.mode = mode, best.BN = BN, best.split = split;
        }
      }
  const int FT = (rows + (best.mode == kPair ? 255 : 127)) / (best.mode == kPair ? 256 : 128);
  // at most so many tiles exist, however the rows fall on the experts
  const long rt = E ? (long)std::min(R, E) + R / best.BN : (R + best.BN - 1) / best.BN;
  best.tiles = rt * FT;
  return best;
}

}  // namespace moe
