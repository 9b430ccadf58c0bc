// Which tiles a product of the dense linear layer takes, from its sizes alone.  Plain host code, so that
// the tests can ask the same rule.
#pragma once
#include <stdint.h>

namespace moe {

constexpr int PBK = 64;  // reduction elements per stage of the pipelined and ring tiles
constexpr int SBK = 32;  // per step of the staged tiles
constexpr int kShapeM[3] = {256, 256, 128}, kShapeN[3] = {256, 128, 128};  // tile shapes

// Tile shape and number of reduction ranges of a product of M x N outputs.
struct Plan {
  int shape, splits;  // shape: 0 = 256 x 256, 1 = 256 x 128, 2 = 128 x 128
};

// The choice minimises an estimate in us: rounds of workgroups over the chip (256 CUs; two 128 x 128
// workgroups fit one) times the stages of a range at the shape's measured time per stage, 6 us of
// launch, first loads and epilogue, and for split reductions the join: a launch, and the partial
// products written and read at 4 TB/s.  Per stage: 256 x 256 1.35 us, 256 x 128 0.92, 128 x 128 0.5
// alone on a CU and 1.0 in pairs.  Measured, us (256 x 256 / 256 x 128 / 128 x 128 / the last in two
// ranges): 8192 x 4096 x 4096 198 / 240 / 252 / 389, 4096 x 2048 x 2048 47 / 35 / 38 / 60, 2048^3 43 / 31 /
// 24 / 35, 512 x 4096 x 4096 74 / 51 / 33 / 31, 64 x 4096 x 4096 71 / 49 / 30 / 21.  Few rows, 128 x 128 in 4 / 6 /
// 8 / 12 / 16 ranges (the rule's in brackets): 32 x 4096 x 4096 13.9 / 13.0 / [12.9] / 14.7 / 14.9, 64 x 4096 x
// 4096 14.4 / 14.2 / [14.6] / 16.9 / 18.1, 128 x 4096 x 4096 16.4 / [17.5] / 18.2 / 21.0 / 23.6, 128 x 7168 x 2048
// 20.5 / 17.3 / [16.6] / 17.8 / 19.2, 8192 x 4096 x 64 [18.7] / 20.9 / 21.6 / 27.5 / 31.2.
inline Plan plan_of(int64_t M, int64_t N, int64_t K) {
  constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
  const int64_t stages = (K + PBK - 1) / PBK;
  Plan best{0, 1};
  double least = 0;
  for (int sh = 0; sh < 3; ++sh) {
    const double tiles = (double)((M + kShapeM[sh] - 1) / kShapeM[sh]) * ((N + kShapeN[sh] - 1) / kShapeN[sh]);
    for (int k : kSplits) {
      if (k > 1 && (stages < 2 * k || tiles * k > 512)) break;
      const double wgs = tiles * k, per = (double)((stages + k - 1) / k);
      double t;
      if (sh == 2)
        t = wgs <= 256 ? per * 0.5 : __builtin_ceil(wgs / 512) * per * 1.0;
      else
        t = __builtin_ceil(wgs / 256) * per * (sh == 0 ? 1.35 : 0.92);
      t += 6;
      if (k > 1) t += 4 + (2.0 * k + 1) * M * N * 4 / 4e6;
      if (least == 0 || t < least) {
        least = t;
        best = Plan{sh, k};
      }
    }
  }
  return best;
}
// The shape of the same estimate for a product that cannot split its reduction (its epilogue needs the sums).
inline int unsplit_shape(int64_t M, int64_t N, int64_t K) {
  const int64_t stages = (K + PBK - 1) / PBK;
  int best = 0;
  double least = 0;
  for (int sh = 0; sh < 3; ++sh) {
    const double wgs = (double)((M + kShapeM[sh] - 1) / kShapeM[sh]) * ((N + kShapeN[sh] - 1) / kShapeN[sh]);
    const double t = sh == 2 ? (wgs <= 256 ? 0.5 : __builtin_ceil(wgs / 512)) * stages
                             : __builtin_ceil(wgs / 256) * stages * (sh == 0 ? 1.35 : 0.92);
    if (least == 0 || t < least) {
      least = t;
      best = sh;
    }
  }
  return best;
}
// The staged kernel's: bf16 takes 128 x 128 tiles (S = 2) where they fill the chip twice; else, and in fp32
// always, 64 x 64 (timed in turn, fp32 4096^3: 1072 us against 1236, 8192 x 2048 x 2048 510 against 626: the fp32
// products are slow enough that the operands' traffic does not matter, and more waves share the CU), with
// the reduction cut until there are about four workgroups per CU, of at least 4 steps each (fp32
// backward of 1237 x 1001 x 499: 128 x 128 tiles uncut 180 us of products, cut 64 x 64 tiles 41).
inline Plan staged_plan(int64_t M, int64_t N, int64_t K, bool bf16) {
  const int64_t t2 = ((M + 127) / 128) * ((N + 127) / 128), t1 = ((M + 63) / 64) * ((N + 63) / 64);
  if (bf16 && t2 >= 512) return Plan{2, 1};
  const int64_t steps = (K + SBK - 1) / SBK;
  int64_t k = t1 > 0 ? 1024 / t1 : 1;
  if (k > steps / 4) k = steps / 4;
  if (k > 16) k = 16;
  return Plan{1, (int)(k < 1 ? 1 : k)};
}
// The cross entropy's fp32 products in three parts of bf16 (shape: S, tiles of 64 S x 64 S; a range's reduction in steps of
// 16), by the same kind of estimate: a step of a CU's c workgroups takes 0.28 c us for S = 1 (0.47 at least), for S = 2, of
// which a CU holds two, 0.79, 1.2 and then 0.67 c, and a tile's ends as much as 3 and 9 steps.  Measured, us, without the join
// (the rule's in brackets): 1074 x 47121 x 600 S = 1 494, [2 413]; 777 x 5003 x 1001 1 100, [2 91]; 132 x 37693 x 6408 [1 707], 2
// 730; 64 x 32000 x 4096 [1 168], 2 220; reductions in ranges, 777 x 1001 x 5003 1 in 4 79, 2 in 4 71, [2 in 8 60]; 1074 x 600 x
// 47121 1 in 6 503, 2 in 4 516, [2 in 8 432].
inline Plan fine_plan(int64_t M, int64_t N, int64_t K, bool split, double *us = nullptr) {
  constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
  const int64_t steps = (K + 15) / 16;
  Plan best{1, 1};
  double least = 0;
  for (int S = 1; S <= 2; ++S) {
    const double tiles = (double)((M + 64 * S - 1) / (64 * S)) * ((N + 64 * S - 1) / (64 * S));
    for (int k : kSplits) {
      if (k > 1 && (!split || steps < 4 * k || tiles * k > 1280 / S)) break;
      const double c = __builtin_ceil(tiles * k / 256), alone = S == 1 ? 0.47 : 0.79, each = S == 1 ? 0.28 : c <= 2 ? 0.6 : 0.67;
      double t = 6 + ((steps + k - 1) / k + (S == 1 ? 3 : 9)) * (each * c > alone ? each * c : alone);
      if (k > 1) t += 4 + (2.0 * k + 1) * M * N * 4 / 4e6;
      if (least == 0 || t < least) {
        least = t;
        best = Plan{S, k};
      }
    }
  }
  if (us) *us = least;
  return best;
}
// Whether the logits' product is better not split, so that it ends in the statistics or the gradient: a split one writes
// logits that have to be read again.  344 x 2838 x 2632: 100 us whole, in ranges 43 and 14 for the join and the logits; 777 x
// 5003 x 1001: 91 whole, 74 and 35.
inline bool fine_whole(int64_t M, int64_t V, int64_t K) {
  double whole, split;
  fine_plan(M, V, K, false, &whole);
  fine_plan(M, V, K, true, &split);
  return whole <= split + 5 + 8.0 * M * V / 4e6;
}
// Rows of one launch, at most M of them.  A dispatch holds fewer than 2^32 work-items: the streamed
// products take 64 per row of x (at most 16 columns), the smallest tiles 256 per 64 x 64 outputs.  Both are
// kept at 2^31; a product of more is cut into runs of equally many rows (whole runs of 64, so that
// alignments stay), each of over 2^17 small tiles, so none of them splits its reduction.
inline int64_t launch_rows(int64_t M, int64_t N) {
  int64_t most = ((int64_t)1 << 29) / ((N + 63) / 64);
  if (most > 1 << 25) most = 1 << 25;
  if (M <= most) return M;
  const int64_t runs = (M + most - 1) / most, per = (M + runs - 1) / runs;
  return (per + 63) / 64 * 64;
}
// Stages of the ring of 128 x 128 tiles (ring_gemm's NST)
inline int ring_stages(int64_t workgroups, int cus) { return workgroups <= cus ? 4 : 2; }

}  // namespace moe
