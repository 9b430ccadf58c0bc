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
// Reduction ranges of a product in fp32 staged tiles of a cross entropy's gradient: the same limits, chosen by rounds of
// workgroups over the 256 CUs (0.63 us per step of each that shares a CU, 0.85 alone) and what the join costs, as plan_of.
// dX of 777 x 5003 x 1001 (208 tiles) in 1 range 133 us, in 4, as above, 102, in 6 90 (and 6 for the join).
inline int rounds_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t t1 = ((M + 63) / 64) * ((N + 63) / 64), steps = (K + SBK - 1) / SBK;
  int best = 1;
  double least = 0;
  for (int k = 1; k <= 16 && (k == 1 || (steps >= 4 * k && t1 * k <= 2560)); ++k) {
    const double each = __builtin_ceil(t1 * k / 256.0) * 0.63;
    double t = (each > 0.85 ? each : 0.85) * __builtin_ceil((double)steps / k);
    if (k > 1) t += 4 + (2.0 * k + 1) * M * N * 4 / 4e6;
    if (k == 1 || t < least) {
      least = t;
      best = k;
    }
  }
  return best;
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
