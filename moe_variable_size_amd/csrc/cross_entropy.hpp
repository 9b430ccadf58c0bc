// What the linear cross entropy's kernels share with the tiles of the dense product (linear.hip).
#pragma once
#include "common.hpp"

namespace moe {

// A row of the backward: dl = scale exp(l - lse) - [v = target] g
struct __attribute__((aligned(16))) CeRow {
  float lse, scale, g;
  int target;  // -1: none (a target outside the vocabulary): dl = 0
};

struct CeArgs {
  // forward
  const void *targets;  // [M] int32 or int64
  bool wide;            // int64
  float2 *part;         // [parts][M]: largest logit, sum of exp(l - largest), of each run of columns
  int part0;            // first of this launch's
  float *target_logit;  // [M]
  // backward
  const CeRow *rows;    // [M]
  int64_t ld;           // dl's row length
  bf16_t *rest;         // what dl's rounding leaves (bf16; NULL: not kept)
  // both
  int64_t col0, V;      // first column of this piece of the vocabulary; the whole vocabulary
};

// Row m's target as a column of this piece; -1 where it is elsewhere or nowhere
MOE_DEV int64_t ce_target_id(const CeArgs &a, int64_t m) {
  const int64_t t = a.wide ? ((const int64_t *)a.targets)[m] : ((const int32_t *)a.targets)[m];
  return t >= 0 && t < a.V ? t : -1;
}
MOE_DEV int ce_target(const CeArgs &a, int64_t m) {
  const int64_t t = ce_target_id(a, m) - a.col0;
  return t >= 0 && t < (1 << 30) ? (int)t : -1;
}

// What is subtracted from logits whose largest is `top`: that, or 0 where nothing is above -inf (its sum stays 0)
MOE_DEV float ce_base(float top) { return top == -INFINITY ? 0.f : top; }
MOE_DEV float2 ce_join(float2 a, float2 b) {
  const float top = fmaxf(a.x, b.x), base = ce_base(top);
  return float2{top, a.y * __expf(a.x - base) + b.y * __expf(b.x - base)};
}
// fp32 operands take the exact exponential (the hardware's is off by some 2^-21 at |l - lse| = 10)
template <typename T>
MOE_DEV float ce_exp(float d) {
  return sizeof(T) == 4 ? expf(d) : __expf(d);
}
template <typename T>
MOE_DEV float ce_dl(const CeRow &r, float l, int64_t col) {
  if (r.target < 0) return 0.f;
  const float d = r.scale * ce_exp<T>(l - r.lse);
  return col == r.target ? d - r.g : d;
}

// Products (linear.hip).
// Whether x W^T takes tiles that can have the epilogues above (bf16 on 16-byte lines)
bool ce_tiles(int64_t M, int64_t K, int64_t V);
// Columns of a tile, for a piece of V columns
int ce_tile_columns(int64_t M, int64_t K, int64_t V);
// dl NULL: the forward's statistics; shape_v: the size that the tile's shape goes by
hipError_t launch_ce_tiles(const void *x, const void *W, void *dl, const CeArgs &ce, int M, int K, int V, int shape_v,
                           hipStream_t st);
// The same in tiles for any alignment, staged ones for bf16 and those of bf16 parts for fp32: whether their reduction is
// whole, the columns of a wave
bool ce_staged(int64_t M, int64_t K, int64_t V, int dtype);
int ce_staged_columns(int64_t M, int64_t K, int64_t V, int dtype);
hipError_t launch_ce_staged(const void *x, const void *W, void *dl, const CeArgs &ce, int M, int K, int V, int shape_v, int dtype,
                            hipStream_t st);
// Workspaces of dX and dW, and of logits that are left in memory; these logits
size_t ce_part_bytes(int64_t M, int64_t K, int64_t V, int dtype);
size_t ce_logits_part_bytes(int64_t M, int64_t K, int64_t V, int dtype);
hipError_t launch_ce_logits(const void *x, const void *W, float *logits, int M, int K, int V, int dtype, void *part, hipStream_t st);
// out = factor dl W + sum (factor [M], NULL: 1; sum NULL: 0; fp32, may be out)
hipError_t launch_ce_dx(const void *dl, int64_t ld, const void *W, const float *sum, const float *factor, void *out, bool out_f32,
                        int M, int K, int V, int dtype, void *part, hipStream_t st);
// dW = factor dl^T x (factor [1], NULL: 1)
hipError_t launch_ce_dw(const void *dl, int64_t ld, const void *x, const float *factor, void *dW, int M, int K, int V, int dtype,
                        void *part, hipStream_t st);
}  // namespace moe
