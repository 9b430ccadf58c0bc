// Cross entropy of the logits l = x W^T over a large vocabulary, and its gradient, without keeping them:
//   lse_m = log sum_v exp l_mv,   loss_m = lse_m - l_m,t + z lse_m^2,
//   dl_mv = g_m ((1 + 2 z lse_m) exp(l_mv - lse_m) - [v = t_m]),   dX = dl W,   dW = dl^T x.
//
// Forward: the product's tiles keep their logits in registers and leave per row the largest and the sum of
// exp(l - largest) of their columns (linear.hip, ce_stats); the parts of a row are joined here.  Backward:
// the vocabulary goes by in pieces; a piece's dl, M x piece, comes out of the product that computes its
// logits again (ce_grad), then dW's rows of the piece are one product, and dX another that adds to a sum in
// fp32.  dl is rounded once, to nearest, to the operands' type, as the matrix instructions take it.  In bf16 a rounding is up to
// 2^-8 of an entry, and the target's entry, g (p - 1) for small p, carries most of its row's gradient: were g in it, rows that share
// g, as those of a mean do, would all be off by the same part in the same direction (with 1020 rows and g = 1 / 1020, 2^-8: the
// gradients by 2.4 times their own rounding in norm).  So dl is taken without g, and g goes in fp32 into dX's epilogue, row by
// row, and where all rows share it into dW's.  Then a target's entry p - 1 is off by at most p, and by 2^-9, and differs from row to
// row as p does.  Where rows differ in g, dW = G dl^T x' with G the largest |g| that is finite and x' = bf16(g / G x): one more
// rounding of its own (none where they are alike), but of every element for itself.  Up to 512 rows of bf16 dl, with g, is two rows,
// its rounding and what that leaves, twice the rows in two of the three products: the gradients then are as good as their own
// rounding at any p.  Backward of 512 and 513 rows x 4096 x 32000: 625 and 564 us; error in norm with p from 0 to 1: 0.0017 and
// 0.0020.  bf16 rows off 16-byte lines do the same in the staged tiles, fp32 in tiles that multiply three parts of bf16.  Few rows, and products so small that their reduction
// is better split, write a piece's logits in fp32 to the workspace and read them back.
//
// bf16, 8192 x 4096 x 65536: 12.7 to 13.1 ms for the loss and both gradients, four products (17.6 TFLOP) at 1.34 to 1.39 PFLOP/s and 68 us
// besides (20 of them x by the rows' weights, not for a mean or a sum); the loss of 2048 x 4096 x 50257 646 to 676 us.  fp32, 1074 x 600 x
// 47121, loss and gradients: 1.60 ms (2.36 by fp32 instructions; 1.99 for logits kept and three such products).  One row x 4096 x 32000: 51 us, 38 of them the streamed product (7.0 TB/s),
// the others two launches.
#include "cross_entropy.hpp"

namespace moe {
namespace {

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
bool on_line(const void *p) { return (uintptr_t)p % 16 == 0; }

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

MOE_DEV void st(float *p, float v) { *p = v; }
MOE_DEV void st(bf16_t *p, float v) { *p = __builtin_bit_cast(bf16_t, (__bf16)v); }

// ---- logits in memory ---------------------------------------------------------
constexpr int CHUNK = 2048;  // columns of a row that a workgroup takes
constexpr int kGrid = 1 << 16;

// part[chunk][m] of a piece of n columns; pieces after the first are joined to what is there
__global__ __launch_bounds__(256) void stats_kernel(const float *__restrict__ l, CeArgs a, int64_t M, int n, int chunks) {
  __shared__ float2 red[4];
  const int64_t total = M * chunks;
  for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
    const int64_t m = b / chunks;
    const int c = (int)(b - m * chunks), hi = min(n, (c + 1) * CHUNK);
    float v[CHUNK / 256], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < CHUNK / 256; ++i) {
      const int col = c * CHUNK + i * 256 + threadIdx.x;
      v[i] = col < hi ? l[m * n + col] : -INFINITY;
      top = fmaxf(top, v[i]);
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    const float base = ce_base(top);
#pragma unroll
    for (int i = 0; i < CHUNK / 256; ++i) sum += expf(v[i] - base);
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = float2{top, sum};
    __syncthreads();
    if (threadIdx.x == 0) {
      float2 r = ce_join(ce_join(red[0], red[1]), ce_join(red[2], red[3]));
      float2 *at = a.part + (int64_t)c * M + m;
      *at = a.col0 ? ce_join(*at, r) : r;
      const int t = ce_target(a, m);
      if (t >= c * CHUNK && t < hi) a.target_logit[m] = l[m * n + t];
    }
    __syncthreads();
  }
}

// dl of a piece, zeros behind it up to its row length
template <typename T>
__global__ __launch_bounds__(256) void dl_kernel(const float *__restrict__ l, CeArgs a, T *__restrict__ dl, int64_t M,
                                                 int n, int chunks) {
  const int64_t total = M * chunks;
  for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
    const int64_t m = b / chunks;
    const int c = (int)(b - m * chunks), hi = min(n, (c + 1) * CHUNK);
    const CeRow r = a.rows[m];
    if (hi == n && threadIdx.x < a.ld - n) {
      st(dl + m * a.ld + n + threadIdx.x, 0.f);
      if (a.rest) st(a.rest + m * a.ld + n + threadIdx.x, 0.f);
    }
#pragma unroll
    for (int i = 0; i < CHUNK / 256; ++i) {
      const int col = c * CHUNK + i * 256 + threadIdx.x;
      if (col >= hi) break;
      const float d = ce_dl<T>(r, l[m * n + col], a.col0 + col);
      st(dl + m * a.ld + col, d);
      if (a.rest) st(a.rest + m * a.ld + col, d - (float)(__bf16)d);
    }
  }
}

// ---- rows -------------------------------------------------------------------------
// loss and lse from a row's parts.  LANES = 64: a wave per row, 4 rows per workgroup; 16: a workgroup takes 16 rows, whose
// parts lie side by side (a line), 16 threads each, from M = 256 on.  8192 rows of 256 parts: 31 us with 4 threads a row.
template <int LANES>
__global__ __launch_bounds__(256) void join_kernel(CeArgs a, int64_t M, int parts, float z, float *loss, float *lse) {
  __shared__ float2 red[16][16];
  const int lane = LANES == 64 ? threadIdx.x & 63 : threadIdx.x >> 4, row = threadIdx.x & 15;
  const int64_t m = LANES == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x * 16 + row;
  float2 r{-INFINITY, 0.f};
  if (m < M) {
#pragma unroll 4
    for (int p = lane; p < parts; p += LANES) r = ce_join(r, a.part[(int64_t)p * M + m]);
  }
  if constexpr (LANES == 64) {
#pragma unroll
    for (int d = 32; d; d >>= 1) r = ce_join(r, float2{__shfl_xor(r.x, d, 64), __shfl_xor(r.y, d, 64)});
  } else {
    red[lane][row] = r;
    __syncthreads();
#pragma unroll
    for (int i = 1; i < 16; ++i) r = ce_join(r, red[i][row]);  // (thread 0 of a row: its own first)
  }
  if (lane || m >= M) return;
  const float v = r.x + logf(r.y);
  lse[m] = v;
  loss[m] = ce_target_id(a, m) < 0 ? 0.f : v - a.target_logit[m] + z * v * v;
}

// {sum of loss, rows that count, sum / rows}; sums in 64 bits, in a fixed order
__global__ __launch_bounds__(1024) void total_kernel(CeArgs a, int64_t M, const float *__restrict__ loss, float *total) {
  __shared__ double s[16];
  __shared__ int64_t c[16];
  double sum = 0;
  int64_t count = 0;
  for (int64_t m = threadIdx.x; m < M; m += 1024) {
    if (ce_target_id(a, m) < 0) continue;
    sum += loss[m];
    ++count;
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    sum += __shfl_xor(sum, d, 64);
    count += __shfl_xor((long long)count, d, 64);
  }
  if ((threadIdx.x & 63) == 0) {
    s[threadIdx.x >> 6] = sum;
    c[threadIdx.x >> 6] = count;
  }
  __syncthreads();
  if (threadIdx.x) return;
  for (int i = 1; i < 16; ++i) {
    sum += s[i];
    count += c[i];
  }
  total[0] = (float)sum;
  total[1] = (float)count;
  total[2] = count ? (float)(sum / (double)count) : 0.f;
}

// factor [M + 1]: g is kept out of dl and put there, 0 for a row that does not count; behind the rows' the one that all share
__global__ __launch_bounds__(256) void rows_kernel(CeArgs a, int64_t M, const float *d_loss, const float *lse,
                                                   const float *total, int reduction, float z, CeRow *rows, float *factor) {
  const int64_t m = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (m >= M) return;
  const int64_t t = ce_target_id(a, m);
  float g = d_loss[reduction == MOE_REDUCE_NONE ? m : 0];
  if (reduction == MOE_REDUCE_MEAN) g = total[1] > 0.f ? g / total[1] : 0.f;
  if (factor) {
    factor[m] = t < 0 ? 0.f : g;
    if (m == 0) factor[M] = reduction == MOE_REDUCE_NONE ? 0.f : g;
    g = 1.f;
  }
  const float v = lse[m];
  rows[m] = CeRow{v, g * (1.f + 2.f * z * v), g, (int)t};
}

// factor[M], 0 so far: the largest of the rows' magnitudes that are finite (whose bits are in the numbers' order)
__global__ __launch_bounds__(256) void largest_kernel(float *factor, int64_t M) {
  float top = 0.f;
  for (int64_t m = (int64_t)blockIdx.x * 256 + threadIdx.x; m < M; m += (int64_t)gridDim.x * 256) {
    const float g = fabsf(factor[m]);
    if (g < INFINITY) top = fmaxf(top, g);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  if ((threadIdx.x & 63) == 0) atomicMax((uint32_t *)factor + M, __float_as_uint(top));
}
// y = x with its rows times their part of factor[M], 8 elements of a row at a time (W: rows on 16-byte lines) or one
template <bool W>
__global__ __launch_bounds__(256) void weigh_kernel(const bf16_t *__restrict__ x, bf16_t *__restrict__ y, const float *factor, int64_t M,
                                                    int64_t K) {
  typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
  constexpr int E = W ? 8 : 1;
  const float top = factor[M] > 0.f ? factor[M] : 1.f;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * E; i < M * K; i += (int64_t)gridDim.x * 256 * E) {
    const float f = factor[i / K] / top;
    if constexpr (W) {
      const bf16x8 v = *(const bf16x8 *)(x + i);
      bf16x8 r;
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = (__bf16)((float)v[e] * f);
      *(bf16x8 *)(y + i) = r;
    } else {
      st(y + i, bf16_to_f32(x[i]) * f);
    }
  }
}

// x twice, for the two parts of dl
__global__ __launch_bounds__(256) void twice_kernel(const bf16_t *__restrict__ x, bf16_t *__restrict__ y, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) y[i] = y[n + i] = x[i];
}
__global__ __launch_bounds__(256) void add_kernel(const float *__restrict__ x, bf16_t *__restrict__ y, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) st(y + i, x[i] + x[n + i]);
}
__global__ __launch_bounds__(256) void round_kernel(const float *__restrict__ x, bf16_t *__restrict__ y, int64_t n, bool wide) {
  const int64_t step = (int64_t)gridDim.x * 1024;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += step) {
    if (wide && i + 4 <= n) {
      const f32x4 v = *(const f32x4 *)(x + i);
      *(bf16x4 *)(y + i) = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    } else {
      for (int e = 0; e < 4 && i + e < n; ++e) st(y + i + e, x[i + e]);
    }
  }
}

// ---- pieces and workspaces, from the sizes alone -----------------------------------
int64_t even_piece(int64_t V, int64_t most) {  // equal pieces of whole tiles, of at most `most` columns (>= 256)
  if (V <= most) return V;
  const int64_t count = (V + most - 1) / most;
  const int64_t p = ((V + count - 1) / count + 255) / 256 * 256;
  return p <= most ? p : most / 256 * 256;
}
int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }
int64_t greatest(int64_t a, int64_t b) { return a > b ? a : b; }
int64_t weight_piece(int64_t K) { return greatest(256, least(((int64_t)1 << 30) / K - 1, 1 << 20) / 256 * 256); }

// How a piece's logits are taken: by the tiles that end in the epilogues above, of which `tiles` need rows on 16-byte
// lines; else through memory.
enum Way { TILES, STAGED, MEMORY };

struct Fwd {
  int64_t piece;
  int columns, parts;               // of a part; parts of a row
  size_t part, logits, gemm, total;  // offsets of the parts (after the targets' logits), ...
};
int64_t fwd_piece(int64_t M, int64_t K, int64_t V, Way way) {
  if (way == TILES) return even_piece(V, weight_piece(K));
  if (way == STAGED) return even_piece(V, ((int64_t)1 << 29) / M * 64 / 256 * 256);  // of one launch
  return even_piece(V, greatest(1024, ((int64_t)1 << 26) / M / 256 * 256));          // 256 MB of logits
}
// (fp32 tiles take no fewer than four columns, the last piece's among them)
bool staged(int64_t M, int64_t K, int64_t V, int64_t piece, int dtype) {
  return ce_staged(M, K, piece, dtype) && (dtype == MOE_BF16 || V % piece == 0 || V % piece >= 4);
}
Way fwd_way(int64_t M, int64_t K, int64_t V, int dtype, bool on_lines) {
  if (on_lines && dtype == MOE_BF16 && ce_tiles(M, K, fwd_piece(M, K, V, TILES))) return TILES;
  return staged(M, K, V, fwd_piece(M, K, V, STAGED), dtype) ? STAGED : MEMORY;
}
Fwd fwd_space(int64_t M, int64_t K, int64_t V, int dtype, Way way) {
  Fwd f;
  f.part = up256((size_t)M * 4);
  f.piece = fwd_piece(M, K, V, way);
  f.columns = way == TILES ? ce_tile_columns(M, K, f.piece) : way == STAGED ? ce_staged_columns(M, K, f.piece, dtype) : CHUNK;
  // (a staged tile has two waves' columns, used or not; parts in memory are shared by the pieces)
  auto of = [&](int64_t n) { return way == STAGED ? (n + 2 * f.columns - 1) / (2 * f.columns) * 2 : (n + f.columns - 1) / f.columns; };
  f.parts = (int)of(f.piece);
  if (way != MEMORY)
    for (int64_t v = f.piece; v < V; v += f.piece) f.parts += (int)of(least(f.piece, V - v));
  f.logits = f.part + up256((size_t)f.parts * M * 8);
  f.gemm = f.logits + (way == MEMORY ? up256((size_t)M * f.piece * 4) : 0);
  size_t g = 0;
  for (int64_t n : {f.piece, V % f.piece}) {
    if (!n || way != MEMORY) continue;
    const size_t b = ce_logits_part_bytes(M, K, n, dtype);
    g = b > g ? b : g;
  }
  f.total = f.gemm + up256(g);
  return f;
}

struct Bwd {
  int64_t piece;
  size_t factor, dl, x2, sum, logits, gemm, total;  // offsets after the rows
};
// Parts of dl; whether it is taken without g
int dl_parts(int64_t M, int dtype) { return dtype == MOE_BF16 && M <= 512 ? 2 : 1; }
bool dl_bare(int64_t M, int dtype) { return dtype == MOE_BF16 && dl_parts(M, dtype) == 1; }
// 256 MB of dl in bf16
int64_t bwd_piece(int64_t M, int64_t K, int64_t V) {
  const int64_t most = greatest(256, ((int64_t)1 << 27) / M / 256 * 256);
  return even_piece(V, least(most, weight_piece(K)));
}
int64_t bwd_ld(int64_t piece) { return (piece + 7) / 8 * 8; }
// Whether dl's rows may be filled up to 16-byte lines: the products that read it then take chunked loads, which
// look at no column past the end but those zeros (the loads of four elements of other tiles would pass the buffer's)
bool bwd_lines(int64_t M, int64_t K, int64_t V, int dtype) {
  const int64_t p = bwd_ld(bwd_piece(M, K, V)), most = (int64_t)1 << 30;
  M *= dl_parts(M, dtype);
  return dtype == MOE_BF16 && K % 8 == 0 && K <= (1 << 20) && p <= (1 << 20) && M * p < most && M * K < most && p * K < most;
}
Way bwd_way(int64_t M, int64_t K, int64_t V, int dtype, bool on_lines) {
  const int64_t p = bwd_piece(M, K, V);
  if (on_lines && bwd_lines(M, K, V, dtype) && ce_tiles(M, K, p)) return TILES;
  return staged(M, K, V, p, dtype) ? STAGED : MEMORY;
}
Bwd bwd_space(int64_t M, int64_t K, int64_t V, int dtype, Way way) {
  const size_t es = dtype == MOE_F32 ? 4 : 2;
  const int parts = dl_parts(M, dtype);
  Bwd w;
  w.piece = bwd_piece(M, K, V);
  const bool bare = dl_bare(M, dtype);
  w.factor = up256((size_t)M * sizeof(CeRow));
  w.dl = w.factor + (bare ? up256((size_t)(M + 1) * 4) : 0);
  w.x2 = w.dl + up256((size_t)parts * M * bwd_ld(w.piece) * es);
  w.sum = w.x2 + (parts == 2 || bare ? up256((size_t)parts * M * K * es) : 0);
  w.logits = w.sum + (parts == 2 || (w.piece < V && dtype == MOE_BF16) ? up256((size_t)parts * M * K * 4) : 0);
  w.gemm = w.logits + (way == MEMORY ? up256((size_t)M * w.piece * 4) : 0);
  size_t g = 0;
  for (int64_t n : {w.piece, V % w.piece}) {
    if (!n) continue;
    for (size_t b : {way == MEMORY ? ce_logits_part_bytes(M, K, n, dtype) : 0, ce_part_bytes(parts * M, K, n, dtype)})
      g = b > g ? b : g;
  }
  w.total = w.gemm + up256(g);
  return w;
}

int chunk_grid(int64_t M, int chunks) { return (int)least(M * chunks, kGrid); }

}  // namespace

// (x and W may lie off 16-byte lines: the larger of both ways)
size_t linear_ce_fwd_workspace(int64_t M, int64_t K, int64_t V, int dtype) {
  const size_t a = fwd_space(M, K, V, dtype, fwd_way(M, K, V, dtype, true)).total;
  const size_t b = fwd_space(M, K, V, dtype, fwd_way(M, K, V, dtype, false)).total;
  return a > b ? a : b;
}
size_t linear_ce_bwd_workspace(int64_t M, int64_t K, int64_t V, int dtype) {
  const size_t a = bwd_space(M, K, V, dtype, bwd_way(M, K, V, dtype, true)).total;
  const size_t b = bwd_space(M, K, V, dtype, bwd_way(M, K, V, dtype, false)).total;
  return a > b ? a : b;
}

hipError_t launch_linear_ce_fwd(const void *x, const void *W, const void *targets, bool wide, int64_t M, int64_t K, int64_t V,
                                float z, float *loss, float *lse, float *total, int dtype, void *ws, hipStream_t st) {
  CeArgs a{};
  a.targets = targets;
  a.wide = wide;
  a.V = V;
  hipError_t e = hipSuccess;
  if (M > 0) {
    const Way way = fwd_way(M, K, V, dtype, on_line(x) && on_line(W));
    const Fwd f = fwd_space(M, K, V, dtype, way);
    const size_t es = dtype == MOE_F32 ? 4 : 2;
    a.target_logit = (float *)ws;
    a.part = (float2 *)((char *)ws + f.part);
    float *logits = (float *)((char *)ws + f.logits);
    for (int64_t v = 0; v < V && e == hipSuccess; v += f.piece) {
      const int n = (int)least(f.piece, V - v);
      const char *w = (const char *)W + (size_t)v * K * es;
      a.col0 = v;
      if (way == TILES) {
        e = launch_ce_tiles(x, w, nullptr, a, (int)M, (int)K, n, (int)f.piece, st);
        a.part0 += (n + f.columns - 1) / f.columns;
        continue;
      }
      if (way == STAGED) {
        e = launch_ce_staged(x, w, nullptr, a, (int)M, (int)K, n, (int)f.piece, dtype, st);
        a.part0 += (n + 2 * f.columns - 1) / (2 * f.columns) * 2;
        continue;
      }
      e = launch_ce_logits(x, w, logits, (int)M, (int)K, n, dtype, (char *)ws + f.gemm, st);
      if (e != hipSuccess) break;
      const int chunks = (n + CHUNK - 1) / CHUNK;
      stats_kernel<<<chunk_grid(M, chunks), 256, 0, st>>>(logits, a, M, n, chunks);
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
    a.col0 = 0;
    if (M < 256) join_kernel<64><<<(int)((M + 3) / 4), 256, 0, st>>>(a, M, f.parts, z, loss, lse);
    else join_kernel<16><<<(int)((M + 15) / 16), 256, 0, st>>>(a, M, f.parts, z, loss, lse);
    e = hipGetLastError();
  }
  if (e == hipSuccess && total) {
    total_kernel<<<1, 1024, 0, st>>>(a, M, loss, total);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_linear_ce_bwd(const float *d_loss, int reduction, const float *total, const void *x, const void *W,
                                const void *targets, bool wide, const float *lse, int64_t M, int64_t K, int64_t V, float z,
                                void *dX, void *dW, int dtype, void *ws, hipStream_t st) {
  const size_t es = dtype == MOE_F32 ? 4 : 2;
  if (M == 0) return dW ? launch_fill_zero(dW, (size_t)V * K * es, nullptr, 0, st) : hipSuccess;
  const bool on = on_line(x) && on_line(W), lines = on && bwd_lines(M, K, V, dtype);
  const Way way = bwd_way(M, K, V, dtype, on);
  const Bwd b = bwd_space(M, K, V, dtype, way);
  CeArgs a{};
  a.targets = targets;
  a.wide = wide;
  a.V = V;
  a.rows = (const CeRow *)ws;
  void *dl = (char *)ws + b.dl;
  float *sum = dtype == MOE_F32 ? (float *)dX : (float *)((char *)ws + b.sum);
  float *logits = (float *)((char *)ws + b.logits);
  void *part = (char *)ws + b.gemm;
  const bool bare = dl_bare(M, dtype);
  float *factor = bare ? (float *)((char *)ws + b.factor) : nullptr;
  rows_kernel<<<(int)((M + 255) / 256), 256, 0, st>>>(a, M, d_loss, lse, total, reduction, z, (CeRow *)ws, factor);
  hipError_t e = hipGetLastError();
  const int parts = dl_parts(M, dtype), rows = (int)M * parts;
  const bool once = b.piece >= V && parts == 1;
  const void *xs = x;
  if (e == hipSuccess && dW && parts == 2) {
    xs = (char *)ws + b.x2;
    twice_kernel<<<(int)least((M * K + 255) / 256, 2048), 256, 0, st>>>((const bf16_t *)x, (bf16_t *)((char *)ws + b.x2), M * K);
    e = hipGetLastError();
  }
  if (e == hipSuccess && dW && bare && reduction == MOE_REDUCE_NONE) {
    bf16_t *y = (bf16_t *)((char *)ws + b.x2);
    xs = y;
    largest_kernel<<<(int)least((M + 255) / 256, 256), 256, 0, st>>>(factor, M);
    if (on_line(x) && K % 8 == 0)
      weigh_kernel<true><<<(int)least((M * K / 8 + 255) / 256, 8192), 256, 0, st>>>((const bf16_t *)x, y, factor, M, K);
    else
      weigh_kernel<false><<<(int)least((M * K + 255) / 256, 8192), 256, 0, st>>>((const bf16_t *)x, y, factor, M, K);
    e = hipGetLastError();
  }
  for (int64_t v = 0; v < V && e == hipSuccess; v += b.piece) {
    const int n = (int)least(b.piece, V - v);
    const char *w = (const char *)W + (size_t)v * K * es;
    a.col0 = v;
    a.ld = lines ? bwd_ld(n) : n;
    a.rest = parts == 2 ? (bf16_t *)dl + M * a.ld : nullptr;
    if (way == TILES) {
      e = launch_ce_tiles(x, w, dl, a, (int)M, (int)K, n, (int)b.piece, st);
    } else if (way == STAGED) {
      e = launch_ce_staged(x, w, dl, a, (int)M, (int)K, n, (int)b.piece, dtype, st);
    } else {
      e = launch_ce_logits(x, w, logits, (int)M, (int)K, n, dtype, part, st);
      if (e != hipSuccess) break;
      const int chunks = (n + CHUNK - 1) / CHUNK;
      if (dtype == MOE_F32) dl_kernel<float><<<chunk_grid(M, chunks), 256, 0, st>>>(logits, a, (float *)dl, M, n, chunks);
      else dl_kernel<bf16_t><<<chunk_grid(M, chunks), 256, 0, st>>>(logits, a, (bf16_t *)dl, M, n, chunks);
      e = hipGetLastError();
    }
    if (e == hipSuccess && dW)
      e = launch_ce_dw(dl, a.ld, xs, bare ? factor + M : nullptr, (char *)dW + (size_t)v * K * es, rows, (int)K, n, dtype, part, st);
    if (e == hipSuccess && dX)
      e = launch_ce_dx(dl, a.ld, w, v ? sum : nullptr, factor, once ? dX : sum, !once, rows, (int)K, n, dtype, part, st);
  }
  if (e == hipSuccess && dX && !once && dtype == MOE_BF16) {
    const int64_t n = M * K;
    if (parts == 2) add_kernel<<<(int)least((n + 255) / 256, 2048), 256, 0, st>>>(sum, (bf16_t *)dX, n);
    else round_kernel<<<(int)least((n + 1023) / 1024, 8192), 256, 0, st>>>(sum, (bf16_t *)dX, n, (uintptr_t)dX % 8 == 0);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace moe
