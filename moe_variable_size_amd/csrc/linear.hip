// Dense linear layer with bias, activation and residual in the product's epilogue, and its
// backward:  z = x W^T + b,  out = act(z) + r;  dz = d_out act'(z),  dx = dz W,  dW = dz^T x,
// db = sum of dz over the rows.
//
// All three products have one form, C[m, n] = sum_k A(m, k) B(n, k): for each operand either the
// reduction index (K-major) or the output index (MN-major) is contiguous in memory.
#include <atomic>
#include <type_traits>

#include "activation.hpp"
#include "common.hpp"
#include "cross_entropy.hpp"
#include "linear_plan.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

MOE_DEV float ldf(const float *p) { return *p; }
MOE_DEV float ldf(const bf16_t *p) { return bf16_to_f32(*p); }
MOE_DEV void stf(float *p, float v) { *p = v; }
MOE_DEV void stf(bf16_t *p, float v) { *p = __builtin_bit_cast(bf16_t, (__bf16)v); }

struct GemmArgs {
  const void *A, *B;
  const void *bias, *res;  // [N] operand type, [M, N] output type; NULL: none
  void *out, *z;           // [M, N]; z (operand type) NULL: not kept
  int M, N, K;
  int64_t lda, ldb;  // K-major: elements between rows; MN-major: between reduction rows
  bool vec;          // N a multiple of 8; out, z, residual and bias on 16-byte lines
  // without an activation, row m's products times factor[m * factor_step], before bias and residual; NULL: 1
  const float *factor = nullptr;
  int64_t factor_step = 0;
};

// buffer resource from wave-uniform values, in scalar registers
MOE_DEV __amdgpu_buffer_rsrc_t uniform_rsrc(const void *p, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return make_rsrc((const void *)(uintptr_t)(((uint64_t)hi << 32) | lo),
                   __builtin_amdgcn_readfirstlane(bytes));
}

// ---- epilogue -----------------------------------------------------------------
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
MOE_DEV f32x4 get4(const float *p) { return *(const f32x4 *)p; }
MOE_DEV f32x4 get4(const bf16_t *p) {
  const bf16x4_t b = *(const bf16x4_t *)p;
  return f32x4{(float)b[0], (float)b[1], (float)b[2], (float)b[3]};
}
MOE_DEV void put8(float *p, const f32x4 (&v)[2]) {
  *(f32x4 *)p = v[0];
  *(f32x4 *)(p + 4) = v[1];
}
MOE_DEV void put8(bf16_t *p, const f32x4 (&v)[2]) {
  *(bf16x8_t *)p = bf16x8_t{(__bf16)v[0][0], (__bf16)v[0][1], (__bf16)v[0][2], (__bf16)v[0][3],
                            (__bf16)v[1][0], (__bf16)v[1][1], (__bf16)v[1][2], (__bf16)v[1][3]};
}
// from z = product + bias: keep z, out = act(z) + residual, for 8 columns on a 16-byte line or one
template <typename T, typename To, int ACT>
MOE_DEV void finish8(const GemmArgs &p, f32x4 (&v)[2], int64_t at) {
  f32x4 r[2] = {};
  if (p.res) {
    r[0] = get4((const To *)p.res + at);
    r[1] = get4((const To *)p.res + at + 4);
  }
  if (p.z) put8((T *)p.z + at, v);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[h][i] = act_fwd<ACT>(v[h][i]) + r[h][i];
  put8((To *)p.out + at, v);
}
template <int ACT>
MOE_DEV float factor_of(const GemmArgs &p, int64_t m) {
  return ACT == MOE_ACT_NONE && p.factor ? p.factor[m * p.factor_step] : 1.f;
}
template <typename T, typename To, int ACT>
MOE_DEV void finish1(const GemmArgs &p, float v, int64_t at) {
  if (p.z) stf((T *)p.z + at, v);
  v = act_fwd<ACT>(v);
  if (p.res) v += ldf((const To *)p.res + at);
  stf((To *)p.out + at, v);
}

// out from the partial products of all ranges, added in order
template <typename T, typename To, int ACT>
__global__ __launch_bounds__(256) void join_kernel(GemmArgs p, const float *part, int splits) {
  const int64_t total = (int64_t)p.M * p.N, step = (int64_t)gridDim.x * 256;
  const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (p.vec) {
    for (int64_t at = i0 * 8; at < total; at += step * 8) {
      f32x4 v[2] = {get4(part + at), get4(part + at + 4)};
#pragma unroll 4
      for (int s = 1; s < splits; ++s) {
        v[0] += get4(part + s * total + at);
        v[1] += get4(part + s * total + at + 4);
      }
      if (ACT == MOE_ACT_NONE && p.factor) {
        const float f = factor_of<ACT>(p, at / p.N);
        v[0] *= f;
        v[1] *= f;
      }
      if (p.bias) {
        const int n = (int)(at % p.N);
        v[0] += get4((const T *)p.bias + n);
        v[1] += get4((const T *)p.bias + n + 4);
      }
      finish8<T, To, ACT>(p, v, at);
    }
  } else {
    for (int64_t at = i0; at < total; at += step) {
      float v = part[at];
      for (int s = 1; s < splits; ++s) v += part[s * total + at];
      if (ACT == MOE_ACT_NONE && p.factor) v *= factor_of<ACT>(p, at / p.N);
      if (p.bias) v += ldf((const T *)p.bias + at % p.N);
      finish1<T, To, ACT>(p, v, at);
    }
  }
}

// The cross entropy's epilogues (cross_entropy.hip), in the place of an activation: logits l = x W^T stay in the
// accumulators.  The forward leaves the largest value and the sum of exponentials of a row's columns in a tile (or a wave
// of it), and the target's logit; the backward leaves dl.  The products bound both: 8192 x 4096 x 65536 in bf16 takes 3.08
// ms with the statistics (1.43 PFLOP/s) and 3.32 with the gradient (1.32), its bf16 stores among them.
constexpr int kCeStats = 16, kCeGrad = 17;

// ---- staged tiles: any alignment and size ------------------------------------
// 64 S x 64 S outputs per 4 waves (2 x 2, S x S blocks of 32 x 32 each), 32 reduction elements per
// step through registers into LDS, element loads with bounds checks.  fp32 multiplies on the
// matrix cores' fp32 instructions (exact products, fp32 sums; 64 clocks per 2 reduction elements of
// a block, so the loads hide behind them); a reduction may be cut into ranges as below.  fp32 4096^3:
// 1068 us (129 TFLOP/s of the instructions' 157).  bf16 4096 x 4095 x 4095, element by element: 282 us (487
// TFLOP/s), 4096 x 4100 x 4096, four by four: 241 (571).
constexpr int SNT = 256;

// LDS layout of a 64 S x 32 operand tile: [row][reduction], 16-byte rows whose 16-byte reads spread over
// the banks; fp32 that is MN-major in memory [reduction][row], so that its loads are stored as they
// come (scattered, 16 lanes met on one bank: the backward of 4096^3 in 128 x 128 tiles took 2508
// us instead of 2236), with a pitch
// that puts the two halves of a wave, four reduction elements apart, on different banks.
template <typename T, int S, bool KMAJ>
struct Tile {
  static constexpr bool BYK = sizeof(T) == 4 && !KMAJ;
  static constexpr int PITCH = BYK ? 64 * S + 8 : sizeof(T) == 2 ? SBK + 8 : SBK + 4;
  static constexpr int SIZE = PITCH * (BYK ? SBK : 64 * S);
  MOE_DEV static int at(int r, int k) { return BYK ? k * PITCH + r : r * PITCH + k; }
};

// Thread t brings 8 S elements of the tile, in runs of E that are contiguous in memory (E = 4 where rows
// are on lines of four elements, else 1; bf16 that is MN-major always 1): the first element of run i
template <int S, int E, bool KMAJ>
MOE_DEV void stage_at(int i, int &r, int &k) {
  constexpr int RUNS = (KMAJ ? SBK : 64 * S) / E;  // per memory row
  const int t = threadIdx.x, c = t % RUNS * E, o = i * (SNT / RUNS) + t / RUNS;
  r = KMAJ ? o : c;
  k = KMAJ ? c : o;
}
template <typename T, int E>
MOE_DEV void buf_load(__amdgpu_buffer_rsrc_t r, uint32_t off, T *v) {
  if constexpr (sizeof(T) * E == 16) {
    const f32x4 x = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x[i];
  } else if constexpr (sizeof(T) * E == 8) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (T)(x[i / 2] >> (16 * (i & 1)));
  } else if constexpr (sizeof(T) == 4) {
    *v = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
  } else {
    *v = __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
  }
}
// p: the operand at the tile's first row (column) and the range's reduction element k0; rows: of the
// operand from there on.  Rows past the end are past the buffer's range; the other direction is checked.
template <typename T, int S, int E, bool KMAJ>
MOE_DEV void stage_load(const T *p, int64_t ld, int rows, int left, T (&v)[8 * S]) {
  const uint32_t es = sizeof(T);
  const int n = KMAJ ? min(rows, 64 * S) : min(left, SBK);  // memory rows of the tile
  const __amdgpu_buffer_rsrc_t r = uniform_rsrc(p, n > 0 ? ((uint32_t)(n - 1) * (uint32_t)ld + (KMAJ ? left : rows)) * es : 0u);
#pragma unroll
  for (int i = 0; i < 8 * S / E; ++i) {
    int row, k;
    stage_at<S, E, KMAJ>(i, row, k);
    const bool ok = KMAJ ? k < left : row < rows;
    const uint32_t off = (uint32_t)(KMAJ ? row : k) * (uint32_t)ld + (KMAJ ? k : row);
    buf_load<T, E>(r, ok ? off * es : kOobOffset, v + i * E);
  }
}
template <typename T, int S, int E, bool KMAJ>
MOE_DEV void stage_store(T *lds, const T (&v)[8 * S]) {
  using L = Tile<T, S, KMAJ>;
  typedef T run_t __attribute__((ext_vector_type(E)));
#pragma unroll
  for (int i = 0; i < 8 * S / E; ++i) {
    int r, k;
    stage_at<S, E, KMAJ>(i, r, k);
    if constexpr (E == 4)  // (KMAJ or BYK: the run is contiguous in LDS too)
      *(run_t *)&lds[L::at(r, k)] = run_t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    else
      lds[L::at(r, k)] = v[i];
  }
}
// elements k .. k + 3 of row r (fp32)
template <int S, bool KMAJ>
MOE_DEV f32x4 stage_four(const float *lds, int r, int k) {
  using L = Tile<float, S, KMAJ>;
  if constexpr (L::BYK) {
    return f32x4{lds[L::at(r, k)], lds[L::at(r, k + 1)], lds[L::at(r, k + 2)], lds[L::at(r, k + 3)]};
  } else {
    return *(const f32x4 *)&lds[L::at(r, k)];
  }
}

// row of register i of a 32 x 32 accumulator
MOE_DEV int acc_row(int i, int lane) { return ((i >> 2) << 3) + ((lane >> 5) << 2) + (i & 3); }

// f over the 32 lanes of a half wave: within 16 by lane permutations of the operand (neighbours, pairs, then halves and
// rows mirrored, once their members are alike), the last step through LDS's crossbar.
template <class F>
MOE_DEV float over_half(float v, F &&f) {
  auto other = [&](auto ctrl) __attribute__((always_inline)) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  v = f(v, other(std::integral_constant<int, 0xB1>()));   // quad_perm 1 0 3 2
  v = f(v, other(std::integral_constant<int, 0x4E>()));   // quad_perm 2 3 0 1
  v = f(v, other(std::integral_constant<int, 0x141>()));  // row_half_mirror
  v = f(v, other(std::integral_constant<int, 0x140>()));  // row_mirror
  return f(v, __shfl_xor(v, 16, 64));
}

// What becomes of a tile's sums: a wave's S x S blocks at row m0 + wm, column n0 + wn
template <typename T, typename To, int S, int ACT>
MOE_DEV void staged_out(const GemmArgs &p, int splits, int split, float *part, const CeArgs &ce, f32x16 (&acc)[S][S], int m0, int n0,
                        int wm, int wn) {
  const int lane = threadIdx.x & 63;
  if constexpr (ACT == kCeStats) {
    const int n = n0 + wn + (lane & 31);
    float2 *out = ce.part + (int64_t)(ce.part0 + (n0 + wn) / (32 * S)) * p.M;
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int m = m0 + wm + i * 32 + acc_row(e, lane), t = m < p.M ? ce_target(ce, m) : -1;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int j = 0; j < S; ++j) {
          if (t >= 0 && t == n + j * 32 && t < p.N) ce.target_logit[m] = acc[i][j][e];
          if (n + j * 32 >= p.N) acc[i][j][e] = -INFINITY;
          top = fmaxf(top, acc[i][j][e]);
        }
        top = over_half(top, [](float a, float b) __attribute__((always_inline)) { return fmaxf(a, b); });
        const float base = ce_base(top);
#pragma unroll
        for (int j = 0; j < S; ++j) sum += ce_exp<T>(acc[i][j][e] - base);
        sum = over_half(sum, [](float a, float b) __attribute__((always_inline)) { return a + b; });
        if ((lane & 31) == 0 && m < p.M) out[m] = float2{top, sum};
      }
    return;
  }
  if constexpr (ACT == kCeGrad) {
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int m = m0 + wm + i * 32 + acc_row(e, lane);
        if (m >= p.M) continue;
        const CeRow row = ce.rows[m];
#pragma unroll
        for (int j = 0; j < S; ++j) {
          const int n = n0 + wn + j * 32 + (lane & 31);
          if (n >= ce.ld) continue;
          const float d = n < p.N ? ce_dl<T>(row, acc[i][j][e], ce.col0 + n) : 0.f;
          stf((To *)p.out + (int64_t)m * ce.ld + n, d);
          if (sizeof(T) == 2 && ce.rest) stf(ce.rest + (int64_t)m * ce.ld + n, d - (float)(__bf16)d);
        }
      }
    return;
  }
  if (splits > 1) part += (int64_t)split * p.M * p.N;
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const int n = n0 + wn + j * 32 + (lane & 31);
    if (n >= p.N) continue;
    const float b = p.bias ? ldf((const T *)p.bias + n) : 0.f;
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int m = m0 + wm + i * 32 + acc_row(e, lane);
        if (m >= p.M) continue;
        const int64_t at = (int64_t)m * p.N + n;
        if (splits > 1)
          part[at] = acc[i][j][e];
        else
          finish1<T, To, ACT>(p, acc[i][j][e] * factor_of<ACT>(p, m) + b, at);
      }
  }
}

// splits > 1: range blockIdx / tiles of the reduction, fp32 products to part [splits][M][N]
template <typename T, typename To, int S, int E, bool AK, bool BKM, int ACT>
__global__ __launch_bounds__(SNT) void staged_gemm(GemmArgs p, int splits, float *part, CeArgs ce) {
  using LA = Tile<T, S, AK>;
  using LB = Tile<T, S, BKM>;
  constexpr int TS = 64 * S, EA = sizeof(T) == 4 || AK ? E : 1, EB = sizeof(T) == 4 || BKM ? E : 1;
  __shared__ __align__(16) T As[LA::SIZE], Bs[LB::SIZE];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int wm = (wid >> 1) * 32 * S, wn = (wid & 1) * 32 * S;
  const int tn = (p.N + TS - 1) / TS, tiles = tn * ((p.M + TS - 1) / TS);
  const int split = blockIdx.x / tiles, tile = blockIdx.x - split * tiles;
  const int m0 = tile / tn * TS, n0 = tile % tn * TS;
  const int steps = (p.K + SBK - 1) / SBK;
  const int kb = (int)((int64_t)steps * split / splits) * SBK;
  const int ke = min(p.K, (int)((int64_t)steps * (split + 1) / splits) * SBK);
  f32x16 acc[S][S] = {};
  T va[8 * S], vb[8 * S];
  auto load = [&](int k0) __attribute__((always_inline)) {
    const T *a = (const T *)p.A + (AK ? (int64_t)m0 * p.lda + k0 : (int64_t)k0 * p.lda + m0);
    const T *b = (const T *)p.B + (BKM ? (int64_t)n0 * p.ldb + k0 : (int64_t)k0 * p.ldb + n0);
    stage_load<T, S, EA, AK>(a, p.lda, p.M - m0, ke - k0, va);
    stage_load<T, S, EB, BKM>(b, p.ldb, p.N - n0, ke - k0, vb);
  };
  load(kb);
  for (int k0 = kb; k0 < ke; k0 += SBK) {
    __syncthreads();
    stage_store<T, S, EA, AK>(As, va);
    stage_store<T, S, EB, BKM>(Bs, vb);
    __syncthreads();
    if (k0 + SBK < ke) load(k0 + SBK);
    const int r = lane & 31, h = lane >> 5;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int s = 0; s < SBK / 16; ++s) {
        bf16x8_t a[S], b[S];
#pragma unroll
        for (int i = 0; i < S; ++i) {
          a[i] = *(const bf16x8_t *)&As[LA::at(wm + i * 32 + r, s * 16 + h * 8)];
          b[i] = *(const bf16x8_t *)&Bs[LB::at(wn + i * 32 + r, s * 16 + h * 8)];
        }
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int j = 0; j < S; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
      }
    } else {
      // four reduction elements per lane and read: element e of both halves of the wave is one
      // 32 x 32 x 2 product (the same two reduction indices in both operands)
#pragma unroll
      for (int s = 0; s < SBK / 8; ++s) {
        f32x4 a[S], b[S];
#pragma unroll
        for (int i = 0; i < S; ++i) {
          a[i] = stage_four<S, AK>(As, wm + i * 32 + r, s * 8 + h * 4);
          b[i] = stage_four<S, BKM>(Bs, wn + i * 32 + r, s * 8 + h * 4);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < S; ++i)
#pragma unroll
            for (int j = 0; j < S; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i][e], b[j][e], acc[i][j], 0, 0, 0);
      }
    }
  }
  staged_out<T, To, S, ACT>(p, splits, split, part, ce, acc, m0, n0, wm, wn);
}

// ---- pipelined tiles: bf16 rows on 16-byte lines -------------------------------
// BM x BN outputs per 8 waves (WGM x WGN), one workgroup per tile and reduction range.
//
// A stage is 64 reduction elements of both operands, each in two halves (A0 A1 B0 B1: the rows
// of every wave's first or second half), double buffered in LDS and filled by direct global->LDS
// loads.  A wave works through the four quarters of its outputs per stage,
//   (A0 B0) (A0 B1) (A1 B1) (A1 B0),
// each a memory part (operand reads of the quarter, one half of a coming stage issued) and a
// multiply part, with a barrier after each.  The waves of the second half of the workgroup run
// one part behind, so on every SIMD one wave multiplies while the other loads.
//
// Order of issue, one half per quarter: B1 and A1 of the next stage, A0 and B0 of the one after.
// A half goes into the place of one that was read two or more quarters before.  The multiply part
// of a quarter consumes the quarter's reads (A0's first step is read a quarter early and consumed
// in the next), and both groups of waves have ended that part before either is two quarters on, so
// no read of the overwritten half is outstanding.  A half is waited for one quarter before its
// first read, when four younger ones are in flight.  (Reads waited for in the memory part instead
// allow one quarter more of lead: the same time within 2 %.)
//
// Measured: 8192^3 723-789 us by card (1390-1520 TFLOP/s), 8192 x 4096 x 4096 198 us (1390).  Without the loads
// (timing only) 8192^3 takes 629 us, without the operand reads 695: the loads, and a clock near
// 1.9 GHz under this load, are the bound; touching coming stages' lines ahead made it slower.
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
#define LDS_AS __attribute__((address_space(3)))

// 16 bytes per lane from rsrc + voff to LDS byte address lds + 16 * lane (lds wave-uniform);
// zeros where voff is out of the buffer
MOE_DEV void dma16(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, uint32_t lds) {
  const uint32_t m0v = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(m0v), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
#define LIN_FENCE() __builtin_amdgcn_sched_barrier(0)

// One half operand tile: W output rows (or columns) x 64 reduction elements, 128 W bytes of LDS.
// K-major: [W][64]: 16-byte chunk c (0..7) of row r at chunk place c ^ ((r >> 1) & 7): the 16
// rows of a fragment read fall on 16 different 16-byte bank groups (64 banks, two rows a line).
// MN-major: [64][W]: chunk c of reduction row k at place c ^ 2 f(k), where f(k) tells apart the 8
// rows k, k+1, k+2, k+3, k+8 .. k+11 that 32 lanes of a transposing read touch (32 bytes each).
template <int W, bool KMAJ>
struct HalfTile {
  static constexpr int PER = W * 128 / 8192;  // 16-byte loads per thread (512 threads)
  static constexpr int ROWB = KMAJ ? 128 : 2 * W;
  static constexpr int CPR = ROWB / 16;       // chunks per LDS row
  MOE_DEV static int f(int k) {
    if constexpr (W >= 128) return (k & 3) | (((k >> 3) & 1) << 2);
    return ((k >> 1) & 1) | (((k >> 3) & 1) << 1);
  }
  MOE_DEV static int place(int row, int c) {
    return KMAJ ? (c ^ ((row >> 1) & 7)) : (c ^ (2 * f(row)));
  }
  // A thread's loads of one half are 64 rows (K-major) or 512 / CPR reduction rows apart, which
  // moves neither its chunk nor the place's XOR, and the second half W rows (columns) on: one base
  // offset, and per half the first reduction element (kk; out of every range where the lane's
  // columns are past the operand's.  Rows past a K-major operand are past its buffer's end.)
  uint32_t base;
  int kk[2];
  static constexpr int RSTEP = 512 / CPR;
  // r0: first row (column) of the tile in the operand, of `rows`; ld in elements
  MOE_DEV void setup(int r0, int rows, int64_t ld) {
    const int row = threadIdx.x / CPR, c = place(row, threadIdx.x % CPR);  // (XOR: its own inverse)
    base = KMAJ ? (uint32_t)(((r0 + row) * ld + 8 * c) * 2) : (uint32_t)((row * ld + r0 + 8 * c) * 2);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      kk[h] = KMAJ ? 8 * c : r0 + h * W + 8 * c < rows ? row : INT32_MAX;
  }
  // half h of stage kt of a reduction that ends at K
  MOE_DEV void issue(__amdgpu_buffer_rsrc_t rs, int h, int kt, int K, uint32_t ld2, uint32_t lds) {
    const uint32_t at = KMAJ ? kt * 128 + h * (W * ld2) : kt * (PBK * ld2) + h * (2 * W);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool in = kk[h] < K - kt * PBK - (KMAJ ? 0 : i * RSTEP);
      dma16(rs, in ? base + (at + i * (RSTEP * ld2)) : kOobOffset, lds + i * 8192);
    }
  }
};

// fragment of 16 rows x 32 reduction elements at rows r0 .. of a half tile: lane l holds row
// l & 15, elements 8 (l >> 4) .. +7 of step s
template <int W, bool KMAJ>
MOE_DEV bf16x8_t frag(const char *half, int r0, int s, int lane) {
  using H = HalfTile<W, KMAJ>;
  if constexpr (KMAJ) {
    const int r = r0 + (lane & 15);
    return *(const bf16x8_t *)(half + r * H::ROWB + (H::place(r, 4 * s + (lane >> 4)) << 4));
  } else {
    // lane j of 16: address of 4 columns of reduction row j >> 2; receives 4 rows of column j
    const int j = lane & 15, k = 32 * s + 8 * (lane >> 4) + (j >> 2);
    const int col = r0 + 4 * (j & 3);
    LDS_AS i16x4 *p0 = (LDS_AS i16x4 *)(LDS_AS char *)(half + k * H::ROWB + (H::place(k, col >> 3) << 4) + (col & 7) * 2);
    LDS_AS i16x4 *p1 = (LDS_AS i16x4 *)((LDS_AS char *)p0 + 4 * H::ROWB);  // f(k + 4) = f(k)
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p0);
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p1);
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

// tile of workgroup b: the hardware deals workgroups to the 8 XCDs in turn; each XCD (one L2)
// takes a run of tiles that walks bands of 8 row blocks
MOE_DEV void tile_of(int b, int total, int tm, int tn, int &mb, int &nb) {
  const int x = b & 7, q = total >> 3, r = total & 7;
  const int t = x * q + min(x, r) + (b >> 3);
  const int band = 8 * tn, g = t / band, rows = min(8, tm - 8 * g);
  const int u = t - g * band;
  mb = 8 * g + u % rows;
  nb = u / rows;
}

// ---- fp32 in three parts of bf16 -----------------------------------------------------
// The cross entropy's fp32 products.  With a1 = bf16(a), a2 = bf16(a - a1) and a3 = a - a1 - a2, all exact (3 x 8 bits),
//     a b = a1 b1 + (a1 b2 + a2 b1) + (a1 b3 + a2 b2 + a3 b1) + what is left out,
// a2 b3 + a3 b2 + a3 b3, at most 2^-23 |a b| (|a2| <= 2^-8 |a|, |a3| <= 2^-16 |a|): two half steps of fp32.  Six products of
// bf16 take 3 / 8 of the matrix cores' time for one of fp32, and add up in fp32 in K / 16 steps each instead of K / 2.
// (What is not finite, or above 3.39e38, makes its row's or column's sums NaN.)  4096^3: 680 us (1.21 PFLOP/s of bf16, the
// clock at 1.9 GHz for the power it takes); by fp32 instructions 1000, at 90 % of what they can do.
//
//
// Tiles of 64 S x 64 S per 4 waves, steps of 16 reduction elements.  The parts are made once per element, on the way from
// registers to LDS, which holds them in three planes [row][reduction], or [reduction][row] where memory has it so, for
// transposing reads.  While a step is multiplied, the next one is split into the other half of LDS and the one after is
// loaded, so there is one barrier per step and a load has a whole step's time.
//
// Loads are runs of four at any alignment, none behind a branch.  A run that would end past its row is taken as the row's
// last four elements instead and moved into place before the step that splits it.  (Rows have at least four.)
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
MOE_DEV uint32_t pack2(float a, float b) { return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)a, (__bf16)b}); }

constexpr int BK = 16;
template <int S, bool KMAJ>
struct Fine {
  static constexpr int RUNS = S;  // of a thread
  static constexpr int PER = (KMAJ ? BK : 64 * S) / 4;
  static constexpr int PITCH = KMAJ ? BK + 8 : 64 * S + 32;
  static constexpr int PLANE = PITCH * (KMAJ ? 64 * S : BK);
  MOE_DEV static int at(int r, int k) { return KMAJ ? r * PITCH + k : k * PITCH + r; }

  const float *p;   // the operand; K-major: from the tile's first row on
  int64_t ld;
  int rows, ke;     // K-major: rows from there; MN-major: all of them
  uint32_t off[RUNS];
  int first, shift;  // first row (reduction element) of the lane's runs; how far those past the end are moved
  bool over;

  MOE_DEV void setup(const void *op, int64_t l, int r0, int total, int end) {
    ld = l;
    ke = end;
    first = threadIdx.x % PER * 4;
    const int o = threadIdx.x / PER;
    if constexpr (KMAJ) {
      p = (const float *)op + r0 * l;
      rows = min(total - r0, 64 * S);
#pragma unroll
      for (int i = 0; i < RUNS; ++i) {
        const int r = o + i * (SNT / PER);
        off[i] = r < rows ? ((uint32_t)r * (uint32_t)ld + first) * 4 : kOobOffset;
      }
      shift = 0;
    } else {
      p = (const float *)op;
      rows = total;
      const int left = total - r0;
      shift = left < 64 * S ? -left & 3 : 0;
      over = first < left && first + 4 > left;
#pragma unroll
      for (int i = 0; i < RUNS; ++i) {
        const int k = o + i * (SNT / PER);
        off[i] = first < left ? ((uint32_t)k * (uint32_t)ld + r0 + first - (over ? shift : 0)) * 4 : kOobOffset;
      }
    }
  }
  // elements k0 .. k0 + BK - 1 (zeros from ke on)
  MOE_DEV void load(int k0, float (&v)[4 * RUNS]) {
    const int left = ke - k0;
    if constexpr (KMAJ) {
      const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(p, ((uint32_t)(rows - 1) * (uint32_t)ld + ke) * 4);
      const uint32_t at = (uint32_t)(first + 4 > left ? k0 - (-left & 3) : k0) * 4;
#pragma unroll
      for (int i = 0; i < RUNS; ++i) buf_load<float, 4>(rs, first < left ? off[i] + at : kOobOffset, v + 4 * i);
    } else {
      const __amdgpu_buffer_rsrc_t rs = uniform_rsrc(p + k0 * ld, left > 0 ? ((uint32_t)(min(left, BK) - 1) * (uint32_t)ld + rows) * 4 : 0u);
#pragma unroll
      for (int i = 0; i < RUNS; ++i) buf_load<float, 4>(rs, off[i], v + 4 * i);
    }
  }
  // runs that were taken from before their place (as loaded for k0)
  MOE_DEV void settle(int k0, float (&v)[4 * RUNS]) {
    const int left = ke - k0, n = KMAJ ? (left < BK ? -left & 3 : 0) : shift;
    const bool mine = KMAJ ? first < left && first + 4 > left : over;
    for (int t = 0; t < n; ++t)
#pragma unroll
      for (int i = 0; i < RUNS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * i + j] = !mine ? v[4 * i + j] : j < 3 ? v[4 * i + j + 1] : 0.f;
  }
  MOE_DEV void store(bf16_t *lds, const float (&v)[4 * RUNS]) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
      const int o = threadIdx.x / PER + i * (SNT / PER);
      float a[4] = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        const u32x2 w = {pack2(a[0], a[1]), pack2(a[2], a[3])};
        *(u32x2 *)&lds[t * PLANE + (KMAJ ? at(o, first) : at(first, o))] = w;
        if (t == 2) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] -= __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
      }
    }
  }
  // 32 rows at r0 of the step: lane l holds row l & 31, elements 8 (l >> 5) .. +7
  MOE_DEV static bf16x8_t frag(const bf16_t *plane, int r0) {
    const int lane = threadIdx.x & 63;
    if constexpr (KMAJ) {
      return *(const bf16x8_t *)&plane[at(r0 + (lane & 31), 8 * (lane >> 5))];
    } else {  // (as frag of the pipelined tiles, 16 columns per 16 lanes)
      const int j = lane & 15, k = 8 * (lane >> 5) + (j >> 2), col = r0 + (lane & 16) + 4 * (j & 3);
      LDS_AS i16x4 *p0 = (LDS_AS i16x4 *)(LDS_AS char *)(char *)&plane[at(col, k)];
      LDS_AS i16x4 *p1 = (LDS_AS i16x4 *)((LDS_AS char *)p0 + 8 * PITCH);
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p0);
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p1);
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};
template <int S, bool AK, bool BKM, int ACT>
__global__ __launch_bounds__(SNT, 2) void fine_gemm(GemmArgs p, int splits, float *part, CeArgs ce) {
  using FA = Fine<S, AK>;
  using FB = Fine<S, BKM>;
  __shared__ __align__(16) bf16_t As[2][3 * FA::PLANE], Bs[2][3 * FB::PLANE];
  const int wid = threadIdx.x >> 6, wm = (wid >> 1) * 32 * S, wn = (wid & 1) * 32 * S;
  const int tm = (p.M + 64 * S - 1) / (64 * S), tn = (p.N + 64 * S - 1) / (64 * S), split = blockIdx.x / (tm * tn);
  int mb, nb;
  tile_of(blockIdx.x - split * (tm * tn), tm * tn, tm, tn, mb, nb);
  const int m0 = mb * 64 * S, n0 = nb * 64 * S;
  const int steps = (p.K + BK - 1) / BK;
  const int ub = (int)((int64_t)steps * split / splits), ue = (int)((int64_t)steps * (split + 1) / splits);
  FA fa;
  FB fb;
  fa.setup(p.A, p.lda, m0, p.M, min(p.K, ue * BK));
  fb.setup(p.B, p.ldb, n0, p.N, min(p.K, ue * BK));
  f32x16 acc[S][S] = {};
  float va[2][4 * FA::RUNS], vb[2][4 * FB::RUNS];
  // step u out of half H, the next one into the other
  auto step = [&](int u, auto half) __attribute__((always_inline)) {
    constexpr int H = decltype(half)::value;
    fa.load((u + 2) * BK, va[H]);
    fb.load((u + 2) * BK, vb[H]);
    fa.settle((u + 1) * BK, va[1 - H]);
    fb.settle((u + 1) * BK, vb[1 - H]);
    bf16x8_t a[S][3], b[S][3];
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        a[i][t] = FA::frag(As[H] + t * FA::PLANE, wm + i * 32);
        b[i][t] = FB::frag(Bs[H] + t * FB::PLANE, wn + i * 32);
      }
#pragma unroll
    for (int sum = 2; sum >= 0; --sum)  // (small ones first)
#pragma unroll
      for (int t = 0; t <= sum; ++t)
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int j = 0; j < S; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i][t], b[j][sum - t], acc[i][j], 0, 0, 0);
    fa.store(As[1 - H], va[1 - H]);
    fb.store(Bs[1 - H], vb[1 - H]);
    __syncthreads();
  };
  fa.load(ub * BK, va[0]);
  fb.load(ub * BK, vb[0]);
  fa.load((ub + 1) * BK, va[1]);
  fb.load((ub + 1) * BK, vb[1]);
  fa.settle(ub * BK, va[0]);
  fb.settle(ub * BK, vb[0]);
  fa.store(As[0], va[0]);
  fb.store(Bs[0], vb[0]);
  __syncthreads();
  for (int u = ub; u < ue; u += 2) {
    step(u, std::integral_constant<int, 0>());
    if (u + 1 < ue) step(u + 1, std::integral_constant<int, 1>());
  }
  staged_out<float, float, S, ACT>(p, splits, split, part, ce, acc, m0, n0, wm, wn);
}

struct PipeArgs {
  GemmArgs g;
  uint32_t a_bytes, b_bytes;
  int tm, tn, splits;  // tiles; reduction ranges (> 1: fp32 partial products to part)
  float *part;         // [splits][M][N]
  CeArgs ce;           // the cross entropy's epilogues alone
};

// Epilogue of a workgroup's tile, half the rows at a time through LDS as fp32 [WA][BN], so that each
// row's columns are read and written in whole lines (16 bytes of bf16 per lane): stored from the
// accumulators' own layout, 32 bytes a row, the forward of 8192 x 4096 x 4096 with gelu, residual and
// kept z took 324 us instead of 236.  16-byte chunk c of row r sits at place c ^ (r & 15): the 16 rows
// of an accumulator store fall on 16 bank groups.  Every wave is done with the LDS when this begins.
template <int HM, int HN, int WGM, int WGN, typename To, int ACT>
MOE_DEV void tile_epilogue(const PipeArgs &q, char *lds, const f32x4 (&acc)[2][2][HM][HN], int wm, int wn,
                           int m0, int n0, int split) {
  constexpr int BM = 32 * HM * WGM, BN = 32 * HN * WGN, WA = BM / 2, WB = BN / 2;
  const GemmArgs &p = q.g;
  const int lane = threadIdx.x & 63;
  auto chunk = [&](int r, int c) __attribute__((always_inline)) {
    return (f32x4 *)(lds + r * (BN * 4) + ((c ^ (r & 15)) << 4));
  };
  constexpr int LPR = BN / 8, RPP = 512 / LPR;  // lanes per row, rows per pass of the workgroup
  const bool part = q.splits > 1;
  float *const pout = q.part + (int64_t)split * p.M * p.N;
#pragma unroll
  for (int mh = 0; mh < 2; ++mh) {
    __syncthreads();
    // lane l of a 16 x 16 block: row l & 15, columns 4 (l >> 4) .. +3
#pragma unroll
    for (int i = 0; i < HM; ++i)
#pragma unroll
      for (int nh = 0; nh < 2; ++nh)
#pragma unroll
        for (int j = 0; j < HN; ++j)
          *chunk(wm * 16 * HM + i * 16 + (lane & 15),
                 (nh * WB + wn * 16 * HN + j * 16) / 4 + (lane >> 4)) = acc[mh][nh][i][j];
    __syncthreads();
    const int r0 = threadIdx.x / LPR, c0 = (threadIdx.x % LPR) * 8;
    if (p.vec) {
      if (n0 + c0 >= p.N) continue;
      f32x4 b[2] = {};
      if (p.bias && !part) {
        b[0] = get4((const bf16_t *)p.bias + n0 + c0);
        b[1] = get4((const bf16_t *)p.bias + n0 + c0 + 4);
      }
#pragma unroll 4
      for (int r = r0; r < WA; r += RPP) {
        const int m = m0 + mh * WA + r;
        if (m >= p.M) break;
        const int64_t at = (int64_t)m * p.N + n0 + c0;
        f32x4 v[2] = {*chunk(r, c0 / 4), *chunk(r, c0 / 4 + 1)};
        if (part) {
          put8(pout + at, v);
          continue;
        }
        if (ACT == MOE_ACT_NONE && p.factor) {
          const float f = factor_of<ACT>(p, m);
          v[0] *= f;
          v[1] *= f;
        }
        v[0] += b[0];
        v[1] += b[1];
        finish8<bf16_t, To, ACT>(p, v, at);
      }
    } else {
      for (int r = r0; r < WA; r += RPP) {
        const int m = m0 + mh * WA + r;
        if (m >= p.M) break;
        for (int c = threadIdx.x % LPR; c < BN && n0 + c < p.N; c += LPR) {
          const int64_t at = (int64_t)m * p.N + n0 + c;
          const float v = ((const float *)chunk(r, c >> 2))[c & 3];
          if (part)
            pout[at] = v;
          else
            finish1<bf16_t, To, ACT>(p, v * factor_of<ACT>(p, m) + (p.bias ? ldf((const bf16_t *)p.bias + n0 + c) : 0.f), at);
        }
      }
    }
  }
}

// ---- the cross entropy's epilogues of these tiles ----------------------------------
// A lane holds 4 HN columns per half of 2 HM rows: its own maximum and sum first, then the 4 lanes of a row,
// then the WGN waves through LDS.
template <int HM, int HN, int WGM, int WGN>
MOE_DEV void ce_stats(const PipeArgs &q, char *lds, f32x4 (&acc)[2][2][HM][HN], int wm, int wn, int m0, int n0,
                      int nb) {
  constexpr int BM = 32 * HM * WGM, WA = BM / 2, WB = 16 * HN * WGN;
  const GemmArgs &p = q.g;
  const int lane = threadIdx.x & 63;
  float2 *red = (float2 *)lds;  // [WGN][BM]
  __syncthreads();
#pragma unroll
  for (int mh = 0; mh < 2; ++mh)
#pragma unroll
    for (int i = 0; i < HM; ++i) {
      const int r = mh * WA + wm * 16 * HM + i * 16 + (lane & 15), m = m0 + r;
      int t = m < p.M ? ce_target(q.ce, m) : -1;
      if (t >= p.N) t = -1;
      float top = -INFINITY;
#pragma unroll
      for (int nh = 0; nh < 2; ++nh)
#pragma unroll
        for (int j = 0; j < HN; ++j) {
          const int n = n0 + nh * WB + wn * 16 * HN + j * 16 + 4 * (lane >> 4);
          f32x4 &a = acc[mh][nh][i][j];
          if (t >= n && t < n + 4) {
            const int e = t - n;
            q.ce.target_logit[m] = e == 0 ? a[0] : e == 1 ? a[1] : e == 2 ? a[2] : a[3];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = n + e < p.N ? a[e] : -INFINITY;
            top = fmaxf(top, a[e]);
          }
        }
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float base = ce_base(top);
      float sum = 0.f;
#pragma unroll
      for (int nh = 0; nh < 2; ++nh)
#pragma unroll
        for (int j = 0; j < HN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum += __expf(acc[mh][nh][i][j][e] - base);
      sum += __shfl_xor(sum, 16, 64);
      sum += __shfl_xor(sum, 32, 64);
      if (lane < 16) red[wn * BM + r] = float2{top, sum};
    }
  __syncthreads();
  const int r = threadIdx.x;
  if (r < BM && m0 + r < p.M) {
    float2 a = red[r];
#pragma unroll
    for (int w = 1; w < WGN; ++w) a = ce_join(a, red[w * BM + r]);
    q.ce.part[(int64_t)(q.ce.part0 + nb) * p.M + m0 + r] = a;
  }
}

// dl in bf16, as the products that follow take it, half the rows at a time through LDS as in tile_epilogue;
// zeros in the columns that fill up its rows
template <int HM, int HN, int WGM, int WGN>
MOE_DEV void ce_grad(const PipeArgs &q, char *lds, const f32x4 (&acc)[2][2][HM][HN], int wm, int wn, int m0, int n0) {
  constexpr int BM = 32 * HM * WGM, BN = 32 * HN * WGN, WA = BM / 2, WB = BN / 2;
  const GemmArgs &p = q.g;
  const int lane = threadIdx.x & 63;
  auto chunk = [&](int r, int c) __attribute__((always_inline)) {
    return (f32x4 *)(lds + r * (BN * 4) + ((c ^ (r & 15)) << 4));
  };
  constexpr int LPR = BN / 8, RPP = 512 / LPR;
#pragma unroll
  for (int mh = 0; mh < 2; ++mh) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < HM; ++i)
#pragma unroll
      for (int nh = 0; nh < 2; ++nh)
#pragma unroll
        for (int j = 0; j < HN; ++j)
          *chunk(wm * 16 * HM + i * 16 + (lane & 15),
                 (nh * WB + wn * 16 * HN + j * 16) / 4 + (lane >> 4)) = acc[mh][nh][i][j];
    __syncthreads();
    const int r0 = threadIdx.x / LPR, c0 = (threadIdx.x % LPR) * 8, n = n0 + c0;
    if (n >= q.ce.ld) continue;
#pragma unroll 4
    for (int r = r0; r < WA; r += RPP) {
      const int m = m0 + mh * WA + r;
      if (m >= p.M) break;
      const CeRow row = q.ce.rows[m];
      f32x4 v[2] = {*chunk(r, c0 / 4), *chunk(r, c0 / 4 + 1)};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = n + 4 * h + e;
          v[h][e] = col < p.N ? ce_dl<bf16_t>(row, v[h][e], q.ce.col0 + col) : 0.f;
        }
      put8((bf16_t *)p.out + (int64_t)m * q.ce.ld + n, v);
      if (!q.ce.rest) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[h][e] -= (float)(__bf16)v[h][e];
      put8(q.ce.rest + (int64_t)m * q.ce.ld + n, v);
    }
  }
}

template <int HM, int HN, int WGM, int WGN, bool AK, bool BKM, typename To, int ACT>
__global__ __launch_bounds__(512, 2) void piped_gemm(PipeArgs q) {
  constexpr int BM = 32 * HM * WGM, BN = 32 * HN * WGN, WA = BM / 2, WB = BN / 2;
  constexpr int AH = WA * 128, BH = WB * 128, STG = 2 * (AH + BH);
  constexpr int PA = HalfTile<WA, AK>::PER, PB = HalfTile<WB, BKM>::PER;
  static_assert(WGM * WGN == 8 && PA >= 1 && PB >= 1, "8 waves, whole loads");
  extern __shared__ __align__(16) char lds[];
  const GemmArgs &p = q.g;
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // waves w and w + 4 share a SIMD: the second four run one part behind
  const int wm = wid % WGM, wn = wid / WGM;
  const int tiles = q.tm * q.tn;
  const int split = blockIdx.x / tiles;
  int mb, nb;
  tile_of(blockIdx.x - split * tiles, tiles, q.tm, q.tn, mb, nb);
  const int m0 = mb * BM, n0 = nb * BN;
  const int stages = (p.K + PBK - 1) / PBK;
  const int kb = (int)((int64_t)stages * split / q.splits), ke = (int)((int64_t)stages * (split + 1) / q.splits);
  const int kend = min(p.K, ke * PBK);  // loads past this range's end give zeros

  HalfTile<WA, AK> ta;
  HalfTile<WB, BKM> tb;
  ta.setup(m0, p.M, p.lda);
  tb.setup(n0, p.N, p.ldb);
  const __amdgpu_buffer_rsrc_t ra = uniform_rsrc(p.A, q.a_bytes), rb = uniform_rsrc(p.B, q.b_bytes);
  const uint32_t lda2 = (uint32_t)(2 * p.lda), ldb2 = (uint32_t)(2 * p.ldb);
  const uint32_t l0 =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(LDS_AS char *)lds) + wid * 1024;

  f32x4 acc[2][2][HM][HN] = {};
  bf16x8_t fan[HM], fa[2][HM], fb[2][HN][2];  // A0 step 0; A0 step 1 / A1; B halves

  auto issueA = [&](int half, int kt) __attribute__((always_inline)) {
    ta.issue(ra, half, kt, kend, lda2, l0 + ((kt - kb) & 1) * STG + half * AH);
  };
  auto issueB = [&](int half, int kt) __attribute__((always_inline)) {
    tb.issue(rb, half, kt, kend, ldb2, l0 + ((kt - kb) & 1) * STG + 2 * AH + half * BH);
  };
  auto readA = [&](int buf, int half, int s, bf16x8_t (&f)[HM]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < HM; ++i)
      f[i] = frag<WA, AK>(lds + buf * STG + half * AH, wm * 16 * HM + i * 16, s, lane);
  };
  auto readB = [&](int buf, int half) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < HN; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        fb[half][i][s] = frag<WB, BKM>(lds + buf * STG + 2 * AH + half * BH, wn * 16 * HN + i * 16, s, lane);
  };
  auto arrive = [&]() __attribute__((always_inline)) {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * PA + 2 * PB) : "memory");
    LIN_FENCE();
    __builtin_amdgcn_s_barrier();
    LIN_FENCE();
  };
  auto multiply = [&](int mh, int nh, bf16x8_t (&s0)[HM], bf16x8_t (&s1)[HM]) __attribute__((always_inline)) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < HM; ++i)
#pragma unroll
        for (int j = 0; j < HN; ++j)
          acc[mh][nh][i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[nh][j][s], s ? s1[i] : s0[i],
                                                                      acc[mh][nh][i][j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
    LIN_FENCE();
    __builtin_amdgcn_s_barrier();
    LIN_FENCE();
  };
  issueA(0, kb);
  issueB(0, kb);
  issueB(1, kb);
  issueA(1, kb);
  issueA(0, kb + 1);
  issueB(0, kb + 1);
  arrive();
  readA(0, 0, 0, fan);
  if (wid >= 4) __builtin_amdgcn_s_barrier();
  LIN_FENCE();
  auto stage = [&](int kt, auto BUF) __attribute__((always_inline)) {
    constexpr int buf = decltype(BUF)::value;
    readB(buf, 0);
    readA(buf, 0, 1, fa[1]);
    issueB(1, kt + 1);
    arrive();
    multiply(0, 0, fan, fa[1]);
    readB(buf, 1);
    issueA(1, kt + 1);
    arrive();
    multiply(0, 1, fan, fa[1]);
    readA(buf, 1, 0, fa[0]);
    readA(buf, 1, 1, fa[1]);
    issueA(0, kt + 2);
    arrive();
    multiply(1, 1, fa[0], fa[1]);
    readA(buf ^ 1, 0, 0, fan);
    issueB(0, kt + 2);
    arrive();
    multiply(1, 0, fa[0], fa[1]);
  };
  int kt = kb;
  for (; kt + 1 < ke; kt += 2) {
    stage(kt, std::integral_constant<int, 0>());
    stage(kt + 1, std::integral_constant<int, 1>());
  }
  if (kt < ke) stage(kt, std::integral_constant<int, 0>());
  if (wid < 4) __builtin_amdgcn_s_barrier();
  // zeros for stages that are not there, and the last early read, before the LDS is used again
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");

  if constexpr (ACT == kCeStats) ce_stats<HM, HN, WGM, WGN>(q, lds, acc, wm, wn, m0, n0, nb);
  else if constexpr (ACT == kCeGrad) ce_grad<HM, HN, WGM, WGN>(q, lds, acc, wm, wn, m0, n0);
  else tile_epilogue<HM, HN, WGM, WGN, To, ACT>(q, lds, acc, wm, wn, m0, n0, split);
}

// The same product with 128 x 128 tiles for problems whose 256-wide tiles leave CUs idle: 8 waves of
// 64 x 32 outputs, NST stages in a ring, one barrier per stage.  A stage is two 32-deep steps; each
// step's fragments are read while the step before multiplies.  The barrier between them also frees
// the stage's place (its reads are waited for just before) for the stage NST ahead.
//   NST = 4 (128 KB of LDS, one workgroup per CU) when there are at most as many workgroups as CUs: then
//           the bytes in flight are the limit; NST = 2 (64 KB, two per CU) otherwise.
template <int NST, bool AK, bool BKM, typename To, int ACT>
__global__ __launch_bounds__(512, NST == 2 ? 4 : 2) void ring_gemm(PipeArgs q) {
  constexpr int HM = 2, HN = 1, WGM = 2, WGN = 4, W = 128, OPB = W * 128, STG = 2 * OPB;
  using TA = HalfTile<W, AK>;
  using TB = HalfTile<W, BKM>;
  constexpr int D = TA::PER + TB::PER;  // loads per thread and stage
  extern __shared__ __align__(16) char lds[];
  const GemmArgs &p = q.g;
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wid % WGM, wn = wid / WGM;
  const int tiles = q.tm * q.tn;
  const int split = blockIdx.x / tiles;
  int mb, nb;
  tile_of(blockIdx.x - split * tiles, tiles, q.tm, q.tn, mb, nb);
  const int m0 = mb * W, n0 = nb * W;
  const int stages = (p.K + PBK - 1) / PBK;
  const int kb = (int)((int64_t)stages * split / q.splits), ke = (int)((int64_t)stages * (split + 1) / q.splits);
  const int kend = min(p.K, ke * PBK);
  TA ta;
  TB tb;
  ta.setup(m0, p.M, p.lda);
  tb.setup(n0, p.N, p.ldb);
  const __amdgpu_buffer_rsrc_t ra = uniform_rsrc(p.A, q.a_bytes), rb = uniform_rsrc(p.B, q.b_bytes);
  const uint32_t lda2 = (uint32_t)(2 * p.lda), ldb2 = (uint32_t)(2 * p.ldb);
  const uint32_t l0 =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(LDS_AS char *)lds) + wid * 1024;
  f32x4 acc[2][2][HM][HN] = {};
  bf16x8_t fa[2][2][HM], fb[2][2][HN];  // [step][half]
  auto issue = [&](int kt) __attribute__((always_inline)) {
    const uint32_t at = l0 + ((kt - kb) & (NST - 1)) * STG;
    ta.issue(ra, 0, kt, kend, lda2, at);
    tb.issue(rb, 0, kt, kend, ldb2, at + OPB);
  };
  auto read = [&](int kt, int s) __attribute__((always_inline)) {
    const char *t = lds + ((kt - kb) & (NST - 1)) * STG;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < HM; ++i) fa[s][h][i] = frag<W, AK>(t, h * 64 + wm * 16 * HM + i * 16, s, lane);
#pragma unroll
      for (int j = 0; j < HN; ++j) fb[s][h][j] = frag<W, BKM>(t + OPB, h * 64 + wn * 16 * HN + j * 16, s, lane);
    }
  };
  auto multiply = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int mh = 0; mh < 2; ++mh)
#pragma unroll
      for (int nh = 0; nh < 2; ++nh)
#pragma unroll
        for (int i = 0; i < HM; ++i)
#pragma unroll
          for (int j = 0; j < HN; ++j)
            acc[mh][nh][i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[s][nh][j], fa[s][mh][i],
                                                                        acc[mh][nh][i][j], 0, 0, 0);
  };
#pragma unroll
  for (int i = 0; i < NST; ++i) issue(kb + i);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NST - 1) * D) : "memory");
  LIN_FENCE();
  __builtin_amdgcn_s_barrier();
  LIN_FENCE();
  read(kb, 0);
  for (int kt = kb; kt < ke; ++kt) {
    LIN_FENCE();
    read(kt, 1);
    LIN_FENCE();
    multiply(0);
    LIN_FENCE();
    // stage kt + 1 has landed; this wave's reads of stage kt are done
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NST - 2) * D) : "memory");
    LIN_FENCE();
    __builtin_amdgcn_s_barrier();
    LIN_FENCE();
    read(kt + 1, 0);
    issue(kt + NST);
    LIN_FENCE();
    multiply(1);
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  if constexpr (ACT == kCeStats) ce_stats<HM, HN, WGM, WGN>(q, lds, acc, wm, wn, m0, n0, nb);
  else if constexpr (ACT == kCeGrad) ce_grad<HM, HN, WGM, WGN>(q, lds, acc, wm, wn, m0, n0);
  else tile_epilogue<HM, HN, WGM, WGN, To, ACT>(q, lds, acc, wm, wn, m0, n0, split);
}

// ---- streamed products: few rows or few columns --------------------------------
// For the forward's operands (both K-major, rows on 16-byte lines) with so few rows of x or of W
// that reading the other one is the work: 16 TI x 16 TJ outputs per workgroup, whose NW waves
// share the reduction (wave w takes the 64-element pieces w, w + NW, ..., whole 128-byte lines of
// bf16) and add up through LDS in wave order.  Operands go from memory to registers, 16 bytes per
// lane, D pieces ahead; the smaller operand comes out of L2.  Workgroups start at different pieces:
// rows are often a power of two apart, and all workgroups on the same piece meet on few channels.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <typename T>
MOE_DEV f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
  } else {
    // element e of every lane's four is one reduction index of a 16 x 16 x 4 product
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], c, 0, 0, 0);
    return c;
  }
}

template <typename T, typename To, int ACT, int TI, int TJ, int NW, int D>
__global__ __launch_bounds__(NW * 64) void stream_gemm(GemmArgs p) {
  constexpr int TM = 16 * TI, TN = 16 * TJ, E = 16 / sizeof(T);  // elements per 16 bytes
  constexpr int PIECE = 8 * E;
  // [NW][TM][TN], the 16-byte chunks of row m at places XORed with m, so that a fragment's rows
  // spread over the banks
  __shared__ __align__(16) float red[NW * TM * TN];
  auto cell = [](int w, int m, int n) __attribute__((always_inline)) {
    return (w * TM + m) * TN + (n ^ ((m & (TN / 4 - 1)) * 4));
  };
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tn = (p.N + TN - 1) / TN;
  const int m0 = blockIdx.x / tn * TM, n0 = blockIdx.x % tn * TN;
  const uint32_t rowb = (uint32_t)p.K * (uint32_t)sizeof(T);
  const __amdgpu_buffer_rsrc_t ra =
      uniform_rsrc((const T *)p.A + (int64_t)m0 * p.K, min(TM, p.M - m0) * rowb);
  const __amdgpu_buffer_rsrc_t rb =
      uniform_rsrc((const T *)p.B + (int64_t)n0 * p.K, min(TN, p.N - n0) * rowb);
  const uint32_t base = (lane & 15) * rowb;
  const int pieces = (p.K + PIECE - 1) / PIECE;
  f32x4 acc[TI][TJ] = {};
  u32x4 a[D][2][TI], b[D][2][TJ];
  const int rot = (int)(blockIdx.x % (uint32_t)pieces);
  auto load = [&](int pc, int d) __attribute__((always_inline)) {
    const bool on = pc < pieces;  // (past the end nothing is read)
    int at = pc + rot;
    at = at >= pieces ? at - pieces : at;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = at * PIECE + s * 4 * E + (lane >> 4) * E;
      const uint32_t off = on && k < p.K ? base + k * (uint32_t)sizeof(T) : kOobOffset;
#pragma unroll
      for (int i = 0; i < TI; ++i)
        a[d][s][i] = __builtin_amdgcn_raw_buffer_load_b128(ra, off + i * 16 * rowb, 0, 0);
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        b[d][s][j] = __builtin_amdgcn_raw_buffer_load_b128(rb, off + j * 16 * rowb, 0, 0);
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(wid + d * NW, d);
  for (int pc = wid; pc < pieces; pc += D * NW) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
          for (int j = 0; j < TJ; ++j) acc[i][j] = mfma16<T>(b[d][s][j], a[d][s][i], acc[i][j]);
      load(pc + (D + d) * NW, d);
    }
  }
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j)
      *(f32x4 *)&red[cell(wid, i * 16 + (lane & 15), j * 16 + 4 * (lane >> 4))] = acc[i][j];
  __syncthreads();
  for (int e = threadIdx.x; e < TM * TN; e += NW * 64) {
    const int m = m0 + e / TN, n = n0 + e % TN;
    if (m >= p.M || n >= p.N) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[cell(w, e / TN, e % TN)];
    if (p.bias) v += ldf((const T *)p.bias + n);
    finish1<T, To, ACT>(p, v, (int64_t)m * p.N + n);
  }
}

// ---- at most 4 rows of x: a wave per output column ---------------------------------
// 64 lanes read a row of W in whole lines, U x 16 bytes per lane in flight, and multiply it by every
// row of x (out of L1); fp32 sums per lane, then across the wave.
template <typename T>
MOE_DEV void dot16(u32x4 a, u32x4 b, float &s) {
  if constexpr (sizeof(T) == 4) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) s = fmaf(x[i], y[i], s);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s = fmaf(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16), s);
      s = fmaf(__uint_as_float(a[i] & 0xffff0000u), __uint_as_float(b[i] & 0xffff0000u), s);
    }
  }
}

template <typename T, typename To, int ACT, int MR>
__global__ __launch_bounds__(512) void row_gemm(GemmArgs p) {
  constexpr int E = 16 / sizeof(T), U = MR == 1 ? 8 : 4;
  const int lane = threadIdx.x & 63;
  const int n = blockIdx.x * 8 + (threadIdx.x >> 6);
  if (n >= p.N) return;
  const u32x4 *w = (const u32x4 *)((const T *)p.B + (int64_t)n * p.K);
  const u32x4 *x[MR];
#pragma unroll
  for (int m = 0; m < MR; ++m) x[m] = (const u32x4 *)((const T *)p.A + (int64_t)min(m, p.M - 1) * p.K);
  float s[MR][2] = {};
  const int chunks = p.K / E;
  for (int c0 = 0; c0 < chunks; c0 += 64 * U) {
    u32x4 wv[U], xv[U][MR];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * 64 + lane;
      wv[u] = c < chunks ? w[c] : u32x4{};
#pragma unroll
      for (int m = 0; m < MR; ++m) xv[u][m] = c < chunks ? x[m][c] : u32x4{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < MR; ++m) dot16<T>(wv[u], xv[u][m], s[m][u & 1]);
  }
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    float v = s[m][0] + s[m][1];
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
    if (lane == m && m < p.M) {
      if (p.bias) v += ldf((const T *)p.bias + n);
      finish1<T, To, ACT>(p, v, (int64_t)m * p.N + n);
    }
  }
}

// ---- dz and the bias gradient ---------------------------------------------------
// dz is rounded once, to nearest, to the operands' type, from fp32: the matrix instructions take both
// operands of a product in bf16.  That is an independent error of half a step in each term, as large in
// norm as the rounding of the outputs: 8192 x 4096 x 2048 with silu, dX and dW are off by 2.34e-3, by
// 1.66e-3 with their own rounding alone.  dz as two bf16 halves would halve the rate (twice the products), fp32
// products would take a tenth of it (275 GFLOP at 154 TFLOP/s: 1.8 ms against 0.23).  The bias gradient
// sums the unrounded values.
//
// Block (bx, by): 32 V columns from 32 V bx, rows from a contiguous range, 8 at a time; V columns
// (16 bytes of bf16 for V = 8) per thread.  Each block's column sums go to part[by][N]; bias_join
// adds them in order.  V = 8 where rows are on 16-byte lines.
constexpr int DZ_RANGES = 128;  // row ranges (at most)

template <typename T, int V>
MOE_DEV void getv(const T *p, float (&v)[V]) {
  if constexpr (V == 8) {
    const f32x4 a = get4(p), b = get4(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
  } else {
    v[0] = ldf(p);
  }
}
template <typename T, int V>
MOE_DEV void putv(T *p, const float (&v)[V]) {
  if constexpr (V == 8) {
    const f32x4 h[2] = {{v[0], v[1], v[2], v[3]}, {v[4], v[5], v[6], v[7]}};
    put8(p, h);
  } else {
    stf(p, v[0]);
  }
}

template <typename T, typename To, int ACT, int V>
__global__ __launch_bounds__(256) void dz_kernel(const To *__restrict__ dout,
                                                 const T *__restrict__ z, T *__restrict__ dz,
                                                 float *__restrict__ part, int64_t M, int N) {
  __shared__ float red[8][32 * V + 1];
  const int n = blockIdx.x * 32 * V + (threadIdx.x & 31) * V, q = threadIdx.x >> 5;
  const int64_t lo = M * blockIdx.y / gridDim.y, hi = M * (blockIdx.y + 1) / gridDim.y;
  float sum[V] = {};
  if (n < N) {
#pragma unroll 4
    for (int64_t m = lo + q; m < hi; m += 8) {
      const int64_t at = m * N + n;
      float d[V], zz[V];
      getv<To, V>(dout + at, d);
      if constexpr (ACT != MOE_ACT_NONE) {
        getv<T, V>(z + at, zz);
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] *= act_grad<ACT>(zz[i]);
      }
      if (dz) putv<T, V>(dz + at, d);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += d[i];
    }
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < V; ++i) red[q][(threadIdx.x & 31) * V + i] = sum[i];
  __syncthreads();
  const int c = threadIdx.x, nc = blockIdx.x * 32 * V + c;
  if (c < 32 * V && nc < N) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][c];
    part[(size_t)blockIdx.y * N + nc] = s;
  }
}

// 64 columns per block, 16 threads each
template <typename T>
__global__ __launch_bounds__(1024) void bias_join(const float *__restrict__ part, T *db, int N, int ranges) {
  __shared__ float red[16][65];
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6, n = blockIdx.x * 64 + c;
  float s = 0.f;
  if (n < N)
    for (int b = q; b < ranges; b += 16) s += part[(size_t)b * N + n];
  red[q][c] = s;
  __syncthreads();
  if (q == 0 && n < N) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += red[i][c];
    stf(db + n, s);
  }
}

bool on_line(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

// f(integral_constant<act>) for the forward (AK and BKM); the backward's products have none
template <bool FWD, class F>
void by_act_of(int act, F &&f) {
  if constexpr (FWD)
    by_act(act, f);
  else
    f(std::integral_constant<int, MOE_ACT_NONE>());
}

// launch of a kernel with more LDS than the default allows; the attribute is set once per device
template <auto KERNEL>
hipError_t launch_lds(int grid, size_t smem, const PipeArgs &q, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    e = hipFuncSetAttribute((const void *)KERNEL, hipFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != hipSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  KERNEL<<<grid, 512, smem, st>>>(q);
  return hipGetLastError();
}

template <bool AK, bool BKM, typename To>
hipError_t run_piped(PipeArgs &q, int shape, int act, hipStream_t st) {
  const int bm = kShapeM[shape], bn = kShapeN[shape];
  q.tm = (q.g.M + bm - 1) / bm;
  q.tn = (q.g.N + bn - 1) / bn;
  const int grid = q.tm * q.tn * q.splits;
  hipError_t e = hipSuccess;
  auto run = [&](auto A) {
    constexpr int ACT = decltype(A)::value;
    if (shape == 0)
      e = launch_lds<piped_gemm<4, 2, 2, 4, AK, BKM, To, ACT>>(grid, 128 << 10, q, st);
    else if (shape == 1)
      e = launch_lds<piped_gemm<2, 2, 4, 2, AK, BKM, To, ACT>>(grid, 96 << 10, q, st);
    else if (ring_stages(grid, device_cu_count()) == 4)
      e = launch_lds<ring_gemm<4, AK, BKM, To, ACT>>(grid, 128 << 10, q, st);
    else
      e = launch_lds<ring_gemm<2, AK, BKM, To, ACT>>(grid, 64 << 10, q, st);
  };
  if constexpr (AK && BKM && sizeof(To) == 2) {
    if (act == kCeGrad) {
      run(std::integral_constant<int, kCeGrad>());
      return e;
    }
  }
  if constexpr (AK && BKM && sizeof(To) == 4) {
    if (act == kCeStats) {
      run(std::integral_constant<int, kCeStats>());
      return e;
    }
  }
  by_act_of<AK && BKM>(act, run);
  return e;
}

// workspace for the partial products of either kernel
size_t part_bytes(int64_t M, int64_t N, int64_t K, bool bf16) {
  const int a = staged_plan(M, N, K, bf16).splits, b = bf16 ? plan_of(M, N, K).splits : 1;
  const int k = a > b ? a : b;
  return k > 1 ? (size_t)k * M * N * 4 : 0;
}

// Whether the forward streams: x or W has at most 16 rows, and rows on 16-byte lines.  (Up to 64 rows,
// as 32 x 64 tiles, the fragments of the smaller operand out of L2 are the limit: 8192 x 4096 x 64 took
// 26 us, as split 128 x 128 tiles 16 and 3 for the join.)
bool streams(const GemmArgs &a, size_t es) {
  return (a.M <= 16 || a.N <= 16) && a.K % (int)(16 / es) == 0 && a.K <= (1 << 22) && on_line(a.A, 16) &&
         on_line(a.B, 16);
}

template <bool FWD, typename T, typename To>
hipError_t join(const GemmArgs &a, int act, const void *part, int splits, hipStream_t st) {
  const int64_t groups = (int64_t)a.M * a.N / (a.vec ? 8 : 1);
  const int grid = (int)(groups < 256 * 4096 ? (groups + 255) / 256 : 4096);
  by_act_of<FWD>(act, [&](auto A) {
    join_kernel<T, To, decltype(A)::value><<<grid, 256, 0, st>>>(a, (const float *)part, splits);
  });
  return hipGetLastError();
}

template <typename T, typename To, int TI, int TJ, int NW, int D>
hipError_t run_stream(const GemmArgs &a, int act, hipStream_t st) {
  const int grid = ((a.M + 16 * TI - 1) / (16 * TI)) * ((a.N + 16 * TJ - 1) / (16 * TJ));
  by_act(act, [&](auto A) {
    stream_gemm<T, To, decltype(A)::value, TI, TJ, NW, D><<<grid, NW * 64, 0, st>>>(a);
  });
  return hipGetLastError();
}

template <bool AK, bool BKM, typename T, typename To>
hipError_t run_staged(const GemmArgs &a, const Plan &pl, int act, void *part, const CeArgs &ce, hipStream_t st) {
  const int ts = 64 * pl.shape;
  // memory rows (of lda, ldb elements, their whole length) on lines of four elements
  const bool fours = a.lda % 4 == 0 && a.ldb % 4 == 0 && on_line(a.A, 4 * sizeof(T)) && on_line(a.B, 4 * sizeof(T));
  const int grid = ((a.N + ts - 1) / ts) * ((a.M + ts - 1) / ts) * pl.splits;
  auto run = [&](auto A) {
    constexpr int ACT = decltype(A)::value;
    float *const out = (float *)part;
    if constexpr (sizeof(T) == 2) {
      if (pl.shape == 2) {
        if (fours) staged_gemm<T, To, 2, 4, AK, BKM, ACT><<<grid, SNT, 0, st>>>(a, pl.splits, out, ce);
        else staged_gemm<T, To, 2, 1, AK, BKM, ACT><<<grid, SNT, 0, st>>>(a, pl.splits, out, ce);
        return;
      }
    }
    if (fours) staged_gemm<T, To, 1, 4, AK, BKM, ACT><<<grid, SNT, 0, st>>>(a, pl.splits, out, ce);
    else staged_gemm<T, To, 1, 1, AK, BKM, ACT><<<grid, SNT, 0, st>>>(a, pl.splits, out, ce);
  };
  if constexpr (AK && BKM && sizeof(T) == 2 && sizeof(To) == 2) {
    if (act >= kCeStats) {
      if (act == kCeStats) run(std::integral_constant<int, kCeStats>());
      else run(std::integral_constant<int, kCeGrad>());
      return hipGetLastError();
    }
  }
  by_act_of<AK && BKM>(act, run);
  return hipGetLastError();
}

template <bool AK, bool BKM, typename T, typename To>
hipError_t gemm(GemmArgs a, int act, void *part, hipStream_t st) {
  if constexpr (AK) {
    // in runs of rows where one launch could not hold them (no sizes in memory make dW's do)
    const int64_t run = launch_rows(a.M, a.N);
    if (run < a.M) {
      for (int64_t m0 = 0; m0 < a.M; m0 += run) {
        GemmArgs b = a;
        b.M = (int)(a.M - m0 < run ? a.M - m0 : run);
        b.A = (const T *)a.A + m0 * a.lda;
        b.out = (To *)a.out + m0 * a.N;
        if (a.res) b.res = (const To *)a.res + m0 * a.N;
        if (a.z) b.z = (T *)a.z + m0 * a.N;
        if (a.factor) b.factor = a.factor + m0 * a.factor_step;
        const hipError_t e = gemm<AK, BKM, T, To>(b, act, part, st);
        if (e != hipSuccess) return e;
      }
      return hipSuccess;
    }
  }
  if constexpr (AK && BKM) {
    if (streams(a, sizeof(T))) {
      if (a.M <= 4) {
        by_act(act, [&](auto A) {
          constexpr int ACT = decltype(A)::value;
          if (a.M == 1)
            row_gemm<T, To, ACT, 1><<<(a.N + 7) / 8, 512, 0, st>>>(a);
          else
            row_gemm<T, To, ACT, 4><<<(a.N + 7) / 8, 512, 0, st>>>(a);
        });
        return hipGetLastError();
      }
      return run_stream<T, To, 1, 1, 16, 4>(a, act, st);
    }
  }
  a.vec = a.N % 8 == 0 && on_line(a.out, 16) && on_line(a.res, 16) && on_line(a.bias, 16) &&
          on_line(a.z, 16);
  if constexpr (sizeof(T) == 2) {
    // 16-byte chunks of both operands lie wholly inside or outside their rows
    const int64_t ra = AK ? a.M : a.K, rb = BKM ? a.N : a.K;
    const bool chunks = a.lda % 8 == 0 && a.ldb % 8 == 0 && on_line(a.A, 16) && on_line(a.B, 16);
    const int64_t ab = 2 * ra * a.lda, bb = 2 * rb * a.ldb;
    // 32-bit offsets, of rows up to a tile past the end too
    const bool small = a.lda <= (1 << 20) && a.ldb <= (1 << 20) && a.N <= (1 << 20) &&
                       ab < (int64_t)kOobOffset && bb < (int64_t)kOobOffset;
    if (chunks && small && a.K > 0) {
      const Plan pl = plan_of(a.M, a.N, a.K);
      PipeArgs q{a, (uint32_t)ab, (uint32_t)bb, 0, 0, pl.splits, (float *)part};
      const hipError_t e = run_piped<AK, BKM, To>(q, pl.shape, act, st);
      if (e != hipSuccess || pl.splits == 1) return e;
      return join<AK && BKM, T, To>(a, act, part, pl.splits, st);
    }
  }
  const Plan pl = staged_plan(a.M, a.N, a.K, sizeof(T) == 2);
  const hipError_t e = run_staged<AK, BKM, T, To>(a, pl, act, part, CeArgs{}, st);
  if (e != hipSuccess || pl.splits == 1) return e;
  return join<AK && BKM, T, To>(a, act, part, pl.splits, st);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
bool needs_dz(int act, int dtype, int out_dtype) { return act != MOE_ACT_NONE || dtype != out_dtype; }
int dz_ranges(int64_t M) { return (int)(M < 8 * DZ_RANGES ? (M + 7) / 8 : DZ_RANGES); }

// workspace of the backward: dz, the column sums' parts, the partial products of dX or dW
struct BwdSpace {
  size_t dz, sums, part, total;
};
BwdSpace bwd_space(int64_t M, int64_t K, int64_t N, bool own_dz, int dtype) {
  BwdSpace w;
  w.dz = 0;
  w.sums = own_dz ? up256((size_t)M * N * (dtype == MOE_F32 ? 4 : 2)) : 0;
  w.part = w.sums + up256((size_t)dz_ranges(M) * N * 4);
  const bool bf16 = dtype == MOE_BF16;
  const size_t px = part_bytes(M, K, N, bf16), pw = part_bytes(N, K, M, bf16);
  w.total = w.part + up256(px > pw ? px : pw);
  return w;
}

template <typename T, typename To>
hipError_t bwd(const void *dout, const void *x, const void *W, const void *z, void *dX, void *dW,
               void *db, int M, int K, int N, int act, bool own_dz, void *ws, hipStream_t st) {
  const BwdSpace w = bwd_space(M, K, N, own_dz, sizeof(T) == 4 ? MOE_F32 : MOE_BF16);
  const T *d = own_dz ? (const T *)ws : (const T *)dout;
  float *sums = (float *)((char *)ws + w.sums);
  void *part = (char *)ws + w.part;
  const int ranges = dz_ranges(M);
  hipError_t e = hipSuccess;
  if (M > 0 && ((own_dz && (dX || dW)) || db)) {
    T *dz = own_dz && (dX || dW) ? (T *)ws : nullptr;
    const bool wide = N % 8 == 0 && on_line(dout, 16) && on_line(z, 16);
    by_act(act, [&](auto A) {
      constexpr int ACT = decltype(A)::value;
      if (wide)
        dz_kernel<T, To, ACT, 8><<<dim3((N + 255) / 256, ranges), 256, 0, st>>>(
            (const To *)dout, (const T *)z, dz, db ? sums : nullptr, M, N);
      else
        dz_kernel<T, To, ACT, 1><<<dim3((N + 31) / 32, ranges), 256, 0, st>>>(
            (const To *)dout, (const T *)z, dz, db ? sums : nullptr, M, N);
    });
    e = hipGetLastError();
  }
  if (e == hipSuccess && db) {
    bias_join<T><<<(N + 63) / 64, 1024, 0, st>>>(sums, (T *)db, N, M > 0 ? ranges : 0);
    e = hipGetLastError();
  }
  if (e == hipSuccess && dX && M > 0)
    e = gemm<true, false, T, T>(GemmArgs{d, W, nullptr, nullptr, dX, nullptr, M, K, N, N, K, false},
                                MOE_ACT_NONE, part, st);
  if (e == hipSuccess && dW)
    e = gemm<false, false, T, T>(GemmArgs{d, x, nullptr, nullptr, dW, nullptr, N, K, M, N, K, false},
                                 MOE_ACT_NONE, part, st);
  return e;
}

}  // namespace

// ---- products of the linear cross entropy ------------------------------------------
bool ce_tiles(int64_t M, int64_t K, int64_t V) {
  const int64_t most = (int64_t)kOobOffset / 2;
  return M > 16 && K % 8 == 0 && K <= (1 << 20) && V <= (1 << 20) && M * K < most && V * K < most &&
         ((M + 127) / 128) * ((V + 127) / 128) <= (1 << 22) && plan_of(M, V, K).splits == 1;
}
int ce_tile_columns(int64_t M, int64_t K, int64_t V) { return kShapeN[unsplit_shape(M, V, K)]; }
hipError_t launch_ce_tiles(const void *x, const void *W, void *dl, const CeArgs &ce, int M, int K, int V, int shape_v,
                           hipStream_t st) {
  PipeArgs q{};
  q.g = GemmArgs{x, W, nullptr, nullptr, dl, nullptr, M, V, K, K, K, false};
  q.a_bytes = (uint32_t)((int64_t)M * K * 2);
  q.b_bytes = (uint32_t)((int64_t)V * K * 2);
  q.splits = 1;
  q.ce = ce;
  const int shape = unsplit_shape(M, shape_v, K);
  return dl ? run_piped<true, true, bf16_t>(q, shape, kCeGrad, st) : run_piped<true, true, float>(q, shape, kCeStats, st);
}
// fp32 (reduction and rows of at least four): what a product's epilogue or its ranges' sums take
template <bool AK, bool BKM, int ACT>
static void launch_fine(const GemmArgs &a, const Plan &pl, void *part, const CeArgs &ce, hipStream_t st) {
  const int ts = 64 * pl.shape, grid = ((a.M + ts - 1) / ts) * ((a.N + ts - 1) / ts) * pl.splits;
  if (pl.shape == 2) fine_gemm<2, AK, BKM, ACT><<<grid, SNT, 0, st>>>(a, pl.splits, (float *)part, ce);
  else fine_gemm<1, AK, BKM, ACT><<<grid, SNT, 0, st>>>(a, pl.splits, (float *)part, ce);
}
template <bool AK, bool BKM>
static hipError_t fine(const GemmArgs &a, void *part, hipStream_t st) {
  const Plan pl = fine_plan(a.M, a.N, a.K, true);
  launch_fine<AK, BKM, MOE_ACT_NONE>(a, pl, part, CeArgs{}, st);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || pl.splits == 1 ? e : join<AK && BKM, float, float>(a, MOE_ACT_NONE, part, pl.splits, st);
}
static size_t fine_bytes(int64_t M, int64_t N, int64_t K) {
  const int k = fine_plan(M, N, K, true).splits;
  return k > 1 ? (size_t)k * M * N * 4 : 0;
}
bool ce_staged(int64_t M, int64_t K, int64_t V, int dtype) {
  if (M <= 16 || V <= 16 || launch_rows(M, V) < M) return false;
  return dtype == MOE_F32 ? K >= 4 && fine_whole(M, V, K) : staged_plan(M, V, K, true).splits == 1;
}
int ce_staged_columns(int64_t M, int64_t K, int64_t V, int dtype) {
  return 32 * (dtype == MOE_F32 ? fine_plan(M, V, K, false) : staged_plan(M, V, K, true)).shape;
}
hipError_t launch_ce_staged(const void *x, const void *W, void *dl, const CeArgs &ce, int M, int K, int V, int shape_v, int dtype,
                            hipStream_t st) {
  const GemmArgs a{x, W, nullptr, nullptr, dl, nullptr, M, V, K, K, K, false};
  if (dtype == MOE_F32) {
    const Plan pl = fine_plan(M, shape_v, K, false);
    if (dl) launch_fine<true, true, kCeGrad>(a, pl, nullptr, ce, st);
    else launch_fine<true, true, kCeStats>(a, pl, nullptr, ce, st);
    return hipGetLastError();
  }
  const Plan pl{staged_plan(M, shape_v, K, true).shape, 1};
  return run_staged<true, true, bf16_t, bf16_t>(a, pl, dl ? kCeGrad : kCeStats, nullptr, ce, st);
}
// Whether products of these sizes take the parts (runs of four have to fit into every row; the logits of few rows of x
// are streamed instead)
static bool takes_parts(int64_t M, int64_t K, int64_t V, int dtype) { return dtype == MOE_F32 && K >= 4 && V >= 4 && M > 0; }
size_t ce_part_bytes(int64_t M, int64_t K, int64_t V, int dtype) {
  size_t most = 0;
  for (size_t b : {part_bytes(M, K, V, dtype == MOE_BF16), part_bytes(V, K, M, dtype == MOE_BF16),
                   takes_parts(M, K, V, dtype) ? fine_bytes(M, K, V) : 0, takes_parts(M, K, V, dtype) ? fine_bytes(V, K, M) : 0})
    most = b > most ? b : most;
  return most;
}
size_t ce_logits_part_bytes(int64_t M, int64_t K, int64_t V, int dtype) {
  const size_t a = part_bytes(M, V, K, dtype == MOE_BF16), b = M > 16 && takes_parts(M, K, V, dtype) ? fine_bytes(M, V, K) : 0;
  return a > b ? a : b;
}
hipError_t launch_ce_logits(const void *x, const void *W, float *logits, int M, int K, int V, int dtype, void *part, hipStream_t st) {
  if (M > 16 && takes_parts(M, K, V, dtype))
    return fine<true, true>(GemmArgs{x, W, nullptr, nullptr, logits, nullptr, M, V, K, K, K, false}, part, st);
  return launch_linear_fwd(x, W, nullptr, nullptr, logits, nullptr, M, K, V, MOE_ACT_NONE, dtype, MOE_F32, part, st);
}
hipError_t launch_ce_dx(const void *dl, int64_t ld, const void *W, const float *sum, const float *factor, void *out, bool out_f32,
                        int M, int K, int V, int dtype, void *part, hipStream_t st) {
  const GemmArgs a{dl, W, nullptr, sum, out, nullptr, M, K, V, ld, K, false, factor, 1};
  if (takes_parts(M, K, V, dtype)) return fine<true, false>(a, part, st);
  if (dtype == MOE_F32) return gemm<true, false, float, float>(a, MOE_ACT_NONE, part, st);
  if (out_f32) return gemm<true, false, bf16_t, float>(a, MOE_ACT_NONE, part, st);
  return gemm<true, false, bf16_t, bf16_t>(a, MOE_ACT_NONE, part, st);
}
hipError_t launch_ce_dw(const void *dl, int64_t ld, const void *x, const float *factor, void *dW, int M, int K, int V, int dtype,
                        void *part, hipStream_t st) {
  const GemmArgs a{dl, x, nullptr, nullptr, dW, nullptr, V, K, M, ld, K, false, factor, 0};
  if (takes_parts(M, K, V, dtype)) return fine<false, false>(a, part, st);
  if (dtype == MOE_F32) return gemm<false, false, float, float>(a, MOE_ACT_NONE, part, st);
  return gemm<false, false, bf16_t, bf16_t>(a, MOE_ACT_NONE, part, st);
}

size_t linear_fwd_workspace(int64_t M, int64_t K, int64_t N, int dtype) {
  return part_bytes(M, N, K, dtype == MOE_BF16);
}

size_t linear_bwd_workspace(int64_t M, int64_t K, int64_t N, int act, int dtype, int out_dtype) {
  return bwd_space(M, K, N, needs_dz(act, dtype, out_dtype), dtype).total;
}

hipError_t launch_linear_fwd(const void *x, const void *W, const void *bias, const void *res,
                             void *out, void *z, int M, int K, int N, int act, int dtype,
                             int out_dtype, void *ws, hipStream_t st) {
  const GemmArgs a{x, W, bias, res, out, z, M, N, K, K, K, false};
  if (dtype == MOE_F32) return gemm<true, true, float, float>(a, act, ws, st);
  if (out_dtype == MOE_F32) return gemm<true, true, bf16_t, float>(a, act, ws, st);
  return gemm<true, true, bf16_t, bf16_t>(a, act, ws, st);
}

hipError_t launch_linear_bwd(const void *dout, const void *x, const void *W, const void *z,
                             void *dX, void *dW, void *db, int M, int K, int N, int act, int dtype,
                             int out_dtype, void *ws, hipStream_t st) {
  const bool own = needs_dz(act, dtype, out_dtype);
  if (dtype == MOE_F32)
    return bwd<float, float>(dout, x, W, z, dX, dW, db, M, K, N, act, own, ws, st);
  if (out_dtype == MOE_F32)
    return bwd<bf16_t, float>(dout, x, W, z, dX, dW, db, M, K, N, act, own, ws, st);
  return bwd<bf16_t, bf16_t>(dout, x, W, z, dX, dW, db, M, K, N, act, own, ws, st);
}

}  // namespace moe
