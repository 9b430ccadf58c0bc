// Dense linear layer with bias, activation and residual in the product's epilogue, and its
// backward:  z = x W^T + b,  out = act(z) + r;  dz = d_out act'(z),  dx = dz W,  dW = dz^T x,
// db = sum of dz over the rows.
//
// All three products have one form, C[m, n] = sum_k A(m, k) B(n, k): for each operand either the
// reduction index (K-major) or the output index (MN-major) is contiguous in memory.
#include <type_traits>

#include "common.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

MOE_DEV float ldf(const float *p) { return *p; }
MOE_DEV float ldf(const bf16_t *p) { return bf16_to_f32(*p); }
MOE_DEV void stf(float *p, float v) { *p = v; }
MOE_DEV void stf(bf16_t *p, float v) { *p = __builtin_bit_cast(bf16_t, (__bf16)v); }

// ---- activations ------------------------------------------------------------
MOE_DEV float sigmoidf(float t) { return 1.f / (1.f + __expf(-t)); }
constexpr float kTanhC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;

template <int ACT>
MOE_DEV float act_fwd(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z < 0.f ? 0.f : z;  // a NaN stays one
  if constexpr (ACT == MOE_ACT_GELU) return 0.5f * z * erfcf(-0.70710678f * z);
  // 0.5 (1 + tanh u) = sigmoid(2 u)
  if constexpr (ACT == MOE_ACT_GELU_TANH)
    return z * sigmoidf(2.f * kTanhC * (z + kTanhA * z * z * z));
  if constexpr (ACT == MOE_ACT_SILU) return z * sigmoidf(z);
  return z;
}

template <int ACT>
MOE_DEV float act_grad(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == MOE_ACT_GELU)
    return 0.5f * erfcf(-0.70710678f * z) + z * 0.3989422804f * __expf(-0.5f * z * z);
  if constexpr (ACT == MOE_ACT_GELU_TANH) {
    const float s = sigmoidf(2.f * kTanhC * (z + kTanhA * z * z * z)), t = s * (1.f - s);
    // far out t is 0 and its factor may overflow
    return t == 0.f ? s : s + z * t * (2.f * kTanhC * (1.f + 3.f * kTanhA * z * z));
  }
  if constexpr (ACT == MOE_ACT_SILU) {
    const float s = sigmoidf(z);
    return s * (1.f + z * (1.f - s));
  }
  return 1.f;
}

// f(integral_constant<act>)
template <class F>
void by_act(int act, F &&f) {
  switch (act) {
    case MOE_ACT_RELU: f(std::integral_constant<int, MOE_ACT_RELU>()); break;
    case MOE_ACT_GELU: f(std::integral_constant<int, MOE_ACT_GELU>()); break;
    case MOE_ACT_GELU_TANH: f(std::integral_constant<int, MOE_ACT_GELU_TANH>()); break;
    case MOE_ACT_SILU: f(std::integral_constant<int, MOE_ACT_SILU>()); break;
    default: f(std::integral_constant<int, MOE_ACT_NONE>());
  }
}

struct GemmArgs {
  const void *A, *B;
  const void *bias, *res;  // [N] operand type, [M, N] output type; NULL: none
  void *out, *z;           // [M, N]; z (operand type) NULL: not kept
  int M, N, K;
  int64_t lda, ldb;  // K-major: elements between rows; MN-major: between reduction rows
  bool quad;         // N a multiple of 4, out, z, residual and bias on lines of four elements
};

// ---- epilogue -----------------------------------------------------------------
// four values of one row at columns n .. n+3, `left` >= 1 of them inside the row; quad: rows are
// multiples of 4 elements and the pointers on 16-byte (fp32) or 8-byte (bf16) lines, so all four
// are inside and moved at once
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
MOE_DEV f32x4 get4(const float *p, int left, bool quad) {
  if (quad) return *(const f32x4 *)p;
  f32x4 v = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) if (i < left) v[i] = p[i];
  return v;
}
MOE_DEV f32x4 get4(const bf16_t *p, int left, bool quad) {
  f32x4 v = {};
  if (quad) {
    const bf16x4_t b = *(const bf16x4_t *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)b[i];
    return v;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) if (i < left) v[i] = ldf(p + i);
  return v;
}
MOE_DEV void put4(float *p, f32x4 v, int left, bool quad) {
  if (quad) { *(f32x4 *)p = v; return; }
#pragma unroll
  for (int i = 0; i < 4; ++i) if (i < left) p[i] = v[i];
}
MOE_DEV void put4(bf16_t *p, f32x4 v, int left, bool quad) {
  if (quad) {
    *(bf16x4_t *)p = bf16x4_t{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) if (i < left) stf(p + i, v[i]);
}
// z = v + bias, out = act(z) + residual
template <typename T, typename To, int ACT>
MOE_DEV void finish4(const GemmArgs &p, f32x4 v, int n, int64_t at, bool quad) {
  const int left = p.N - n;
  if (p.bias) v += get4((const T *)p.bias + n, left, quad);
  if (p.z) put4((T *)p.z + at, v, left, quad);
  if constexpr (ACT != MOE_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = act_fwd<ACT>(v[i]);
  }
  if (p.res) v += get4((const To *)p.res + at, left, quad);
  put4((To *)p.out + at, v, left, quad);
}

// out[m, n .. n+3] from the partial products of all ranges, added in order
template <typename T, typename To, int ACT>
__global__ __launch_bounds__(256) void join_kernel(GemmArgs p, const float *part, int splits) {
  const int per = (p.N + 3) / 4;
  const int64_t total = (int64_t)p.M * per, size = (int64_t)p.M * p.N;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / per;
    const int n = (int)(i - m * per) * 4;
    const int64_t at = m * p.N + n;
    const bool pq = (p.N & 3) == 0;
    f32x4 v = get4(part + at, p.N - n, pq);
    for (int s = 1; s < splits; ++s) v += get4(part + s * size + at, p.N - n, pq);
    finish4<T, To, ACT>(p, v, n, at, p.quad);
  }
}

// ---- staged tiles: any alignment and size ------------------------------------
// 128 x 128 outputs per 4 waves (2 x 2, 64 x 64 each), 32 reduction elements per
// step through registers into LDS, element loads with bounds checks.
constexpr int SBM = 128, SBN = 128, SBK = 32, SNT = 256;

template <typename T>
struct Pitch {  // LDS row pitch in elements: rows 16-byte aligned, spread over the banks
  static constexpr int v = sizeof(T) == 2 ? SBK + 8 : SBK + 1;
};

// a 128 x 32 tile of an operand: element (r, k) to lds[r][k]; thread t brings 16 elements
template <typename T, bool KMAJ>
MOE_DEV void stage_load(const T *p, int64_t ld, int r0, int rows, int k0, int K, T (&v)[16]) {
  const int t = threadIdx.x;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = KMAJ ? i * 8 + (t >> 5) : t & 127;
    const int k = KMAJ ? t & 31 : i * 2 + (t >> 7);
    const bool ok = r0 + r < rows && k0 + k < K;
    const int64_t at = KMAJ ? (int64_t)(r0 + r) * ld + k0 + k : (int64_t)(k0 + k) * ld + r0 + r;
    v[i] = ok ? p[at] : (T)0;
  }
}
template <typename T, bool KMAJ>
MOE_DEV void stage_store(T *lds, const T (&v)[16]) {
  const int t = threadIdx.x;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = KMAJ ? i * 8 + (t >> 5) : t & 127;
    const int k = KMAJ ? t & 31 : i * 2 + (t >> 7);
    lds[r * Pitch<T>::v + k] = v[i];
  }
}

// row of register i of a 32 x 32 accumulator
MOE_DEV int acc_row(int i, int lane) { return ((i >> 2) << 3) + ((lane >> 5) << 2) + (i & 3); }

template <typename T, typename To, bool AK, bool BKM, int ACT>
__global__ __launch_bounds__(SNT) void staged_gemm(GemmArgs p) {
  constexpr int P = Pitch<T>::v;
  __shared__ T As[SBM * P], Bs[SBN * P];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int wm = (wid >> 1) * 64, wn = (wid & 1) * 64;
  const int tn = (p.N + SBN - 1) / SBN;
  const int m0 = blockIdx.x / tn * SBM, n0 = blockIdx.x % tn * SBN;
  f32x16 acc[2][2] = {};
  T va[16], vb[16];
  stage_load<T, AK>((const T *)p.A, p.lda, m0, p.M, 0, p.K, va);
  stage_load<T, BKM>((const T *)p.B, p.ldb, n0, p.N, 0, p.K, vb);
  for (int k0 = 0; k0 < p.K; k0 += SBK) {
    __syncthreads();
    stage_store<T, AK>(As, va);
    stage_store<T, BKM>(Bs, vb);
    __syncthreads();
    if (k0 + SBK < p.K) {
      stage_load<T, AK>((const T *)p.A, p.lda, m0, p.M, k0 + SBK, p.K, va);
      stage_load<T, BKM>((const T *)p.B, p.ldb, n0, p.N, k0 + SBK, p.K, vb);
    }
    const int r = lane & 31, h = lane >> 5;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int s = 0; s < SBK / 16; ++s) {
        bf16x8_t a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[i] = *(const bf16x8_t *)&As[(wm + i * 32 + r) * P + s * 16 + h * 8];
          b[i] = *(const bf16x8_t *)&Bs[(wn + i * 32 + r) * P + s * 16 + h * 8];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int s = 0; s < SBK / 2; ++s) {
        float a[2], b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[i] = As[(wm + i * 32 + r) * P + s * 2 + h];
          b[i] = Bs[(wn + i * 32 + r) * P + s * 2 + h];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[j], acc[i][j], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int n = n0 + wn + j * 32 + (lane & 31);
    if (n >= p.N) continue;
    const float b = p.bias ? ldf((const T *)p.bias + n) : 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int m = m0 + wm + i * 32 + acc_row(e, lane);
        if (m >= p.M) continue;
        const int64_t at = (int64_t)m * p.N + n;
        float v = acc[i][j][e] + b;
        if (p.z) stf((T *)p.z + at, v);
        v = act_fwd<ACT>(v);
        if (p.res) v += ldf((const To *)p.res + at);
        stf((To *)p.out + at, v);
      }
  }
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
// Order of issue: A0 B0 B1 of a stage two ahead (into the buffer whose halves the quarters before
// have read), A1 of the next.  A half is waited for one quarter before its first read, five
// halves after its issue.  The reads of a memory part are complete (lgkmcnt 0) before its
// barrier, so the halves it read may be overwritten after it.
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
#define LDS_AS __attribute__((address_space(3)))
constexpr int PBK = 64;

// 16 bytes per lane from rsrc + voff to LDS byte address lds + 16 * lane (lds wave-uniform);
// zeros where voff is out of the buffer
MOE_DEV void dma16(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, uint32_t lds) {
  const uint32_t m0v = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(m0v), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
MOE_DEV __amdgpu_buffer_rsrc_t uniform_rsrc(const void *p, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return make_rsrc((const void *)(uintptr_t)(((uint64_t)hi << 32) | lo),
                   __builtin_amdgcn_readfirstlane(bytes));
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

struct PipeArgs {
  GemmArgs g;
  uint32_t a_bytes, b_bytes;
  int tm, tn, splits;  // tiles; reduction ranges (> 1: fp32 partial products to part)
  float *part;         // [splits][M][N]
};

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
  auto arrive = [&](auto VM) __attribute__((always_inline)) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(VM)::value) : "memory");
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
  using V1 = std::integral_constant<int, 3 * PA + 2 * PB>;
  using V2 = std::integral_constant<int, 2 * PA + 3 * PB>;

  issueA(0, kb);
  issueB(0, kb);
  issueB(1, kb);
  issueA(1, kb);
  issueA(0, kb + 1);
  issueB(0, kb + 1);
  issueB(1, kb + 1);
  arrive(V2());
  readA(0, 0, 0, fan);
  if (wid >= 4) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
  }
  LIN_FENCE();
  auto stage = [&](int kt, auto BUF) __attribute__((always_inline)) {
    constexpr int buf = decltype(BUF)::value;
    readB(buf, 0);
    readA(buf, 0, 1, fa[1]);
    issueA(1, kt + 1);
    arrive(V1());
    multiply(0, 0, fan, fa[1]);
    readB(buf, 1);
    issueA(0, kt + 2);
    arrive(V1());
    multiply(0, 1, fan, fa[1]);
    readA(buf, 1, 0, fa[0]);
    readA(buf, 1, 1, fa[1]);
    issueB(0, kt + 2);
    arrive(V2());
    multiply(1, 1, fa[0], fa[1]);
    readA(buf ^ 1, 0, 0, fan);
    issueB(1, kt + 2);
    arrive(V2());
    multiply(1, 0, fa[0], fa[1]);
  };
  int kt = kb;
  for (; kt + 1 < ke; kt += 2) {
    stage(kt, std::integral_constant<int, 0>());
    stage(kt + 1, std::integral_constant<int, 1>());
  }
  if (kt < ke) stage(kt, std::integral_constant<int, 0>());
  if (wid < 4) __builtin_amdgcn_s_barrier();
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (zeros for stages that are not there)

  // lane l of a 16 x 16 block: row l & 15, columns 4 (l >> 4) .. +3
  const bool quad = p.quad;
#pragma unroll
  for (int mh = 0; mh < 2; ++mh)
#pragma unroll
    for (int i = 0; i < HM; ++i) {
      const int m = m0 + mh * WA + wm * 16 * HM + i * 16 + (lane & 15);
      if (m >= p.M) continue;
#pragma unroll
      for (int nh = 0; nh < 2; ++nh)
#pragma unroll
        for (int j = 0; j < HN; ++j) {
          const int n = n0 + nh * WB + wn * 16 * HN + j * 16 + 4 * (lane >> 4);
          if (n >= p.N) continue;
          const f32x4 v = acc[mh][nh][i][j];
          const int64_t at = (int64_t)m * p.N + n;
          if (q.splits > 1)
            put4(q.part + (int64_t)split * p.M * p.N + at, v, p.N - n, (p.N & 3) == 0);
          else
            finish4<bf16_t, To, ACT>(p, v, n, at, quad);
        }
    }
}

// ---- dz and the bias gradient ---------------------------------------------------
// Block (bx, by): columns 64 bx .. +63, rows by, by + gridDim.y, ... (4 at a time).  Each block's
// column sums go to part[by][N]; bias_join adds them in order.
constexpr int DZ_BLOCKS = 64;

template <typename T, typename To, int ACT>
__global__ __launch_bounds__(256) void dz_kernel(const To *__restrict__ dout,
                                                 const T *__restrict__ z, T *__restrict__ dz,
                                                 float *__restrict__ part, int64_t M, int N) {
  __shared__ float red[256];
  const int n = blockIdx.x * 64 + (threadIdx.x & 63), q = threadIdx.x >> 6;
  float sum = 0.f;
  if (n < N)
    for (int64_t m = (int64_t)blockIdx.y * 4 + q; m < M; m += (int64_t)gridDim.y * 4) {
      const int64_t at = m * N + n;
      float d = ldf(dout + at);
      if constexpr (ACT != MOE_ACT_NONE) d *= act_grad<ACT>(ldf(z + at));
      if (dz) stf(dz + at, d);
      sum += d;
    }
  if (!part) return;
  red[threadIdx.x] = sum;
  __syncthreads();
  if (q == 0 && n < N)
    part[(size_t)blockIdx.y * N + n] =
        (red[threadIdx.x] + red[threadIdx.x + 64]) + (red[threadIdx.x + 128] + red[threadIdx.x + 192]);
}

template <typename T>
__global__ __launch_bounds__(256) void bias_join(const float *__restrict__ part, T *db, int N, int blocks) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float s = 0.f;
  for (int b = 0; b < blocks; ++b) s += part[(size_t)b * N + n];
  stf(db + n, s);
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

template <int HM, int HN, int WGM, int WGN, bool AK, bool BKM, typename To>
hipError_t run_piped(PipeArgs &q, int act, hipStream_t st) {
  constexpr int BM = 32 * HM * WGM, BN = 32 * HN * WGN, SMEM = 2 * 128 * (BM + BN);
  q.tm = (q.g.M + BM - 1) / BM;
  q.tn = (q.g.N + BN - 1) / BN;
  const int grid = q.tm * q.tn * q.splits;
  hipError_t e = hipSuccess;
  by_act_of<AK && BKM>(act, [&](auto A) {
    auto k = piped_gemm<HM, HN, WGM, WGN, AK, BKM, To, decltype(A)::value>;
    e = hipFuncSetAttribute((const void *)k, hipFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e == hipSuccess) {
      k<<<grid, 512, SMEM, st>>>(q);
      e = hipGetLastError();
    }
  });
  return e;
}

template <bool AK, bool BKM, typename T, typename To>
hipError_t gemm(GemmArgs a, int act, hipStream_t st) {
  a.quad = a.N % 4 == 0 && on_line(a.out, 4 * sizeof(To)) && on_line(a.res, 4 * sizeof(To)) &&
           on_line(a.bias, 4 * sizeof(T)) && on_line(a.z, 4 * sizeof(T));
  if constexpr (sizeof(T) == 2) {
    // 16-byte chunks of both operands lie wholly inside or outside their rows
    const int64_t ra = AK ? a.M : a.K, rb = BKM ? a.N : a.K;
    const bool chunks = a.lda % 8 == 0 && a.ldb % 8 == 0 && on_line(a.A, 16) && on_line(a.B, 16);
    const int64_t ab = 2 * ra * a.lda, bb = 2 * rb * a.ldb;
    // offsets of rows up to a tile past the end must not wrap
    if (chunks && a.lda <= (1 << 21) && a.ldb <= (1 << 21) && ab < (int64_t)kOobOffset && bb < (int64_t)kOobOffset && a.K > 0) {
      PipeArgs q{a, (uint32_t)ab, (uint32_t)bb, 0, 0, 1, nullptr};
      return run_piped<4, 2, 2, 4, AK, BKM, To>(q, act, st);
    }
  }
  const int grid = ((a.N + SBN - 1) / SBN) * ((a.M + SBM - 1) / SBM);
  by_act_of<AK && BKM>(act, [&](auto A) {
    staged_gemm<T, To, AK, BKM, decltype(A)::value><<<grid, SNT, 0, st>>>(a);
  });
  return hipGetLastError();
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
bool needs_dz(int act, int dtype, int out_dtype) { return act != MOE_ACT_NONE || dtype != out_dtype; }
int dz_blocks(int64_t M) { return (int)(M < 4 * DZ_BLOCKS ? (M + 3) / 4 : DZ_BLOCKS); }

template <typename T, typename To>
hipError_t bwd(const void *dout, const void *x, const void *W, const void *z, void *dX, void *dW,
               void *db, int M, int K, int N, int act, bool own_dz, void *ws, hipStream_t st) {
  const T *d = own_dz ? (const T *)ws : (const T *)dout;
  float *part = (float *)((char *)ws + (own_dz ? up256((size_t)M * N * sizeof(T)) : 0));
  const int blocks = dz_blocks(M);
  hipError_t e = hipSuccess;
  if (M > 0 && ((own_dz && (dX || dW)) || db)) {
    const dim3 grid((N + 63) / 64, blocks);
    by_act(act, [&](auto A) {
      dz_kernel<T, To, decltype(A)::value><<<grid, 256, 0, st>>>(
          (const To *)dout, (const T *)z, own_dz ? (T *)ws : nullptr, db ? part : nullptr, M, N);
    });
    e = hipGetLastError();
  }
  if (e == hipSuccess && db) {
    bias_join<T><<<(N + 255) / 256, 256, 0, st>>>(part, (T *)db, N, M > 0 ? blocks : 0);
    e = hipGetLastError();
  }
  if (e == hipSuccess && dX && M > 0)
    e = gemm<true, false, T, T>(GemmArgs{d, W, nullptr, nullptr, dX, nullptr, M, K, N, N, K, false},
                                MOE_ACT_NONE, st);
  if (e == hipSuccess && dW)
    e = gemm<false, false, T, T>(GemmArgs{d, x, nullptr, nullptr, dW, nullptr, N, K, M, N, K, false},
                                 MOE_ACT_NONE, st);
  return e;
}

}  // namespace

size_t linear_fwd_workspace(int64_t M, int64_t K, int64_t N, int dtype) { return 0; }

size_t linear_bwd_workspace(int64_t M, int64_t K, int64_t N, int act, int dtype, int out_dtype) {
  const size_t es = dtype == MOE_F32 ? 4 : 2;
  return (needs_dz(act, dtype, out_dtype) ? up256((size_t)M * N * es) : 0) +
         up256((size_t)dz_blocks(M) * N * 4);
}

hipError_t launch_linear_fwd(const void *x, const void *W, const void *bias, const void *res,
                             void *out, void *z, int M, int K, int N, int act, int dtype,
                             int out_dtype, void *ws, hipStream_t st) {
  const GemmArgs a{x, W, bias, res, out, z, M, N, K, K, K, false};
  if (dtype == MOE_F32) return gemm<true, true, float, float>(a, act, st);
  if (out_dtype == MOE_F32) return gemm<true, true, bf16_t, float>(a, act, st);
  return gemm<true, true, bf16_t, bf16_t>(a, act, st);
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
