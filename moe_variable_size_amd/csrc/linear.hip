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
};

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

template <bool AK, bool BKM, typename T, typename To>
hipError_t gemm(const GemmArgs &a, int act, hipStream_t st) {
  const int grid = ((a.N + SBN - 1) / SBN) * ((a.M + SBM - 1) / SBM);
  by_act(act, [&](auto A) { staged_gemm<T, To, AK, BKM, decltype(A)::value><<<grid, SNT, 0, st>>>(a); });
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
    e = gemm<true, false, T, T>(GemmArgs{d, W, nullptr, nullptr, dX, nullptr, M, K, N, N, K},
                                MOE_ACT_NONE, st);
  if (e == hipSuccess && dW)
    e = gemm<false, false, T, T>(GemmArgs{d, x, nullptr, nullptr, dW, nullptr, N, K, M, N, K},
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
  const GemmArgs a{x, W, bias, res, out, z, M, N, K, K, K};
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
