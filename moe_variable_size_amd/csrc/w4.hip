// Products with 4-bit weights, W[n, k] = (q[n, k] - z[n, g]) s[n, g] in groups g of 32, 64 or 128 reduction
// elements, for few rows of bf16 x: what there is to do is to read the codes.
//
// The codes become bf16 in registers and go into the matrix cores as they are: with a nibble shifted to the
// upper mantissa bits, 0x4180 | q << 3 is the bf16 number 16 + q (exact), two of them for a shift and an
// and-or.  A group's sum is taken from there,
//     sum (q - z) x = sum (16 + q) x - (16 + z) sum x,
// with sum x from the matrix cores too (a product with ones; 16 of it is what the group's accumulator begins
// with), and the scale applied to it in fp32.  So no weight is rounded, and products and sums are as exact as bf16's.
//
// A 128-element block of a row is 64 bytes, 16 for each quarter q of a wave's lanes: word j holds elements 32 j + 8
// q .. +7, what lane quarter q feeds into the block's j-th 16 x 16 x 32 product, so that a lane loads 16 bytes at a
// time and each product lies in one group.
#include "activation.hpp"
#include "common.hpp"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int BLK = 128;  // reduction elements of a block, 64 bytes of codes

MOE_DEV __amdgpu_buffer_rsrc_t uniform_rsrc(const void *p, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return make_rsrc((const void *)(uintptr_t)(((uint64_t)hi << 32) | lo), __builtin_amdgcn_readfirstlane(bytes));
}

// 16 + q of a word's eight codes, elements 0 .. 7
MOE_DEV bf16x8 unpack(uint32_t w) {
  constexpr uint32_t M = 0x00780078u, O = 0x41804180u;
  const u32x4 v = {((w << 3) & M) | O, ((w >> 1) & M) | O, ((w >> 5) & M) | O, ((w >> 9) & M) | O};
  return __builtin_bit_cast(bf16x8, v);
}
MOE_DEV bf16x8 all_of(uint32_t two) { return __builtin_bit_cast(bf16x8, u32x4{two, two, two, two}); }

struct Weight {
  const uint8_t *codes;
  const bf16_t *scales;
  const uint8_t *zeros;
  int64_t per_codes, per_scales;  // of one expert, in bytes of codes and in scales
  int N, K, cols;                 // cols: N filled up to 16, the row length of scales and zeros
  int blocks, groups;             // of a row
};

// The sums of 16 TI rows of x and 16 TJ columns over a wave's share of the blocks, those numbered wid, wid + NW, ...
// acc of lane l: column l & 15, rows 4 (l >> 4) .. +3 (so that a lane needs one scale and one zero point).  GP: groups
// of a block.  Codes are loaded D blocks ahead, x (out of L2) DX ahead; a block's offset is the loads' scalar one, which
// no bounds check sees: every lane that loads is inside its row at every block, the others are out of range anyway.
template <int TI, int TJ, int GP, bool ZEROS, int D, int DX>
struct Wave {
  static_assert(D % DX == 0, "");
  u32x4 w[D][TJ], x[DX][4][TI];
  uint32_t s[D][TJ], z[D][TJ];  // lane quarter q: of group q (q % 2, 0) of the block
  f32x4 acc[TI][TJ];
  uint32_t wo[TJ], so[TJ], xo[TI];

  // xo: byte offsets of the rows (l & 15 of each tile) in x, out of range for none
  MOE_DEV void setup(const Weight &p, int n0) {
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int n = n0 + j * 16 + r;
      wo[j] = n < p.N ? (uint32_t)n * ((uint32_t)p.blocks * 64) + q * 16 : kOobOffset;
      so[j] = n < p.N ? (uint32_t)(q & (GP - 1)) * (uint32_t)p.cols + n : kOobOffset;
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      xo[i] += xo[i] < kOobOffset ? q * 16 : 0;
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{};
    }
  }
  MOE_DEV void load_w(int d, const Weight &p, __amdgpu_buffer_rsrc_t rw, __amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t rz, int b) {
    const bool in = b * GP + (int)((threadIdx.x & 63) >> 4 & (GP - 1)) < p.groups;
    const uint32_t g = (uint32_t)(b * GP) * (uint32_t)p.cols;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      w[d][j] = __builtin_amdgcn_raw_buffer_load_b128(rw, wo[j], b * 64, 0);
      s[d][j] = __builtin_amdgcn_raw_buffer_load_b16(rs, in && so[j] < kOobOffset ? 2 * so[j] : kOobOffset, 2 * g, 0);
      if constexpr (ZEROS) z[d][j] = __builtin_amdgcn_raw_buffer_load_b8(rz, in ? so[j] : kOobOffset, g, 0);
    }
  }
  MOE_DEV void load_x(int d, const Weight &p, __amdgpu_buffer_rsrc_t rx, int b) {
    const int k = b * BLK + (int)((threadIdx.x & 63) >> 4) * 8;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < TI; ++i)
        x[d][t][i] = __builtin_amdgcn_raw_buffer_load_b128(rx, k + 32 * t < p.K ? xo[i] + 64 * t : kOobOffset, b * 256, 0);
  }
  // weight: of the rows' assignments, 1 where it is applied later
  MOE_DEV void multiply(int d, int dx, float weight) {
    constexpr int PER = 4 / GP;  // products of a group
    // One column tile and group after the other (empty assembly keeps its order): the compiler begins all of them at
    // once otherwise, and spills their sums
    constexpr bool ORDER = GP * TI * TJ > 4;
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      f32x4 sum[TI], base[TI];  // sum x; what the accumulators begin with
      float zero_sum = 0.f;
      if constexpr (ORDER) asm volatile("" : "+v"(zero_sum));
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        sum[i] = base[i] = f32x4{zero_sum, zero_sum, zero_sum, zero_sum};
#pragma unroll
        for (int t = 0; t < PER; ++t) {
          const bf16x8 xv = __builtin_bit_cast(bf16x8, x[dx][g * PER + t][i]);
          if constexpr (ZEROS)
            sum[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, all_of(0x3F803F80u), sum[i], 0, 0, 0);  // 1
          else
            base[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, all_of(0xC1C0C1C0u), base[i], 0, 0, 0);  // -24
        }
        if constexpr (ZEROS) base[i] = -16.f * sum[i];
      }
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        f32x4 part[TI];
#pragma unroll
        for (int t = 0; t < PER; ++t) {
          uint32_t word = w[d][j][g * PER + t];
          if constexpr (ORDER) asm volatile("" : "+v"(word));
          const bf16x8 wv = unpack(word);
#pragma unroll
          for (int i = 0; i < TI; ++i)
            part[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[dx][g * PER + t][i]), wv,
                                                              t ? part[i] : base[i], 0, 0, 0);
        }
        uint32_t sc = s[d][j], zc = ZEROS ? z[d][j] : 0;
        if constexpr (GP > 1) {  // from the quarter that has this group's
          const int from = ((threadIdx.x & 15) + 16 * g) * 4;
          sc = __builtin_amdgcn_ds_bpermute(from, sc);
          if constexpr (ZEROS) zc = __builtin_amdgcn_ds_bpermute(from, zc);
        }
        const float scale = __uint_as_float(sc << 16) * weight, zero = (float)zc;
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = ZEROS ? fmaf(-zero, sum[i][e], part[i][e]) : part[i][e];
            acc[i][j][e] = fmaf(scale, v, acc[i][j][e]);
          }
        if constexpr (ORDER) {
#pragma unroll
          for (int i = 0; i < TI; ++i) asm volatile("" : "+v"(acc[i][j]));
        }
      }
    }
  }
  // all of the wave's blocks; they begin at another place in each workgroup, since rows are often a power of two
  // apart and all workgroups on the same block would meet on few channels
  template <int NW>
  MOE_DEV void run(const Weight &p, __amdgpu_buffer_rsrc_t rw, __amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t rz,
                   __amdgpu_buffer_rsrc_t rx, int n0, uint32_t place) {
    setup(p, n0);
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), rot = (int)(place % (uint32_t)p.blocks);
    auto block = [&](int u) __attribute__((always_inline)) { return u + rot >= p.blocks ? u + rot - p.blocks : u + rot; };
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (wid + d * NW < p.blocks) load_w(d, p, rw, rs, rz, block(wid + d * NW));
#pragma unroll
    for (int d = 0; d < DX; ++d)
      if (wid + d * NW < p.blocks) load_x(d, p, rx, block(wid + d * NW));
    for (int b = wid; b < p.blocks; b += D * NW) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const int u = b + d * NW;
        if (u >= p.blocks) break;
        multiply(d, d % DX, 1.f);
        if (u + D * NW < p.blocks) load_w(d, p, rw, rs, rz, block(u + D * NW));
        if (u + DX * NW < p.blocks) load_x(d % DX, p, rx, block(u + DX * NW));
      }
    }
  }
};

// The waves' sums of 16 rows (`rows` of them in use), added in wave order through red [NW][16][16 TJ + 4]; f(row, column,
// sum) for each
template <int TJ>
constexpr int kPitch = 16 * TJ + 4;
template <int TJ, int NW, class F>
MOE_DEV void join_waves(float *red, const f32x4 (&acc)[TJ], int rows, F &&f) {
  constexpr int TN = 16 * TJ;
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < TJ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 4 * (lane >> 4) + e;
      if (r < rows) red[(wid * 16 + r) * kPitch<TJ> + j * 16 + (lane & 15)] = acc[j][e];
    }
  __syncthreads();
  for (int e = threadIdx.x; e < min(rows, 16) * TN; e += NW * 64) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += red[(w * 16 + e / TN) * kPitch<TJ> + e % TN];
    f(e / TN, e % TN, v);
  }
}

// ---- dense -------------------------------------------------------------------------
struct DenseArgs {
  Weight w;
  const bf16_t *x, *bias;
  const void *res;
  void *out;
  int M;
};
MOE_DEV float ldf(const float *p) { return *p; }
MOE_DEV float ldf(const bf16_t *p) { return bf16_to_f32(*p); }
MOE_DEV void stf(float *p, float v) { *p = v; }
MOE_DEV void stf(bf16_t *p, float v) { *p = __builtin_bit_cast(bf16_t, (__bf16)v); }

template <int TI, int TJ, int NW, int GP, bool ZEROS, int D, int DX, typename To>
__global__ __launch_bounds__(NW * 64) void dense_kernel(DenseArgs a, int act) {
  __shared__ __align__(16) float red[NW * 16 * kPitch<TJ>];
  const int tm = (a.M + 16 * TI - 1) / (16 * TI);
  // the row tiles of one column tile are neighbours: its codes come from L2 from the second on
  const int m0 = blockIdx.x % tm * (16 * TI), n0 = blockIdx.x / tm * (16 * TJ);
  const int lane = threadIdx.x & 63;
  const Weight &p = a.w;
  const auto rw = uniform_rsrc(p.codes, (uint32_t)p.per_codes), rs = uniform_rsrc(p.scales, (uint32_t)(2 * p.per_scales));
  const auto rz = uniform_rsrc(ZEROS ? p.zeros : p.codes, ZEROS ? (uint32_t)p.per_scales : 0u);
  const auto rx = uniform_rsrc(a.x + (int64_t)m0 * p.K, (uint32_t)min(16 * TI, a.M - m0) * (uint32_t)p.K * 2);
  Wave<TI, TJ, GP, ZEROS, D, DX> v;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int r = i * 16 + (lane & 15);
    v.xo[i] = m0 + r < a.M ? (uint32_t)r * (uint32_t)p.K * 2 : kOobOffset;
  }
  v.template run<NW>(p, rw, rs, rz, rx, n0, blockIdx.x);
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int rows = a.M - m0 - i * 16;
    if (rows <= 0) break;
    join_waves<TJ, NW>(red, v.acc[i], rows, [&](int r, int c, float s) {
      if (n0 + c >= p.N) return;
      const int64_t at = (int64_t)(m0 + i * 16 + r) * p.N + n0 + c;
      if (a.bias) s += bf16_to_f32(a.bias[n0 + c]);
      s = act_fwd_of(act, s);
      if (a.res) s += ldf((const To *)a.res + at);
      stf((To *)a.out + at, s);
    });
  }
}

// ---- experts, through a schedule ---------------------------------------------------
struct ExpertArgs {
  Weight w;
  const bf16_t *x;
  float *y;
  const int32_t *counts, *offsets, *row_to_token;
  const float *row_weight;
  int T, layout, capacity, tn, e0;  // e0: first expert of the launch
};

template <int TI, int TJ, int NW, int GP, bool ZEROS, int D, int DX>
MOE_DEV void expert_rows(const ExpertArgs &a, float *red, int e, int n0, int row0, int rows) {
  const int lane = threadIdx.x & 63;
  const Weight &p = a.w;
  const auto rw = uniform_rsrc(p.codes + e * p.per_codes, (uint32_t)p.per_codes);
  const auto rs = uniform_rsrc(p.scales + e * p.per_scales, (uint32_t)(2 * p.per_scales));
  const auto rz = uniform_rsrc(ZEROS ? p.zeros + e * p.per_scales : p.codes, ZEROS ? (uint32_t)p.per_scales : 0u);
  const auto rx = uniform_rsrc(a.x, (uint32_t)a.T * (uint32_t)p.K * 2);
  Wave<TI, TJ, GP, ZEROS, D, DX> v;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int r = i * 16 + (lane & 15), t = r < rows ? a.row_to_token[row0 + r] : -1;
    v.xo[i] = t >= 0 ? (uint32_t)t * (uint32_t)p.K * 2 : kOobOffset;
  }
  v.template run<NW>(p, rw, rs, rz, rx, n0, blockIdx.x);
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    if (i * 16 >= rows) break;
    join_waves<TJ, NW>(red, v.acc[i], rows - i * 16, [&](int r, int c, float s) {
      r += i * 16;
      if (n0 + c >= p.N) return;
      const int t = a.row_to_token[row0 + r];
      if (t >= 0) unsafeAtomicAdd(a.y + (int64_t)t * p.N + n0 + c, s * a.row_weight[row0 + r]);
    });
  }
}

// One workgroup per expert and column tile; an expert's rows 16 TI at a time (the last ones 16 if that will do), its
// codes then coming out of the caches.
template <int TI, int TJ, int NW, int GP, bool ZEROS, int D, int DX>
__global__ __launch_bounds__(NW * 64) void expert_kernel(ExpertArgs a) {
  __shared__ __align__(16) float red[NW * 16 * kPitch<TJ>];
  const int e = a.e0 + blockIdx.x / a.tn, n0 = blockIdx.x % a.tn * (16 * TJ);
  const int count = __builtin_amdgcn_readfirstlane(a.counts[e]);
  const int first = a.layout == MOE_LAYOUT_MASKED ? e * a.capacity : __builtin_amdgcn_readfirstlane(a.offsets[e]) - count;
  for (int r = 0; r < count; r += 16 * TI) {
    if (TI > 1 && count - r <= 16) expert_rows<1, TJ, NW, GP, ZEROS, D, DX>(a, red, e, n0, first + r, count - r);
    else expert_rows<TI, TJ, NW, GP, ZEROS, D, DX>(a, red, e, n0, first + r, min(count - r, 16 * TI));
  }
}

// ---- experts of single tokens --------------------------------------------------------
struct TokenArgs {
  Weight w;
  const bf16_t *x;
  const int32_t *ids;
  const float *weights;
  float *y;
  int k, E, tn;
};

// One workgroup per token and column tile: its waves share the blocks of all k experts, whose routing weights go into
// the scales; plain stores.
template <int TJ, int NW, int GP, bool ZEROS, int D, int DX>
__global__ __launch_bounds__(NW * 64) void token_kernel(TokenArgs a) {
  __shared__ __align__(16) float red[NW * 16 * kPitch<TJ>];
  const int64_t t = blockIdx.x / a.tn;
  const int n0 = (int)(blockIdx.x - t * a.tn) * (16 * TJ);
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Weight &p = a.w;
  const auto rx = uniform_rsrc(a.x + t * p.K, (uint32_t)p.K * 2);
  Wave<1, TJ, GP, ZEROS, D, DX> v;
  v.xo[0] = (lane & 15) == 0 ? 0u : kOobOffset;
  v.setup(p, n0);
  float weight[D];
  const int total = a.k * p.blocks;
  auto load = [&](int d, int u) __attribute__((always_inline)) {
    const int slot = u / p.blocks, e = __builtin_amdgcn_readfirstlane(a.ids[t * a.k + slot]);
    const bool use = e >= 0 && e < a.E;
    const int64_t at = use ? e : 0;  // (a slot that is left out: sums that count 0)
    weight[d] = use ? (a.weights ? a.weights[t * a.k + slot] : 1.f) : 0.f;
    const auto rw = uniform_rsrc(p.codes + at * p.per_codes, use ? (uint32_t)p.per_codes : 0u);
    const auto rs = uniform_rsrc(p.scales + at * p.per_scales, use ? (uint32_t)(2 * p.per_scales) : 0u);
    const auto rz = uniform_rsrc(ZEROS ? p.zeros + at * p.per_scales : p.codes, use && ZEROS ? (uint32_t)p.per_scales : 0u);
    v.load_w(d, p, rw, rs, rz, u - slot * p.blocks);
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (wid + d * NW < total) load(d, wid + d * NW);
#pragma unroll
  for (int d = 0; d < DX; ++d)
    if (wid + d * NW < total) v.load_x(d, p, rx, (wid + d * NW) % p.blocks);
  for (int b = wid; b < total; b += D * NW) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int u = b + d * NW;
      if (u >= total) break;
      v.multiply(d, d % DX, weight[d]);
      if (u + D * NW < total) load(d, u + D * NW);
      if (u + DX * NW < total) v.load_x(d % DX, p, rx, (u + DX * NW) % p.blocks);
    }
  }
  join_waves<TJ, NW>(red, v.acc[0], 1, [&](int, int c, float s) {
    if (n0 + c < p.N) a.y[t * p.N + n0 + c] = s;
  });
}

// ---- codes from weights and back -------------------------------------------------------
// 8 elements per lane, G / 8 lanes per group; a wave takes 512 elements of a row.
MOE_DEV uint32_t word_at(int k) { return (uint32_t)(k / BLK) * 64 + (k % 32 / 8) * 16 + (k % BLK / 32) * 4; }

template <typename T, int G>
__global__ __launch_bounds__(256) void quantize_kernel(const T *__restrict__ W, Weight p, int64_t rows, uint8_t *codes, bf16_t *scales,
                                                       uint8_t *zeros) {
  const int runs = (p.blocks * BLK + 511) / 512, lane = threadIdx.x & 63;
  const int64_t total = rows * runs;
  for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < total; u += (int64_t)gridDim.x * 4) {
    const int64_t row = u / runs;
    const int k = (int)(u - row * runs) * 512 + lane * 8;
    float v[8], lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = k + i < p.K ? ldf(W + row * p.K + k + i) : 0.f;
      lo = fminf(lo, v[i]);
      hi = fmaxf(hi, v[i]);
    }
#pragma unroll
    for (int d = 1; d < G / 8; d <<= 1) {
      lo = fminf(lo, __shfl_xor(lo, d, 64));
      hi = fmaxf(hi, __shfl_xor(hi, d, 64));
    }
    const float wide = zeros ? (hi - lo) / 15.f : fmaxf(-lo, hi) / 7.f;
    const __bf16 s16 = (__bf16)wide;
    const float s = (float)s16, inv = s >= 0x1p-126f ? 1.f / s : 0.f;  // (no scale: every code the zero point)
    const float z = zeros ? fminf(fmaxf(rintf(-lo * inv), 0.f), 15.f) : 8.f;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = fminf(fmaxf(rintf(v[i] * inv) + z, 0.f), 15.f);
      word |= (uint32_t)q << (4 * ((i & 1) * 4 + i / 2));
    }
    if (k < p.blocks * BLK) *(uint32_t *)(codes + row * p.blocks * 64 + word_at(k)) = word;
    if (k % G == 0 && k < p.K) {
      const int64_t e = row / p.N, n = row - e * p.N, at = e * p.per_scales + (int64_t)(k / G) * p.cols + n;
      scales[at] = inv > 0.f ? __builtin_bit_cast(bf16_t, s16) : 0;
      if (zeros) zeros[at] = (uint8_t)z;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void dequantize_kernel(Weight p, int64_t rows, int group, T *__restrict__ W) {
  const int runs = (p.K + 511) / 512, lane = threadIdx.x & 63;
  const int64_t total = rows * runs;
  for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < total; u += (int64_t)gridDim.x * 4) {
    const int64_t row = u / runs;
    const int k = (int)(u - row * runs) * 512 + lane * 8;
    if (k >= p.K) continue;
    const int64_t e = row / p.N, n = row - e * p.N, at = e * p.per_scales + (int64_t)(k / group) * p.cols + n;
    const uint32_t word = *(const uint32_t *)(p.codes + row * p.blocks * 64 + word_at(k));
    const float s = bf16_to_f32(p.scales[at]), z = p.zeros ? (float)p.zeros[at] : 8.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < p.K) stf(W + row * p.K + k + i, ((float)(word >> (4 * ((i & 1) * 4 + i / 2)) & 15u) - z) * s);
  }
}

// ---- launches ----------------------------------------------------------------------------
Weight weight_of(const moe_w4_weight &w) {
  Weight p;
  p.codes = (const uint8_t *)w.codes;
  p.scales = (const bf16_t *)w.scales;
  p.zeros = (const uint8_t *)w.zeros;
  p.N = (int)w.N;
  p.K = (int)w.K;
  p.cols = (int)((w.N + 15) / 16 * 16);
  p.blocks = (int)((w.K + BLK - 1) / BLK);
  p.groups = (int)((w.K + w.group - 1) / w.group);
  p.per_codes = w.N * p.blocks * 64;
  p.per_scales = (int64_t)p.groups * p.cols;
  return p;
}

// f(groups per block, zeros?) as constants
template <class F>
void by_form(const moe_w4_weight &w, F &&f) {
  auto z = [&](auto gp) {
    if (w.zeros) f(gp, std::true_type());
    else f(gp, std::false_type());
  };
  if (w.group == 32) z(std::integral_constant<int, 4>());
  else if (w.group == 64) z(std::integral_constant<int, 2>());
  else z(std::integral_constant<int, 1>());
}

template <int TI, int TJ, int NW, int D, int DX, typename To>
hipError_t run_dense(const moe_w4_weight &w, DenseArgs a, int act, hipStream_t st) {
  const int64_t tn = (w.N + 16 * TJ - 1) / (16 * TJ), M = a.M;
  // workgroups of one launch: below 2^31 work-items
  const int64_t most = (((int64_t)1 << 31) / (NW * 64) / tn - 1) * 16 * TI, run = M < most ? M : most;
  for (int64_t m = 0; m < M; m += run) {
    DenseArgs b = a;
    b.M = (int)(M - m < run ? M - m : run);
    b.x += m * w.K;
    b.out = (To *)a.out + m * w.N;
    if (a.res) b.res = (const To *)a.res + m * w.N;
    const int grid = (int)(tn * ((b.M + 16 * TI - 1) / (16 * TI)));
    by_form(w, [&](auto gp, auto z) {
      dense_kernel<TI, TJ, NW, decltype(gp)::value, decltype(z)::value, D, DX, To><<<grid, NW * 64, 0, st>>>(b, act);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <typename To>
hipError_t dense(const moe_w4_weight &w, const DenseArgs &a, int act, hipStream_t st) {
  if (a.M > 32) return run_dense<4, 2, 8, 2, 1, To>(w, a, act, st);
  if (a.M > 16) return run_dense<2, 2, 8, 2, 1, To>(w, a, act, st);
  return run_dense<1, 1, 8, 4, 2, To>(w, a, act, st);
}

}  // namespace

hipError_t launch_w4_quantize(const void *W, const moe_w4_weight &w, int dtype, hipStream_t st) {
  const Weight p = weight_of(w);
  const int64_t rows = w.E * w.N;
  const int grid = 4096;
  auto run = [&](auto t, auto g) {
    using T = decltype(t);
    quantize_kernel<T, decltype(g)::value><<<grid, 256, 0, st>>>((const T *)W, p, rows, (uint8_t *)w.codes, (bf16_t *)w.scales,
                                                                 (uint8_t *)w.zeros);
  };
  auto by_group = [&](auto t) {
    if (w.group == 32) run(t, std::integral_constant<int, 32>());
    else if (w.group == 64) run(t, std::integral_constant<int, 64>());
    else run(t, std::integral_constant<int, 128>());
  };
  if (dtype == MOE_F32) by_group(float());
  else by_group(bf16_t());
  return hipGetLastError();
}

hipError_t launch_w4_dequantize(const moe_w4_weight &w, void *W, int dtype, hipStream_t st) {
  const Weight p = weight_of(w);
  const int64_t rows = w.E * w.N;
  if (dtype == MOE_F32) dequantize_kernel<float><<<4096, 256, 0, st>>>(p, rows, w.group, (float *)W);
  else dequantize_kernel<bf16_t><<<4096, 256, 0, st>>>(p, rows, w.group, (bf16_t *)W);
  return hipGetLastError();
}

hipError_t launch_linear_w4(const void *x, const moe_w4_weight &w, const void *bias, const void *res, void *out, int64_t M, int act,
                            int out_dtype, hipStream_t st) {
  const DenseArgs a{weight_of(w), (const bf16_t *)x, (const bf16_t *)bias, res, out, (int)M};
  return out_dtype == MOE_F32 ? dense<float>(w, a, act, st) : dense<bf16_t>(w, a, act, st);
}

hipError_t launch_fused_w4(const void *x, const moe_w4_weight &w, const moe_schedule &s, float *y, hipStream_t st) {
  ExpertArgs a{weight_of(w), (const bf16_t *)x, y, s.counts, s.offsets, s.row_to_token, s.row_weight, (int)s.T, s.layout, s.capacity, 0, 0};
  const bool few = s.S <= 12 * (int64_t)s.E;
  a.tn = (a.w.N + 63) / 64;
  const int run = (1 << 22) / a.tn;  // experts of one launch: at most 2^31 work-items
  for (; a.e0 < s.E; a.e0 += run) {
    const int grid = a.tn * (s.E - a.e0 < run ? s.E - a.e0 : run);
    by_form(w, [&](auto gp, auto z) {
      constexpr int GP = decltype(gp)::value;
      constexpr bool Z = decltype(z)::value;
      if (few) expert_kernel<1, 4, 8, GP, Z, 2, 2><<<grid, 512, 0, st>>>(a);
      else expert_kernel<2, 4, 8, GP, Z, 2, 1><<<grid, 512, 0, st>>>(a);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_token_w4(const void *x, const moe_w4_weight &w, const int32_t *ids, const float *weights, int64_t T, int k, float *y,
                           hipStream_t st) {
  TokenArgs a{weight_of(w), (const bf16_t *)x, ids, weights, y, k, (int)w.E, 0};
  a.tn = (a.w.N + 15) / 16;
  const int64_t run = ((int64_t)1 << 31) / 1024 / a.tn;  // tokens of one launch
  for (int64_t t = 0; t < T; t += run) {
    TokenArgs b = a;
    b.x += t * w.K;
    b.ids += t * k;
    if (weights) b.weights += t * k;
    b.y += t * w.N;
    const int grid = (int)((T - t < run ? T - t : run) * a.tn);
    by_form(w, [&](auto gp, auto z) { token_kernel<1, 16, decltype(gp)::value, decltype(z)::value, 4, 2><<<grid, 1024, 0, st>>>(b); });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
