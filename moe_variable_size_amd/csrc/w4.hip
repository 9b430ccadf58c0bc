// Products with 4-bit weights, W[n, k] = (q[n, k] - z[n, g]) s[n, g] in groups g of 32, 64 or 128 reduction
// elements, for few rows of bf16 x: what there is to do is to read the codes.
//
// The codes become bf16 in registers and go into the matrix cores as they are: with a nibble shifted to the
// upper mantissa bits, 0x4180 | q << 3 is the bf16 number 16 + q (exact), two of them for a shift and an
// and-or.  A group's sum is taken from there,
//     sum (q - z) x = sum (16 + q) x - (16 + z) sum x,
// with sum x from the matrix cores too (a product with ones; 16 of it is what the group's accumulator begins
// with), and the scale applied to it in fp32.  So no weight is rounded, and products and sums are as exact as bf16's.
// Where x is infinite, or so large that a sum with the 16s in it is, the difference is not the result: a sum that is not finite
// is taken again, weight by weight (plain_sum).
//
// A 128-element block of a row is 64 bytes, 16 for each quarter q of a wave's lanes: word j holds elements 32 j + 8
// q .. +7, what lane quarter q feeds into the block's j-th 16 x 16 x 32 product, so that a lane loads 16 bytes at a
// time and each product lies in one group.
#include <atomic>

#include "activation.hpp"
#include "common.hpp"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int BLK = 128;   // reduction elements of a block, 64 bytes of codes
constexpr int WAVES = 8;   // of a workgroup, but for single tokens' experts
constexpr int TOKEN_W = 16;

MOE_DEV __amdgpu_buffer_rsrc_t uniform_rsrc(const void *p, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  return make_rsrc((const void *)(uintptr_t)(((uint64_t)hi << 32) | lo), __builtin_amdgcn_readfirstlane(bytes));
}

// 16 + q of a word's eight codes, elements 0 .. 7
MOE_DEV bf16x8 unpack(uint32_t w) {
  // (in registers, so that and and or are one instruction: it takes no literals)
  uint32_t M = 0x00780078u, O = 0x41804180u;
  asm("" : "+s"(M));
  asm("" : "+v"(O));
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

// Buffers of one expert's codes, scales and zero points
struct Buffers {
  const void *w, *s, *z;
  uint32_t wn, sn, zn;  // bytes
  MOE_DEV static Buffers of(const Weight &p, int64_t e) {
    return Buffers{p.codes + e * p.per_codes, p.scales + e * p.per_scales, p.zeros + e * p.per_scales,
                   (uint32_t)p.per_codes, (uint32_t)(2 * p.per_scales), (uint32_t)p.per_scales};
  }
};

// One group's products and their sum into acc: v = sum (q - z) x of each row, from part, which holds sum (16 + q) x, or
// that less 24 sum x where there are no zero points
template <bool ZEROS>
MOE_DEV void add_group(f32x4 &acc, f32x4 part, f32x4 sum, float scale, float zero) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = fmaf(scale, ZEROS ? fmaf(-zero, sum[e], part[e]) : part[e], acc[e]);
}
MOE_DEV f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
template <bool ZEROS>
MOE_DEV bf16x8 sum_factor() {  // 1, or -24
  return all_of(ZEROS ? 0x3F803F80u : 0xC1C0C1C0u);
}

// byte, in its row, of the word with the codes of element k and the seven behind it (k a multiple of 8)
MOE_DEV uint32_t word_at(int k) { return (uint32_t)(k / BLK) * 64 + (k % 32 / 8) * 16 + (k % BLK / 32) * 4; }
MOE_DEV bool is_finite(float s) { return fabsf(s) < INFINITY; }

// x . W[n] of expert e by the formula itself, (q - z) s x, in fp32 (until it is NaN, which it stays).  For results that are not
// finite alone: one thread each, 0.2 us for a word (16 x 8192 x 8192 with an infinity in one row: 211 us, without 16).
template <int GP, bool ZEROS>
MOE_DEV float plain_sum(const Weight &p, int64_t e, int n, const bf16_t *x) {
  const uint8_t *codes = p.codes + e * p.per_codes + (int64_t)n * p.blocks * 64;
  const int64_t first = e * p.per_scales + n;
  float sum = 0.f;
  for (int k0 = 0; k0 < p.K && sum == sum; k0 += BLK) {
#pragma unroll 2
    for (int k = k0; k < min(k0 + BLK, p.K); k += 8) {
      const int64_t g = first + (int64_t)(k / (BLK / GP)) * p.cols;
      const uint32_t word = *(const uint32_t *)(codes + word_at(k));
      const u32x4 v = *(const u32x4 *)(x + k);
      const float s = bf16_to_f32(p.scales[g]), z = ZEROS ? (float)p.zeros[g] : 8.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        sum = fmaf(((float)(word >> (4 * ((i & 1) * 4 + i / 2)) & 15u) - z) * s,
                   __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16), sum);
    }
  }
  return sum;
}

// ---- some rows: 5 and more -------------------------------------------------------------
// The sums of 16 TI rows of x and 16 TJ columns over a wave's share of the blocks.  acc of lane l: column l & 15, rows 4
// (l >> 4) .. +3 (so that a lane needs one scale and one zero point).  GP: groups of a block.  Two blocks are in flight
// while one is multiplied; loads return in their order, so those of x are issued with the codes'.
// A block's offset is the loads' scalar one, which no bounds check sees: lanes of rows and columns that exist are inside
// their row at every whole block, the others out of range anyway, and a block that does not exist is loaded from a buffer
// of no bytes.
template <int TI, int TJ, int GP, bool ZEROS>
struct Wave {
  static constexpr int D = 2;
  u32x4 w[D][TJ], x[D][4][TI];
  uint32_t s[D][TJ], z[D][TJ];  // lane quarter q: of group q (q % 2, 0) of the block
  f32x4 acc[TI][TJ];
  uint32_t wo[TJ], so[TJ], xo[TI];

  // xo: byte offsets in x of the rows (l & 15 of each tile), out of range for none
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
  // whole block b to place d; TAIL: the last block, in which x ends, and the groups may
  template <bool TAIL>
  MOE_DEV void load(int d, const Weight &p, const Buffers &f, const void *xp, uint32_t xn, bool on, int b) {
    const int q = (int)((threadIdx.x & 63) >> 4);
    const auto rw = uniform_rsrc(f.w, on ? f.wn : 0), rs = uniform_rsrc(f.s, on ? f.sn : 0), rx = uniform_rsrc(xp, on ? xn : 0);
    const bool group = !TAIL || b * GP + (q & (GP - 1)) < p.groups;
    const uint32_t g = (uint32_t)(b * GP) * (uint32_t)p.cols;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      w[d][j] = __builtin_amdgcn_raw_buffer_load_b128(rw, wo[j], b * 64, 0);
      const bool in = group && so[j] < kOobOffset;
      s[d][j] = __builtin_amdgcn_raw_buffer_load_b16(rs, in ? 2 * so[j] : kOobOffset, 2 * g, 0);
      if constexpr (ZEROS) z[d][j] = __builtin_amdgcn_raw_buffer_load_b8(uniform_rsrc(f.z, on ? f.zn : 0), in ? so[j] : kOobOffset, g, 0);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const bool in = !TAIL || b * BLK + t * 32 + q * 8 < p.K;
        x[d][t][i] = __builtin_amdgcn_raw_buffer_load_b128(rx, in ? xo[i] + 64 * t : kOobOffset, b * 256, 0);
      }
  }
  MOE_DEV void multiply(int d) {
    constexpr int PER = 4 / GP;  // products of a group
    // Empty assembly keeps its order, one column tile and group after the other: the compiler begins all of them at once
    // otherwise, and spills their sums
    constexpr bool ORDER = GP * TI * TJ > 4;
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      f32x4 sum[TI];
      float none = 0.f;
      if constexpr (ORDER) asm volatile("" : "+v"(none));
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        sum[i] = f32x4{none, none, none, none};
#pragma unroll
        for (int t = 0; t < PER; ++t)
          sum[i] = mfma(__builtin_bit_cast(bf16x8, x[d][g * PER + t][i]), sum_factor<ZEROS>(), sum[i]);
      }
      const int from = ((threadIdx.x & 15) + 16 * g) * 4;  // the quarter that has this group's
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        f32x4 part[TI];
#pragma unroll
        for (int t = 0; t < PER; ++t) {
          uint32_t word = w[d][j][g * PER + t];
          if constexpr (ORDER) asm volatile("" : "+v"(word));
          const bf16x8 v = unpack(word);
#pragma unroll
          for (int i = 0; i < TI; ++i)
            part[i] = mfma(__builtin_bit_cast(bf16x8, x[d][g * PER + t][i]), v, t ? part[i] : ZEROS ? f32x4{} : sum[i]);
        }
        uint32_t sc = s[d][j], zc = ZEROS ? z[d][j] : 0;
        if constexpr (GP > 1) {
          sc = __builtin_amdgcn_ds_bpermute(from, sc);
          if constexpr (ZEROS) zc = __builtin_amdgcn_ds_bpermute(from, zc);
        }
        const float scale = __uint_as_float(sc << 16), zero = 16.f + (float)(zc & 0xffu);
#pragma unroll
        for (int i = 0; i < TI; ++i) {
          add_group<ZEROS>(acc[i][j], part[i], sum[i], scale, zero);
          if constexpr (ORDER) asm volatile("" : "+v"(acc[i][j]));
        }
      }
    }
  }
  // all of the wave's blocks; they begin at another place in each workgroup, since rows are often a power of two apart and
  // all workgroups on the same block would meet on few channels
  MOE_DEV void run(const Weight &p, const Buffers &f, const void *x, uint32_t xn, int n0, uint32_t place) {
    setup(p, n0);
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), whole = p.K / BLK;
    const int rot = whole ? (int)(place % (uint32_t)whole) : 0;
    // No branch around a load (the compiler could not count what is in flight, and would wait for all of it), and none
    // moved down to its use.
    auto fetch = [&](int d, int u) __attribute__((always_inline)) {
      const int b = u + rot;
      load<false>(d, p, f, x, xn, u < whole, u >= whole ? 0 : b >= whole ? b - whole : b);
    };
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, wid + d * WAVES);
    for (int u = wid; u < whole; u += D * WAVES) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        __builtin_amdgcn_sched_barrier(0);
        multiply(d);
        __builtin_amdgcn_sched_barrier(0);
        fetch(d, u + (D + d) * WAVES);
      }
    }
    if (whole < p.blocks && wid == whole % WAVES) {
      load<true>(0, p, f, x, xn, true, whole);
      multiply(0);
    }
  }
};

// The waves' sums of 16 rows (`rows` of them in use), added in wave order through red [WAVES][16][16 TJ + 4]; f(row, column,
// sum) for each
template <int TJ>
constexpr int kPitch = 16 * TJ + 4;
template <int TJ, class F>
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
  for (int e = threadIdx.x; e < min(rows, 16) * TN; e += WAVES * 64) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += red[(w * 16 + e / TN) * kPitch<TJ> + e % TN];
    f(e / TN, e % TN, v);
  }
}

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
template <typename To>
MOE_DEV void finish(const DenseArgs &a, int act, int m, int n, float s) {
  const int64_t at = (int64_t)m * a.w.N + n;
  if (a.bias) s += bf16_to_f32(a.bias[n]);
  s = act_fwd_of(act, s);
  if (a.res) s += ldf((const To *)a.res + at);
  stf((To *)a.out + at, s);
}

template <int TI, int TJ, int GP, bool ZEROS, typename To>
__global__ __launch_bounds__(WAVES * 64) void dense_kernel(DenseArgs a, int act) {
  __shared__ __align__(16) float red[WAVES * 16 * kPitch<TJ>];
  const int tm = (a.M + 16 * TI - 1) / (16 * TI);
  // the row tiles of one column tile are neighbours: its codes come from L2 from the second on
  const int m0 = blockIdx.x % tm * (16 * TI), n0 = blockIdx.x / tm * (16 * TJ);
  const int lane = threadIdx.x & 63;
  const Weight &p = a.w;
  Wave<TI, TJ, GP, ZEROS> v;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int r = i * 16 + (lane & 15);
    v.xo[i] = m0 + r < a.M ? (uint32_t)r * (uint32_t)p.K * 2 : kOobOffset;
  }
  v.run(p, Buffers::of(p, 0), a.x + (int64_t)m0 * p.K, (uint32_t)min(16 * TI, a.M - m0) * (uint32_t)p.K * 2, n0, blockIdx.x);
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int rows = a.M - m0 - i * 16;
    if (rows <= 0) break;
    join_waves<TJ>(red, v.acc[i], rows, [&](int r, int c, float s) {
      if (n0 + c >= p.N) return;
      const int m = m0 + i * 16 + r;
      if (!is_finite(s)) s = plain_sum<GP, ZEROS>(p, 0, n0 + c, a.x + (int64_t)m * p.K);
      finish<To>(a, act, m, n0 + c, s);
    });
  }
}

// ---- experts, through a schedule
struct ExpertArgs {
  Weight w;
  const bf16_t *x;
  float *y;
  const int32_t *counts, *offsets, *row_to_token;
  const float *row_weight;
  int T, layout, capacity, tn, e0;  // e0: first expert of the launch
};

template <int TI, int TJ, int GP, bool ZEROS>
MOE_DEV void expert_rows(const ExpertArgs &a, float *red, int e, int n0, int row0, int rows) {
  const int lane = threadIdx.x & 63;
  const Weight &p = a.w;
  Wave<TI, TJ, GP, ZEROS> v;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int r = i * 16 + (lane & 15), t = r < rows ? a.row_to_token[row0 + r] : -1;
    v.xo[i] = t >= 0 ? (uint32_t)t * (uint32_t)p.K * 2 : kOobOffset;
  }
  v.run(p, Buffers::of(p, e), a.x, (uint32_t)a.T * (uint32_t)p.K * 2, n0, blockIdx.x);
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    if (i * 16 >= rows) break;
    join_waves<TJ>(red, v.acc[i], rows - i * 16, [&](int r, int c, float s) {
      r += i * 16;
      if (n0 + c >= p.N) return;
      const int t = a.row_to_token[row0 + r];
      if (t < 0) return;
      if (!is_finite(s)) s = plain_sum<GP, ZEROS>(p, e, n0 + c, a.x + (int64_t)t * p.K);
      unsafeAtomicAdd(a.y + (int64_t)t * p.N + n0 + c, s * a.row_weight[row0 + r]);
    });
  }
}

// One workgroup per expert and column tile; an expert's rows 16 TI at a time (the last ones 16 if that will do), its
// codes then coming out of the caches.
template <int TI, int TJ, int GP, bool ZEROS>
__global__ __launch_bounds__(WAVES * 64) void expert_kernel(ExpertArgs a) {
  __shared__ __align__(16) float red[WAVES * 16 * kPitch<TJ>];
  const int e = a.e0 + blockIdx.x / a.tn, n0 = blockIdx.x % a.tn * (16 * TJ);
  const int count = __builtin_amdgcn_readfirstlane(a.counts[e]);
  const int first = a.layout == MOE_LAYOUT_MASKED ? e * a.capacity : __builtin_amdgcn_readfirstlane(a.offsets[e]) - count;
  for (int r = 0; r < count; r += 16 * TI) {
    if (TI > 1 && count - r <= 16) expert_rows<1, TJ, GP, ZEROS>(a, red, e, n0, first + r, count - r);
    else expert_rows<TI, TJ, GP, ZEROS>(a, red, e, n0, first + r, min(count - r, 16 * TI));
  }
}

// ---- experts, enough of them to fill the chip: no split of the reduction -------------------
// 16 columns per wave, 128 per workgroup, all waves at the same place of the reduction, whose rows of x they share
// in LDS (out of L2 they were as many bytes as the codes: 64 experts of 7168 x 2048 with 16 rows took 190 us).  A stage is
// two blocks of everything, so that codes are whole lines: x's rows, each wave's codes, scales and zero points, all by
// direct global->LDS loads (a wave waits for exactly the loads it has issued; nothing else is in flight), one stage ahead
// of the one that is multiplied, two workgroups per CU.
//
// One barrier per stage, after the wait for the own loads of the stage about to be read: then every wave's have landed,
// and every wave has read the stage before, whose place the loads issued next go into.
//
// Measured, 64 experts of 7168 x 2048, 6 to 26 rows each, us: groups of 32 125, of 128 110 (477 MB; without the
// arithmetic, for timing, 98).  Two or three stages ahead with one workgroup per CU 145-154 and 109; 16 waves of 16
// columns 132 and 111, 8 of 32 columns 136 and 108; stages of one block, half lines of codes, 143 and 137.
#define LDS_AS __attribute__((address_space(3)))
MOE_DEV void dma16(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  const uint32_t m0v = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(m0v), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}
// the same, for lines that nothing else reads
MOE_DEV void dma16_nt(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  const uint32_t m0v = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
               :
               : "s"(m0v), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}
MOE_DEV void dma4(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  const uint32_t m0v = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(m0v), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}

template <int TI, int GP, bool ZEROS>
struct Stream {
  static constexpr int G2 = 2 * GP;                               // groups of a stage
  static constexpr int XB = TI * 8192;                            // x: [16 TI][512 bytes]
  static constexpr int WB = 2048 + 256 + (ZEROS ? 256 : 0);       // a wave's codes, scales [G2][16], zeros [G2][16]
  static constexpr int STAGE = XB + WAVES * WB;
  static constexpr int XL = TI * 8 / WAVES;                    // a wave's loads of x
};

template <int TI, int GP, bool ZEROS>
MOE_DEV void stream_rows(const ExpertArgs &a, char *lds, int e, int n0, int row0, int rows) {
  using S = Stream<TI, GP, ZEROS>;
  constexpr int PER = 4 / GP;
  const Weight &p = a.w;
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
  const Buffers f = Buffers::of(p, e);
  const auto rw = uniform_rsrc(f.w, f.wn), rs = uniform_rsrc(f.s, f.sn), rx = uniform_rsrc(a.x, (uint32_t)a.T * (uint32_t)p.K * 2);
  const auto rz = uniform_rsrc(ZEROS ? f.z : f.s, ZEROS ? f.zn : 0);
  n0 += wid * 16;
  // x: 16-byte chunk c of row m at place c ^ (m & 15), so that the 16 rows of an operand read fall on 16 bank groups; a
  // load fills 2 rows, lane l place l & 31 of row l >> 5
  uint32_t xo[S::XL];
  int xk[S::XL];  // first reduction element of the lane's chunk in a stage
#pragma unroll
  for (int i = 0; i < S::XL; ++i) {
    const int m = (wid * S::XL + i) * 2 + (lane >> 5), c = (lane & 31) ^ (m & 15);
    const int t = m < rows ? a.row_to_token[row0 + m] : -1;
    xk[i] = c * 8;
    xo[i] = t >= 0 ? (uint32_t)t * (uint32_t)p.K * 2 + c * 16 : kOobOffset;
  }
  // codes: chunk c (of 8) of row n at place c ^ (n >> 1 & 7): the 16 rows of an operand read, two to a line of the
  // banks, fall on 16 bank groups; a load fills 8 rows, whole lines of memory
  uint32_t wo[2];
  const int wc = (lane & 7) ^ (lane >> 4);  // (n >> 1 & 7 of row 8 h + (lane >> 3) is 4 h + (lane >> 4))
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = n0 + h * 8 + (lane >> 3);
    wo[h] = n < p.N ? (uint32_t)n * ((uint32_t)p.blocks * 64) + (wc ^ (4 * h)) * 16 : kOobOffset;
  }
  // scales: lane l columns 2 (l & 7) .. of group l >> 3; zero points: columns 4 (l & 3) .. of group l >> 2.  (cols: whole 16s)
  const int sg = lane >> 3, sn = n0 + 2 * (lane & 7), zg = lane >> 2, zn = n0 + 4 * (lane & 3);
  const uint32_t so = sg < S::G2 && sn < p.cols ? 2 * ((uint32_t)sg * (uint32_t)p.cols + sn) : kOobOffset;
  const uint32_t zo = zg < S::G2 && zn < p.cols ? (uint32_t)zg * (uint32_t)p.cols + zn : kOobOffset;
  const uint32_t base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(LDS_AS char *)lds);
  const int stages = (p.blocks + 1) / 2, rot = (int)(blockIdx.x % (uint32_t)stages);
  auto issue = [&](int u, int slot) __attribute__((always_inline)) {
    const bool on = u < stages;
    const int b = !on ? 0 : u + rot >= stages ? u + rot - stages : u + rot;
    const uint32_t at = base + (uint32_t)slot * S::STAGE, mine = at + S::XB + wid * S::WB;
#pragma unroll
    for (int i = 0; i < S::XL; ++i)
      dma16(rx, on && b * 256 + xk[i] < p.K ? xo[i] : kOobOffset, b * 512, at + (wid * S::XL + i) * 1024);
#pragma unroll
    for (int h = 0; h < 2; ++h)  // (an odd number of blocks: the last stage has one)
      dma16_nt(rw, on && 2 * b + ((wc ^ (4 * h)) >> 2) < p.blocks ? wo[h] : kOobOffset, b * 128, mine + h * 1024);
    dma4(rs, on && b * S::G2 + sg < p.groups ? so : kOobOffset, 2 * b * S::G2 * p.cols, mine + 2048);
    if constexpr (ZEROS) dma4(rz, on && b * S::G2 + zg < p.groups ? zo : kOobOffset, b * S::G2 * p.cols, mine + 2304);
  };
  f32x4 acc[TI] = {};
  issue(0, 0);
  for (int u = 0; u < stages; ++u) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    issue(u + 1, (u + 1) & 1);
    const char *at = lds + (u & 1) * S::STAGE, *mine = at + S::XB + wid * S::WB;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      bf16x8 xv[TI][4];
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) xv[i][t] = *(const bf16x8 *)(at + (i * 16 + r) * 512 + (((b * 16 + t * 4 + q) ^ r) << 4));
      const u32x4 w = *(const u32x4 *)(mine + r * 128 + (((b * 4 + q) ^ (r >> 1)) << 4));
#pragma unroll
      for (int g = 0; g < GP; ++g) {
        f32x4 sum[TI], part[TI];
#pragma unroll
        for (int i = 0; i < TI; ++i) {
          sum[i] = f32x4{};
#pragma unroll
          for (int t = 0; t < PER; ++t) sum[i] = mfma(xv[i][g * PER + t], sum_factor<ZEROS>(), sum[i]);
        }
#pragma unroll
        for (int t = 0; t < PER; ++t) {
          const bf16x8 v = unpack(w[g * PER + t]);
#pragma unroll
          for (int i = 0; i < TI; ++i) part[i] = mfma(xv[i][g * PER + t], v, t ? part[i] : ZEROS ? f32x4{} : sum[i]);
        }
        const int of = (b * GP + g) * 16 + r;
        const float scale = bf16_to_f32(((const bf16_t *)(mine + 2048))[of]);
        const float zero = ZEROS ? 16.f + (float)((const uint8_t *)(mine + 2304))[of] : 0.f;
#pragma unroll
        for (int i = 0; i < TI; ++i) add_group<ZEROS>(acc[i], part[i], sum[i], scale, zero);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // loads of stages that are not there end before the LDS is used again, by whomever
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int e2 = 0; e2 < 4; ++e2) {
      const int m = i * 16 + 4 * q + e2;
      if (m >= rows) continue;
      const int t = a.row_to_token[row0 + m];
      if (t < 0) continue;
      const float weight = a.row_weight[row0 + m];
      if (n0 + r >= p.N) continue;
      float s = acc[i][e2];
      if (!is_finite(s)) s = plain_sum<GP, ZEROS>(p, e, n0 + r, a.x + (int64_t)t * p.K);
      unsafeAtomicAdd(a.y + (int64_t)t * p.N + n0 + r, s * weight);
    }
}

template <int GP, bool ZEROS>
__global__ __launch_bounds__(WAVES * 64, 4) void stream_kernel(ExpertArgs a) {
  extern __shared__ __align__(16) char lds[];
  const int e = a.e0 + blockIdx.x / a.tn, n0 = blockIdx.x % a.tn * (16 * WAVES);
  const int count = __builtin_amdgcn_readfirstlane(a.counts[e]);
  const int first = a.layout == MOE_LAYOUT_MASKED ? e * a.capacity : __builtin_amdgcn_readfirstlane(a.offsets[e]) - count;
  for (int r = 0; r < count; r += 32) {
    if (count - r <= 16) stream_rows<1, GP, ZEROS>(a, lds, e, n0, first + r, count - r);
    else stream_rows<2, GP, ZEROS>(a, lds, e, n0, first + r, min(count - r, 32));
  }
}

// ---- at most 4 rows, and single tokens through their experts ----------------------------------
// Rows of x in LDS, tiles of 8 columns: a load of codes is an operand as it comes, its 16 columns being the 8 of the
// first and the 8 of the second block of a pair; x's 16 rows are those of both blocks in turn (row r: r >> 1, block r &
// 1; rows that are not there repeat the first), and of the products' 16 x 16 sums those of one block with itself count.
// Since the other operand is in LDS, codes can be loaded D pairs ahead.
template <int TJ, int GP, bool ZEROS>
struct Few {
  static constexpr int D = 2;
  u32x4 w[D][TJ];
  uint32_t s[D][TJ], z[D][TJ];  // lane quarter q: of group q (q % 2, 0) of the lane's block
  f32x4 acc[TJ];
  uint32_t wo[TJ], so[TJ], xo;

  // x: LDS bytes of this wave's rows, pitch apart
  MOE_DEV void setup(const Weight &p, int n0, int rows, int pitch) {
    const int lane = threadIdx.x & 63, hb = lane >> 3 & 1, q = lane >> 4, m = (lane & 15) >> 1;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int n = n0 + j * 8 + (lane & 7);
      wo[j] = n < p.N ? (uint32_t)n * ((uint32_t)p.blocks * 64) + hb * 64 + q * 16 : kOobOffset;
      so[j] = n < p.N ? (uint32_t)(hb * GP + (q & (GP - 1))) * (uint32_t)p.cols + n : kOobOffset;
      acc[j] = f32x4{};
    }
    xo = (m < rows ? m : 0) * pitch + (lane & 1) * 256 + q * 16;
  }
  template <bool TAIL>
  MOE_DEV void load(int d, const Weight &p, const Buffers &f, bool on, int u) {
    const int lane = threadIdx.x & 63, hb = lane >> 3 & 1, q = lane >> 4;
    const auto rw = uniform_rsrc(f.w, on ? f.wn : 0), rs = uniform_rsrc(f.s, on ? f.sn : 0);
    const uint32_t g = (uint32_t)(u * 2 * GP) * (uint32_t)p.cols;
    const bool block = !TAIL || 2 * u + hb < p.blocks, group = !TAIL || (2 * u + hb) * GP + (q & (GP - 1)) < p.groups;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      w[d][j] = __builtin_amdgcn_raw_buffer_load_b128(rw, block ? wo[j] : kOobOffset, u * 128, 0);
      const bool in = group && so[j] < kOobOffset;
      s[d][j] = __builtin_amdgcn_raw_buffer_load_b16(rs, in ? 2 * so[j] : kOobOffset, 2 * g, 0);
      if constexpr (ZEROS) z[d][j] = __builtin_amdgcn_raw_buffer_load_b8(uniform_rsrc(f.z, on ? f.zn : 0), in ? so[j] : kOobOffset, g, 0);
    }
  }
  // weight: of the row's assignment, 1 without
  MOE_DEV void multiply(int d, const char *x, int u, float weight) {
    constexpr int PER = 4 / GP;
    bf16x8 xv[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) xv[t] = *(const bf16x8 *)(x + xo + u * 512 + t * 64);
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      f32x4 sum = {};
#pragma unroll
      for (int t = 0; t < PER; ++t) sum = mfma(xv[g * PER + t], sum_factor<ZEROS>(), sum);
      // (a quarter's sums of x are the same in every column)
      const int from = ((threadIdx.x & 15) + 16 * g) * 4;
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        f32x4 part = ZEROS ? f32x4{} : sum;
#pragma unroll
        for (int t = 0; t < PER; ++t) part = mfma(xv[g * PER + t], unpack(w[d][j][g * PER + t]), part);
        uint32_t sc = s[d][j], zc = ZEROS ? z[d][j] : 0;
        if constexpr (GP > 1) {  // from the quarter that has this group's
          sc = __builtin_amdgcn_ds_bpermute(from, sc);
          if constexpr (ZEROS) zc = __builtin_amdgcn_ds_bpermute(from, zc);
        }
        add_group<ZEROS>(acc[j], part, sum, __uint_as_float(sc << 16) * weight, 16.f + (float)(zc & 0xffu));
      }
    }
  }
};

// The sums of at most 4 rows and 8 TJ columns over the waves' two blocks each, in order; f(row, column, sum)
template <int TJ, int NW, class F>
MOE_DEV void join_few(float *red, const f32x4 (&acc)[TJ], int rows, F &&f) {  // red [2 NW][4][8 TJ]
  constexpr int TN = 8 * TJ;
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, hb = lane >> 3 & 1;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < TJ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 4 * (lane >> 4) + e, m = r >> 1;
      if ((r & 1) == hb && m < rows) red[((2 * wid + hb) * 4 + m) * TN + j * 8 + (lane & 7)] = acc[j][e];
    }
  __syncthreads();
  for (int e = threadIdx.x; e < rows * TN; e += NW * 64) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 2 * NW; ++w) v += red[w * 4 * TN + e];
    f(e / TN, e % TN, v);
  }
}

// rows of x [rows][K] to LDS, zeros up to a whole pair; pitch: their distance, 64 bytes apart on the banks
MOE_DEV int few_pitch(int K) { return (K + 2 * BLK - 1) / (2 * BLK) * 512 + 64; }
MOE_DEV void stage_rows(char *lds, const bf16_t *x, int rows, int K, int threads) {
  const int pitch = few_pitch(K), per = (pitch - 64) / 16;
  for (int c = threadIdx.x; c < rows * per; c += threads) {
    const int m = c / per, k = (c - m * per) * 8;
    *(u32x4 *)(lds + m * pitch + 2 * k) = k < K ? *(const u32x4 *)(x + (int64_t)m * K + k) : u32x4{};
  }
}

template <int TJ, int GP, bool ZEROS, typename To>
__global__ __launch_bounds__(WAVES * 64) void few_kernel(DenseArgs a, int act) {
  extern __shared__ __align__(16) char lds[];
  const Weight &p = a.w;
  const int n0 = blockIdx.x * (8 * TJ), wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pairs = p.K / (2 * BLK), rot = pairs ? (int)(blockIdx.x % (uint32_t)pairs) : 0;
  const Buffers f = Buffers::of(p, 0);
  using F = Few<TJ, GP, ZEROS>;
  constexpr int D = F::D;
  F v;
  v.setup(p, n0, a.M, few_pitch(p.K));
  auto place = [&](int u) __attribute__((always_inline)) { return u >= pairs ? 0 : u + rot >= pairs ? u + rot - pairs : u + rot; };
#pragma unroll
  for (int d = 0; d < D; ++d) v.template load<false>(d, p, f, wid + d * WAVES < pairs, place(wid + d * WAVES));
  stage_rows(lds, a.x, a.M, p.K, WAVES * 64);
  __syncthreads();
  for (int u = wid; u < pairs; u += D * WAVES) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int at = u + d * WAVES, next = at + D * WAVES;
      __builtin_amdgcn_sched_barrier(0);
      if (at < pairs) v.multiply(d, lds, place(at), 1.f);
      __builtin_amdgcn_sched_barrier(0);
      v.template load<false>(d, p, f, next < pairs, place(next));
    }
  }
  if (pairs * 2 * BLK < p.K && wid == pairs % WAVES) {
    v.template load<true>(0, p, f, true, pairs);
    v.multiply(0, lds, pairs, 1.f);
  }
  join_few<TJ, WAVES>((float *)lds, v.acc, a.M, [&](int r, int c, float s) {
    if (n0 + c >= p.N) return;
    if (!is_finite(s)) s = plain_sum<GP, ZEROS>(p, 0, n0 + c, a.x + (int64_t)r * p.K);
    finish<To>(a, act, r, n0 + c, s);
  });
}

struct TokenArgs {
  Weight w;
  const bf16_t *x;
  const int32_t *ids;
  const float *weights;
  float *y;
  int k, E, tn;
};

// A walk over the pairs of all of a token's experts, dealt to the waves in turn
struct Walk {
  int slot, u;
  MOE_DEV void go(int step, int pairs, int k) {
    u += step;
    while (u >= pairs && slot < k) {
      u -= pairs;
      ++slot;
    }
  }
};

// One workgroup per token and column tile: its waves share the pairs of all k experts, whose routing weights go into
// the scales; plain stores.  8 of 64 experts of 7168 x 2048, us: 18.1 with 16 waves and tiles of 8 columns, 20.8 with 8
// waves, 22.5 with tiles of 16 columns, 36 with x from memory.
template <int GP, bool ZEROS>
__global__ __launch_bounds__(TOKEN_W * 64) void token_kernel(TokenArgs a) {
  extern __shared__ __align__(16) char lds[];
  const Weight &p = a.w;
  const int64_t t = blockIdx.x / a.tn;
  const int n0 = (int)(blockIdx.x - t * a.tn) * 8, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pairs = p.K / (2 * BLK);
  using F = Few<1, GP, ZEROS>;
  constexpr int D = F::D;
  F v;
  v.setup(p, n0, 1, few_pitch(p.K));
  float weight[D];
  int at[D];  // -1: no expert
  // whether a slot has an expert
  auto slot_of = [&](int slot, Buffers &f, float &weight) __attribute__((always_inline)) {
    const int e = slot < a.k ? __builtin_amdgcn_readfirstlane(a.ids[t * a.k + slot]) : -1;
    const bool use = e >= 0 && e < a.E;
    f = Buffers::of(p, use ? e : 0);
    weight = use ? (a.weights ? a.weights[t * a.k + slot] : 1.f) : 0.f;
    return use;
  };
  Walk walk{0, 0};
  auto load = [&](int d) __attribute__((always_inline)) {
    Buffers f;
    const bool use = slot_of(walk.slot, f, weight[d]);
    at[d] = use ? walk.u : -1;
    v.template load<false>(d, p, f, use, use ? walk.u : 0);
    walk.go(TOKEN_W, pairs, a.k);
  };
  if (pairs) {
    walk.go(wid, pairs, a.k);
#pragma unroll
    for (int d = 0; d < D; ++d) load(d);
  }
  stage_rows(lds, a.x + t * p.K, 1, p.K, TOKEN_W * 64);
  __syncthreads();
  for (int u = wid; u < a.k * pairs; u += D * TOKEN_W) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      __builtin_amdgcn_sched_barrier(0);
      if (at[d] >= 0) v.multiply(d, lds, at[d], weight[d]);
      __builtin_amdgcn_sched_barrier(0);
      load(d);
    }
  }
  if (pairs * 2 * BLK < p.K) {
    for (int slot = wid; slot < a.k; slot += TOKEN_W) {
      Buffers f;
      float w;
      if (!slot_of(slot, f, w)) continue;
      v.template load<true>(0, p, f, true, pairs);
      v.multiply(0, lds, pairs, w);
    }
  }
  join_few<1, TOKEN_W>((float *)lds, v.acc, 1, [&](int, int c, float s) {
    if (n0 + c >= p.N) return;
    if (!is_finite(s)) {
      s = 0.f;
      for (int j = 0; j < a.k; ++j) {
        const int e = a.ids[t * a.k + j];
        if (e >= 0 && e < a.E)
          s = fmaf(a.weights ? a.weights[t * a.k + j] : 1.f, plain_sum<GP, ZEROS>(p, e, n0 + c, a.x + t * p.K), s);
      }
    }
    a.y[t * p.N + n0 + c] = s;
  });
}

// ---- codes from weights and back -------------------------------------------------------
// 8 elements per lane, G / 8 lanes per group; a wave takes 512 elements of a row.
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
    // (hi - lo may be past the largest number, a fifteenth of it is not)
    const float range = is_finite(hi - lo) ? (hi - lo) / 15.f : (hi * 0.0625f - lo * 0.0625f) / 15.f * 16.f;
    const float wide = zeros ? range : fmaxf(-lo, hi) / 7.f;
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

// more LDS than the default allows; the attribute is set once per device
template <auto KERNEL>
hipError_t allow_lds(size_t bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    e = hipFuncSetAttribute((const void *)KERNEL, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  }
  return e;
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

template <int TI, int TJ, typename To>
hipError_t run_dense(const moe_w4_weight &w, const DenseArgs &a, int act, hipStream_t st) {
  const int64_t tn = (w.N + 16 * TJ - 1) / (16 * TJ), M = a.M;
  // workgroups of one launch: below 2^31 work-items
  const int64_t most = (((int64_t)1 << 31) / (WAVES * 64) / tn - 1) * 16 * TI, run = M < most ? M : most;
  for (int64_t m = 0; m < M; m += run) {
    DenseArgs b = a;
    b.M = (int)(M - m < run ? M - m : run);
    b.x += m * w.K;
    b.out = (To *)a.out + m * w.N;
    if (a.res) b.res = (const To *)a.res + m * w.N;
    const int grid = (int)(tn * ((b.M + 16 * TI - 1) / (16 * TI)));
    by_form(w, [&](auto gp, auto z) {
      dense_kernel<TI, TJ, decltype(gp)::value, decltype(z)::value, To><<<grid, WAVES * 64, 0, st>>>(b, act);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// LDS of few_kernel and token_kernel: the rows, then the sums; 0 where that is over 64 KB
size_t few_lds(int rows, int64_t K, int NW, int TJ) {
  const size_t x = (size_t)rows * ((K + 2 * BLK - 1) / (2 * BLK) * 512 + 64), red = (size_t)2 * NW * 4 * 8 * TJ * 4;
  return x > 65536 ? 0 : x > red ? x : red;
}
template <int TJ, typename To>
hipError_t run_few(const moe_w4_weight &w, const DenseArgs &a, int act, hipStream_t st) {
  const int grid = (int)((w.N + 8 * TJ - 1) / (8 * TJ));
  by_form(w, [&](auto gp, auto z) {
    few_kernel<TJ, decltype(gp)::value, decltype(z)::value, To><<<grid, WAVES * 64, few_lds(a.M, w.K, WAVES, TJ), st>>>(a, act);
  });
  return hipGetLastError();
}

// Which kernel and tile: narrow columns while they leave CUs without a workgroup, wide ones (fewer rows of x to
// fetch for the codes) from then on.  us, groups of 128:
// At most 2 rows, 4 below 4096 columns, with x in LDS; M x K x N, tiles of 8, 16, 32 columns | dense of 16, 32:
//     1 x 8192 x 2048     5.0   5.9   8.3 |  6.5   8.4        4 x 8192 x 2048    7.0   8.1       |  7.9
//     1 x 4096 x 4096     5.4   5.2   6.6 |  4.8   5.9        3 x 4096 x 4096    5.8   5.6   7.1 |  5.2   6.2
//     1 x 8192 x 8192    11.3  10.1  10.6 | 13.4  10.1        3 x 8192 x 8192   15.6  11.6  12.0 | 14.0  10.6
//     1 x 8192 x 12288   15.2  13.2  14.5 | 18.4  17.8        3 x 8192 x 12288  19.5  14.9  16.2 | 19.8  18.4
//     1 x 8192 x 16384   20.1  17.4  15.9 | 23.2  18.5        3 x 8192 x 16384  24.8  19.6  17.5 | 24.9  19.2
// up to 16 rows, tiles of 16, 32 columns: 16 x 4096 x 4096 7.4 and 8.7, 16 x 8192 x 8192 21.7 and 14.5
// more, tiles of 32 rows and 32, 64 columns: 64 x 8192 x 4096 23.0 and 27.9, 64 x 8192 x 8192 44.1 and 29.1.
// (From some 256 rows on, 107 us for 256 x 8192 x 8192, weights are better dequantised for a matrix product.)
template <typename To>
hipError_t dense(const moe_w4_weight &w, const DenseArgs &a, int act, hipStream_t st) {
  const bool narrow = (w.N + 15) / 16 < 256;
  if (a.M <= (narrow ? 4 : 2) && few_lds(a.M, w.K, WAVES, 4)) {
    if (narrow) return run_few<1, To>(w, a, act, st);
    if ((w.N + 31) / 32 >= 512) return run_few<4, To>(w, a, act, st);
    return run_few<2, To>(w, a, act, st);
  }
  const int64_t tm = (a.M + 31) / 32;
  if (a.M > 16) {
    if (tm * ((w.N + 63) / 64) >= 256) return run_dense<2, 4, To>(w, a, act, st);
    return run_dense<2, 2, To>(w, a, act, st);
  }
  if ((w.N + 31) / 32 >= 256) return run_dense<1, 2, To>(w, a, act, st);
  return run_dense<1, 1, To>(w, a, act, st);
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
  // workgroups of one launch: at most 2^31 work-items
  auto by_experts = [&](int columns, auto &&launch) {
    a.tn = (a.w.N + columns - 1) / columns;
    const int run = (1 << 22) / a.tn;
    for (a.e0 = 0; a.e0 < s.E; a.e0 += run) {
      by_form(w, [&](auto gp, auto z) { launch(gp, z, a.tn * (s.E - a.e0 < run ? s.E - a.e0 : run)); });
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  };
  // 128 columns per workgroup where that leaves few CUs without one: 8 experts of 4096 x 2048 (128 workgroups) with 12 rows
  // each take 15.4 us by tiles of 32 columns and 19.2 so, 4 of 4096 x 7168 (224) 28.7 and 20.3, 16 of 4096 x 2048 (256)
  // 29.4 and 20.7, 64 105.9 and 59.8
  if ((int64_t)s.E * ((a.w.N + 127) / 128) >= 192)
    return by_experts(128, [&](auto gp, auto z, int grid) {
      constexpr int GP = decltype(gp)::value;
      constexpr bool Z = decltype(z)::value;
      hipError_t e = allow_lds<stream_kernel<GP, Z>>(2 * Stream<2, GP, Z>::STAGE);
      if (e == hipSuccess) stream_kernel<GP, Z><<<grid, WAVES * 64, 2 * Stream<2, GP, Z>::STAGE, st>>>(a);
    });
  // 16 rows at a time, or 32 where most experts have more than 16: 8 experts of 4096 x 2048 take 12.5 and 14.3 us with 4
  // rows each, 16.5 and 18.9 with 16, 30.2 and 27.8 with 32
  const bool few = s.S <= 16 * (int64_t)s.E;
  return by_experts(32, [&](auto gp, auto z, int grid) {
    constexpr int GP = decltype(gp)::value;
    constexpr bool Z = decltype(z)::value;
    if (few) expert_kernel<1, 2, GP, Z><<<grid, WAVES * 64, 0, st>>>(a);
    else expert_kernel<2, 2, GP, Z><<<grid, WAVES * 64, 0, st>>>(a);
  });
}

int64_t token_w4_width() { return (65536 - 64) / 512 * 2 * BLK; }
hipError_t launch_token_w4(const void *x, const moe_w4_weight &w, const int32_t *ids, const float *weights, int64_t T, int k, float *y,
                           hipStream_t st) {
  TokenArgs a{weight_of(w), (const bf16_t *)x, ids, weights, y, k, (int)w.E, 0};
  a.tn = (a.w.N + 7) / 8;
  const int64_t run = ((int64_t)1 << 31) / (TOKEN_W * 64) / a.tn;  // tokens of one launch
  for (int64_t t = 0; t < T; t += run) {
    TokenArgs b = a;
    b.x += t * w.K;
    b.ids += t * k;
    if (weights) b.weights += t * k;
    b.y += t * w.N;
    const int grid = (int)((T - t < run ? T - t : run) * a.tn);
    by_form(w, [&](auto gp, auto z) {
      token_kernel<decltype(gp)::value, decltype(z)::value><<<grid, TOKEN_W * 64, few_lds(1, w.K, TOKEN_W, 1), st>>>(b);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
