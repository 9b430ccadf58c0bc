// Routing to experts and the losses that keep a router balanced: from a row of
// logits to the expert ids and weights a schedule is built from, and back.
//
// All kernels are bound by reading or writing [T, E] once; what keeps them from
// it is the work per row.  LPR = 16 lanes (E <= 256; 32 up to 512, 64 up to 1024)
// share a row, V values each in registers, so a wave works on 64 / LPR rows and
// row-wide sums and maxima are 4 steps inside 16 lanes (data-parallel moves, no
// LDS) instead of 6 across the wave.  A wave per row, which the first kernels
// took, against this: routing 65536 x 256 with groups and bias 240 against 35 us,
// the routing gradient of 65536 x 128 27 against 14.3 (5.1 TB/s), the losses there
// 80 + 69 (join) + 22 against 10.8 + 10 + 15.
#include <type_traits>

#include "common.hpp"

namespace moe {
namespace {

constexpr int NT = 256, NW = NT / kWave;
constexpr int64_t kBarred = INT64_MIN;  // key of an expert (or group) that may not be chosen

MOE_DEV float ldf(const float *p) { return *p; }
MOE_DEV float ldf(const bf16_t *p) { return bf16_to_f32(*p); }
MOE_DEV void stf(float *p, float v) { *p = v; }
// rounds to nearest even and keeps a NaN a NaN (a gradient may hold one)
MOE_DEV void stf(bf16_t *p, float v) { *p = v != v ? (bf16_t)0x7FC0u : f32_to_bf16(v); }

MOE_DEV int64_t order_key(double c) {
  if (c != c) return INT64_MAX;
  const int64_t u = __builtin_bit_cast(int64_t, c + 0.0);  // -0 -> +0: equal values, equal keys
  return u >= 0 ? u : (int64_t)(~(uint64_t)u ^ 0x8000000000000000ull);
}
MOE_DEV double key_value(int64_t k) {
  if (k == INT64_MAX) return __builtin_nan("");
  return __builtin_bit_cast(double, k >= 0 ? k : (int64_t)(~((uint64_t)k ^ 0x8000000000000000ull)));
}

template <class T>
MOE_DEV T wave_sum(T v) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, kWave);
  return v;
}
MOE_DEV float wave_max(float v) {  // NaN is passed over
#pragma unroll
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, kWave));
  return v;
}

// ---- rows shared by LPR lanes ----------------------------------------------------
// data-parallel moves inside 16 lanes: exchange with the lane 1 and 2 away in the quad,
// mirrored in 8, mirrored in 16: after all four every lane has seen all 16
template <int CTRL>
MOE_DEV uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
MOE_DEV int64_t dpp64(int64_t x) {
  return (int64_t)(((uint64_t)dpp<CTRL>((uint32_t)((uint64_t)x >> 32)) << 32) | dpp<CTRL>((uint32_t)x));
}
template <int LPR, class Op>
MOE_DEV uint32_t row_reduce(uint32_t v, Op op) {
  v = op(v, dpp<0xB1>(v));
  v = op(v, dpp<0x4E>(v));
  v = op(v, dpp<0x141>(v));
  v = op(v, dpp<0x140>(v));
#pragma unroll
  for (int d = 16; d < LPR; d <<= 1) v = op(v, (uint32_t)__shfl_xor((int)v, d, kWave));
  return v;
}
MOE_DEV uint32_t f2u(float f) { return __float_as_uint(f); }
MOE_DEV float u2f(uint32_t u) { return __uint_as_float(u); }
template <int LPR>
MOE_DEV float row_sum(float v) {
  return u2f(row_reduce<LPR>(f2u(v), [](uint32_t a, uint32_t b) { return f2u(u2f(a) + u2f(b)); }));
}
template <int LPR>
MOE_DEV float row_max(float v) {  // NaN is passed over
  return u2f(row_reduce<LPR>(f2u(v), [](uint32_t a, uint32_t b) { return f2u(fmaxf(u2f(a), u2f(b))); }));
}
template <int LPR>
MOE_DEV uint32_t row_umax(uint32_t v) {
  return row_reduce<LPR>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int LPR>
MOE_DEV uint32_t row_umin(uint32_t v) {
  return row_reduce<LPR>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}

// Expert of a lane's value i: runs of C = min(V, 4) experts dealt to the row's lanes in turn.
template <int LPR, int V>
struct RowMap {
  static constexpr int C = V < 4 ? V : 4;
  MOE_DEV static int expert(int sub, int i) { return i / C * (C * LPR) + sub * C + i % C; }
};
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
MOE_DEV void ld4(const float *p, float (&v)[4]) {
  const f32x4 a = *(const f32x4 *)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = a[i];
}
MOE_DEV void ld4(const bf16_t *p, float (&v)[4]) {
  const u32x2 a = *(const u32x2 *)p;
  v[0] = u2f(a[0] << 16);
  v[1] = u2f(a[0] & 0xffff0000u);
  v[2] = u2f(a[1] << 16);
  v[3] = u2f(a[1] & 0xffff0000u);
}
MOE_DEV void st4(float *p, const float (&v)[4]) { *(f32x4 *)p = f32x4{v[0], v[1], v[2], v[3]}; }
MOE_DEV void st4(bf16_t *p, const float (&v)[4]) {
  typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
  *(bf16x4_t *)p = bf16x4_t{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
}
// a row's values, -inf past E; vec: E a multiple of 4 and rows on lines of four elements
template <int LPR, int V, typename T>
MOE_DEV void load_row(const T *row, int E, int sub, bool vec, float (&l)[V]) {
  using M = RowMap<LPR, V>;
  if constexpr (M::C == 4) {
    if (vec) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const int e = M::expert(sub, 4 * q);
        float v[4] = {-__builtin_inff(), -__builtin_inff(), -__builtin_inff(), -__builtin_inff()};
        if (e < E) ld4(row + e, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) l[4 * q + i] = v[i];
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = M::expert(sub, i);
    l[i] = e < E ? ldf(row + e) : -__builtin_inff();
  }
}
template <int LPR, int V, typename T>
MOE_DEV void store_row(T *row, int E, int sub, bool vec, const float (&d)[V]) {
  using M = RowMap<LPR, V>;
  if constexpr (M::C == 4) {
    if (vec) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const int e = M::expert(sub, 4 * q);
        const float v[4] = {d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]};
        if (e < E) st4(row + e, v);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = M::expert(sub, i);
    if (e < E) stf(row + e, d[i]);
  }
}
// exp through the hardware's exp2: log2(e) is off by 0.23 2^-24, its product with x is rounded once, and the
// instruction adds 2: relative error (1.23 |x| + 2) 2^-24
MOE_DEV float fexp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

struct RouteArgs {
  const void *logits;
  const float *bias;
  int32_t *ids;
  float *w;
  int64_t T;
  int E, k, G, keep;
  int sigmoid, top2, renorm;
  float scale;
  bool vec, vec_bias;  // load_row
  uint32_t per_magic;  // e * per_magic >> 20 = e / (E / G) for e < 1024 (2^20 > e (E / G - 1))
};

// LDS written by lanes of a wave, read by others of the same wave: the hardware keeps a wave's LDS
// accesses in order, the compiler has to as well
MOE_DEV void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// score of a logit relative to exp(shift): exp(l - shift) (softmax, shift = the
// row's or the chosen maximum) or sigmoid(l) exp(-shift) (shift = min(maximum,
// 0), so that a row of very negative logits keeps a nonzero sum)
MOE_DEV float shifted_score(float l, float shift, bool sigmoid) {
  if (!sigmoid) return fexp(l - shift);
  return fexp(fminf(l, 0.f) - shift) * __builtin_amdgcn_rcpf(1.f + fexp(-fabsf(l)));
}

// ---- the choice in 64 bits, by a whole wave --------------------------------------
// Experts are ranked by a 64-bit key that orders like the choice value with NaN above everything
// and an expert that may not be chosen below everything; equal keys go to the lower expert.  k
// rounds of wave-wide maximum take the k best; lane j returns slot j (-1: nothing left).
// lds: VPL * 64 + 64 keys of this wave (used with groups only).
template <typename T, int VPL>
MOE_DEV int choose_exact(const RouteArgs &p, const T *row, int64_t *lds, int lane) {
  int64_t *keys = lds, *gval = lds + VPL * 64;
  float l[VPL];
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < p.E ? ldf(row + e) : -__builtin_inff();
    m = fmaxf(m, l[i]);
  }
  m = wave_max(m);
  const bool scored = p.bias || (p.G > 1 && p.top2);
  int64_t key[VPL];
  double s[VPL];
  if (scored) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] = p.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i]))
                       : (l[i] == -__builtin_inff() ? 0.0 : exp((double)l[i] - (double)m));
      sum += s[i];
    }
    if (!p.sigmoid) {
      sum = wave_sum(sum);
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] /= sum;
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 64 + lane;
    const float b = p.bias && e < p.E ? p.bias[e] : 0.f;
    const bool barred = l[i] == -__builtin_inff() || b == -__builtin_inff();
    key[i] = barred ? kBarred : order_key(p.bias ? s[i] + (double)b : (double)l[i]);
  }
  if (p.G > 1) {
    const int per = p.E / p.G;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      keys[i * 64 + lane] = key[i] == kBarred ? kBarred : p.bias || !p.top2 ? key[i] : order_key(s[i]);
    wave_lds_sync();
    int64_t gk = kBarred;
    if (lane < p.G) {
      int64_t a = kBarred, b = kBarred;  // the two best
#pragma unroll 8
      for (int j = 0; j < per; ++j) {
        const int64_t v = keys[lane * per + j];
        if (v > a) { b = a; a = v; } else if (v > b) b = v;
      }
      gk = !p.top2 || b == kBarred ? a : order_key(key_value(a) + key_value(b));
      gval[lane] = gk;
    }
    wave_lds_sync();
    bool kept = false;
    if (lane < p.G && gk != kBarred) {
      int rank = 0;
      for (int g = 0; g < p.G; ++g) rank += gval[g] > gk || (gval[g] == gk && g < lane);
      kept = rank < p.keep;
    }
    const uint64_t mask = __ballot(kept);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int g = (i * 64 + lane) / per;
      if (g >= p.G || !((mask >> g) & 1)) key[i] = kBarred;
    }
    wave_lds_sync();
  }
  int id = -1;
  for (int j = 0; j < p.k; ++j) {
    int64_t best = kBarred;
    int at = INT32_MAX;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > best) { best = key[i]; at = i * 64 + lane; }
    auto take = [&](int64_t ok, int oa) __attribute__((always_inline)) {
      if (ok > best || (ok == best && oa < at)) { best = ok; at = oa; }
    };
    take(dpp64<0xB1>(best), (int)dpp<0xB1>(at));
    take(dpp64<0x4E>(best), (int)dpp<0x4E>(at));
    take(dpp64<0x141>(best), (int)dpp<0x141>(at));
    take(dpp64<0x140>(best), (int)dpp<0x140>(at));
    take(__shfl_xor(best, 16, kWave), __shfl_xor(at, 16, kWave));
    take(__shfl_xor(best, 32, kWave), __shfl_xor(at, 32, kWave));
    if (best == kBarred) break;
    if (lane == j) id = at;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (at == i * 64 + lane) key[i] = kBarred;
  }
  return id;
}

// weight of a lane's chosen expert (id, or -1) with logit lj, chosen experts in the first lanes of
// the LPR that share the row; m, sum: the row's maximum and sum of exp(l - m) (plain softmax);
// bad: a NaN if the row holds one (softmax), else 0
template <int LPR>
MOE_DEV float chosen_weight(const RouteArgs &p, int id, float lj, float m, float sum, float bad) {
  const bool on = id >= 0;
  float w;
  if (p.renorm) {
    const float mc = row_max<LPR>(on ? lj : -__builtin_inff());
    const float sj = on ? shifted_score(lj, p.sigmoid ? fminf(mc, 0.f) : mc, p.sigmoid) : 0.f;
    w = sj / (row_sum<LPR>(sj) + bad) * p.scale;
  } else if (p.sigmoid) {
    w = shifted_score(lj, 0.f, true) * p.scale;
  } else {
    w = fexp(lj - m) / sum * p.scale;
  }
  return on ? w : 0.f;
}

// ---- 64 / LPR rows per wave: E <= LPR V, k <= LPR, groups <= LPR ---------------------
// 32-bit keys that order like the choice value in fp32 (that of -inf: never chosen), in registers and in
// LDS by expert.  Every lane keeps the best of its V experts.  A round reduces the row's best and
// its expert over the lanes, strikes it out in LDS, and the lanes look at the struck owner's V
// values, one each, for the owner's new best: about 36 instructions a round for all rows of the
// wave, where striking out and searching again in registers takes 80.  65536 x 256, k = 8: 18.9 us by
// the logits (3.7 TB/s), 5.5 more for scores and bias, 8 for groups, 3 for rows chosen again.
//
// Without a bias the keys are the logits' own order: exact.  With one (and for groups by sums of
// scores) the values are fp32 approximations, u = 2^-24:
//   sigmoid: the exponential e is off by (1.23 |l| + 2) u, 1 + e by u, the reciprocal by 2 u:
//     s (1 - s) (1.23 |l| + 2) u + 3 s u, which is at most 5 u times the largest score of the row (times
//     1 - max l where that is below 0);
//   softmax: with x the distance from the maximum, its own rounding and the exponential's 2.23 x, and 30
//     more of the exponential, a sum 22 additions deep, the reciprocal and the product; the sum's terms
//     carry 2.23 x u each, weighted by their share at most 2.23 ln E = 15.5 u: e^-x (2.23 x + 15.5 + 30) u
//     <= 46 u times the largest score.
// Adding the bias rounds once more.  Where two values next to each other in the order are closer than
// their two errors, the slots' values are compared in 64 bits; where that does not settle it, or the
// groups on both sides of the cut are that close, or the row holds a NaN, the wave chooses that row
// again in 64 bits.  (Without the first step one row in about 1700 of 65536 x 256 is chosen again,
// which costs 3 us of 39: the last waves wait for it.)
MOE_DEV uint32_t key32(float c) {
  const uint32_t u = f2u(c + 0.f);  // -0 -> +0
  return c != c ? 0xFFFFFFFFu : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
MOE_DEV uint32_t key32_number(float c) {  // of a number, and of no -0
  const uint32_t u = f2u(c);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
MOE_DEV float key32_value(uint32_t k) {
  return k == 0xFFFFFFFFu ? __builtin_nanf("") : u2f((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// What the fp32 keys are: the logits' own; score + bias; the logits', with groups ranked by scores.
enum { BY_LOGIT = 0, BY_BIASED = 1, GROUPS_BY_SCORE = 2 };
constexpr uint32_t kBarred32 = 0x007FFFFFu;  // key of -inf

// the keys of a lane to the row's table in LDS (by expert)
template <int LPR, int V>
MOE_DEV void put_keys(uint32_t *keys, int sub, const uint32_t (&key)[V]) {
  using M = RowMap<LPR, V>;
  if constexpr (M::C == 4) {
#pragma unroll
    for (int q = 0; q < V / 4; ++q)
      *(u32x4 *)(keys + M::expert(sub, 4 * q)) = u32x4{key[4 * q], key[4 * q + 1], key[4 * q + 2], key[4 * q + 3]};
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) keys[M::expert(sub, i)] = key[i];
  }
}

template <typename T, int LPR, int V, int MODE>
__global__ __launch_bounds__(NT) void route_kernel(RouteArgs p) {
  using M = RowMap<LPR, V>;
  constexpr int RPW = 64 / LPR, EP = LPR * V;   // rows per wave, experts (padded)
  constexpr int PITCH = EP + 16;                // keys per row: the rows of a wave on other banks
  constexpr int XV = (EP + 63) / 64;            // values per lane of a whole wave
  constexpr int WORDS = RPW * PITCH > 2 * (XV * 64 + 64) ? RPW * PITCH : 2 * (XV * 64 + 64);
  __shared__ __align__(16) uint32_t smem[NW * WORDS];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int sub = lane & (LPR - 1), rw = lane / LPR;
  uint32_t *const keys = smem + wid * WORDS + rw * PITCH;
  const int64_t t = ((int64_t)blockIdx.x * NW + wid) * RPW + rw;
  const bool live = t < p.T;
  const T *row = (const T *)p.logits + (live ? t : 0) * p.E;
  float l[V];
  load_row<LPR, V>(row, p.E, sub, p.vec, l);
  float m = 0.f, sum = 0.f;  // the softmax's maximum and sum, and the maximum for the error bound
  if (MODE != BY_LOGIT || !(p.sigmoid || p.renorm)) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
    m = row_max<LPR>(m);
    if (!p.sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) sum += l[i] == -__builtin_inff() ? 0.f : fexp(l[i] - m);
      sum = row_sum<LPR>(sum);
    }
  }
  float bad = 0.f;  // a NaN if the row holds one
  if (p.renorm && !p.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) bad += l[i] != l[i] ? l[i] : 0.f;
    bad = row_sum<LPR>(bad);
  }
  uint32_t key[V];
  float err = 0.f;  // of two scores together
  bool doubt = false;
  if constexpr (MODE == BY_LOGIT) {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = key32(l[i]);
  } else {
    const float inv = __builtin_amdgcn_rcpf(sum);
    float nan = 0.f, c[V];
    if (p.sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = __builtin_amdgcn_rcpf(1.f + fexp(-l[i]));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = fexp(l[i] - m) * inv;
    }
    if constexpr (MODE == BY_BIASED) {
      float bs[V];
      load_row<LPR, V>(p.bias, p.E, sub, p.vec_bias, bs);
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] += bs[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = l[i] == -__builtin_inff() ? -__builtin_inff() : c[i];
      nan += c[i];
      key[i] = key32_number(c[i]);
    }
    const float top = p.sigmoid ? __builtin_amdgcn_rcpf(1.f + fexp(-m)) : inv;
    err = 2.f * top * (p.sigmoid ? 5.f * (1.f + fmaxf(-m, 0.f)) : 46.f) * 0x1p-24f;
    nan = row_sum<LPR>(nan);  // (of -inf and +inf too)
    doubt = nan != nan;
  }
  if (p.G > 1) {
    const int per = p.E / p.G;
    put_keys<LPR, V>(keys, sub, key);
    if constexpr (MODE == GROUPS_BY_SCORE) {
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = key32(l[i]);
    }
    wave_lds_sync();
    // lanes g, g + G', ... of the row scan group g (G' = the power of two above G - 1)
    int gp = 1;
    while (gp < p.G) gp <<= 1;
    const int g = sub & (gp - 1), part = sub / gp, parts = LPR / gp;
    uint32_t a = 0, b = 0;  // the two best
    if (g < p.G)
#pragma unroll 8
      for (int j = part; j < per; j += parts) {
        const uint32_t v = keys[g * per + j];
        b = max(b, min(a, v));
        a = max(a, v);
      }
    for (int d = gp; d < LPR; d <<= 1) {
      const uint32_t oa = __shfl_xor(a, d, kWave), ob = __shfl_xor(b, d, kWave);
      b = max(min(a, oa), max(b, ob));
      a = max(a, oa);
    }
    const bool two = p.top2 && b > kBarred32;
    const float fa = key32_value(a), fb = two ? key32_value(b) : 0.f;
    const uint32_t gv = two ? key32(fa + fb) : a;
    // rank of the lane's group; the kept one of lowest value and the best of the others
    int rank = 0;
    for (int d = 0; d < p.G; ++d) {
      const uint32_t o = __shfl(gv, d, LPR);
      rank += o > gv || (o == gv && d < g);
    }
    const bool kept = g < p.G && gv > kBarred32 && rank < p.keep;
    if (MODE != BY_LOGIT && p.keep < p.G) {
      const float lo = key32_value(row_umin<LPR>(kept ? gv : 0xFFFFFFFFu));
      const uint32_t hi = row_umax<LPR>(kept || g >= p.G ? 0u : gv);
      // one score each (and the value's rounding), or two (and each value's and the sum's)
      const float mag = row_max<LPR>(g < p.G && a > kBarred32 ? fabsf(fa) + fabsf(fb) : 0.f);
      doubt |= hi > kBarred32 && !(lo - key32_value(hi) > (p.top2 ? 2.f * err + mag * 0x1p-22f : err + mag * 0x1p-23f));
    }
    using Mask = std::conditional_t<LPR == 64, uint64_t, uint32_t>;
    const Mask mask = (Mask)(__ballot(kept && sub < gp) >> (lane & ~(LPR - 1)));
    if (M::C == 4 && per % 4 == 0) {
#pragma unroll
      for (int q = 0; q < (V + 3) / 4; ++q) {
        const int e = M::expert(sub, 4 * q < V ? 4 * q : 0);
        const bool in = e < p.E && ((mask >> (__umul24(e, p.per_magic) >> 20)) & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * q + i < V) key[4 * q + i] = in ? key[4 * q + i] : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = M::expert(sub, i);
        if (e >= p.E || !((mask >> (__umul24(e, p.per_magic) >> 20)) & 1)) key[i] = 0u;
      }
    }
    wave_lds_sync();
  }
  put_keys<LPR, V>(keys, sub, key);
  uint32_t best = kBarred32, at = 0xFFFFFFFFu;  // the lane's best key, and its expert
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (key[i] > best) { best = key[i]; at = M::expert(sub, i); }
  wave_lds_sync();
  int id = -1;
  uint32_t won = 0;  // key of the lane's slot
  for (int j = 0; j < p.k; ++j) {
    const uint32_t mx = row_umax<LPR>(best);
    const uint32_t e = row_umin<LPR>(best == mx ? at : 0xFFFFFFFFu);
    const bool hit = mx > kBarred32;
    if (sub == j && hit) {
      id = (int)e;
      won = mx;
    }
    const int owner = hit ? (int)(e / M::C) & (LPR - 1) : 0;
    if (hit && sub == 0) keys[e] = 0u;
    wave_lds_sync();
    const int oe = M::expert(owner, sub & (V - 1));
    const uint32_t v = keys[oe];
    const uint32_t nb = row_umax<LPR>(v);
    const uint32_t ne = row_umin<LPR>(v == nb ? (uint32_t)oe : 0xFFFFFFFFu);
    if (hit && sub == owner) { best = nb; at = ne; }
  }
  if constexpr (MODE != BY_LOGIT) {
    if (MODE == BY_BIASED) {  // each slot's value against the next one's, the last against the best one left
      const uint32_t left = row_umax<LPR>(best);
      uint32_t next = __shfl_down(won, 1, LPR);
      if (sub == p.k - 1) next = left;
      const float hi = key32_value(won), lo = key32_value(next);
      bool soft = sub < p.k && next > kBarred32 && !(hi - lo > err + (fabsf(hi) + fabsf(lo)) * 0x1p-24f);
      if (__any(soft)) {
        // most of these are in order all the same: each slot's value in 64 bits against the next slot's,
        // the last's against the most that the best one left, and so any other, can be
        double c = 0.0;
        if (p.sigmoid) {
          if (id >= 0) c = 1.0 / (1.0 + exp(-(double)ldf(row + id))) + (double)p.bias[id];
        } else {
          double all = 0.0;
#pragma unroll
          for (int i = 0; i < V; ++i) all += l[i] == -__builtin_inff() ? 0.0 : exp((double)l[i] - (double)m);
#pragma unroll
          for (int d = 1; d < LPR; d <<= 1) all += __shfl_xor(all, d, kWave);
          if (id >= 0) c = exp((double)ldf(row + id) - (double)m) / all + (double)p.bias[id];
        }
        const double cn = __shfl_down(c, 1, LPR);
        const int idn = __shfl_down(id, 1, LPR);
        const bool ok = sub == p.k - 1 ? c > (double)lo + 0.5 * err + fabsf(lo) * 0x1p-24
                                       : c > cn || (c == cn && id < idn);
        soft = soft && !ok;
      }
      doubt |= soft;
    }
    // every lane of a row has the same doubt
    doubt = row_umax<LPR>(doubt) != 0u;
    uint64_t again = __ballot(doubt && live && sub == 0);
    while (again) {
      const int r = (__ffsll((unsigned long long)again) - 1) / LPR;
      again &= again - 1;
      const int64_t tr = ((int64_t)blockIdx.x * NW + wid) * RPW + r;
      const int x = choose_exact<T, XV>(p, (const T *)p.logits + tr * p.E, (int64_t *)(smem + wid * WORDS), lane);
      const int mine = __shfl(x, sub, kWave);
      if (rw == r) id = mine;
    }
  }
  const float w = chosen_weight<LPR>(p, id, id >= 0 ? ldf(row + id) : 0.f, m, sum, bad);
  if (live && sub < p.k) {
    p.ids[t * p.k + sub] = id;
    p.w[t * p.k + sub] = w;
  }
}

struct RouteBwdArgs {
  const float *g;
  const void *logits;
  const int32_t *ids;
  const float *w;
  void *d;
  int64_t T;
  int E, k, sigmoid, renorm;
  float scale;
  bool vec;
};

// g_j = dL/dw_j.  With D = sum_j g_j w_j:
//   renormalised: dl_j = w_j (g_j - D / scale), times 1 - s_j for the sigmoid;
//   plain softmax: dl_i = w_i g_i [i chosen] - p_i D;  plain sigmoid: dl_j = g_j w_j (1 - s_j).
template <typename T, int LPR, int V>
__global__ __launch_bounds__(NT) void route_bwd_kernel(RouteBwdArgs p) {
  using M = RowMap<LPR, V>;
  constexpr int RPW = 64 / LPR, EP = LPR * V, NS = 64 / LPR;  // NS: slots per lane (k <= 64)
  __shared__ __align__(16) float rows[NW * RPW * EP];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int sub = lane & (LPR - 1), rw = lane / LPR;
  float *buf = rows + (wid * RPW + rw) * EP;
  const int64_t t = ((int64_t)blockIdx.x * NW + wid) * RPW + rw;
  const bool live = t < p.T;
  const T *row = (const T *)p.logits + (live ? t : 0) * p.E;
  const bool dense = !p.renorm && !p.sigmoid;
  float l[V], m = -__builtin_inff();
  if (dense) load_row<LPR, V>(row, p.E, sub, p.vec, l);
  int id[NS];
  float w[NS], g[NS], D = 0.f;
#pragma unroll
  for (int q = 0; q < NS; ++q) {
    const int j = q * LPR + sub;
    id[q] = live && j < p.k ? p.ids[t * p.k + j] : -1;
    if (id[q] >= p.E) id[q] = -1;
    w[q] = id[q] >= 0 ? p.w[t * p.k + j] : 0.f;
    g[q] = id[q] >= 0 ? p.g[t * p.k + j] : 0.f;
    D += g[q] * w[q];
  }
  D = row_sum<LPR>(D);
#pragma unroll
  for (int i = 0; i < V; ++i) buf[M::expert(sub, i)] = 0.f;
  wave_lds_sync();
#pragma unroll
  for (int q = 0; q < NS; ++q) {
    if (id[q] < 0) continue;
    float c = w[q] * (p.renorm ? g[q] - D / p.scale : g[q]);
    if (p.sigmoid) c *= shifted_score(-ldf(row + id[q]), 0.f, true);  // 1 - s = sigmoid(-l)
    atomicAdd(&buf[id[q]], c);  // ids of one row differ; repeated ones add up
  }
  wave_lds_sync();
  float d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = buf[M::expert(sub, i)];
  if (dense) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
    m = row_max<LPR>(m);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] = l[i] == -__builtin_inff() ? 0.f : fexp(l[i] - m);
      sum += l[i];
    }
    sum = row_sum<LPR>(sum);
    const float f = sum > 0.f || sum != sum ? D / sum : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] -= l[i] * f;
  }
  if (live) store_row<LPR, V>((T *)p.d + t * p.E, p.E, sub, p.vec, d);
}

// ---- losses --------------------------------------------------------------------
// Forward: every block sums its rows' probabilities and counts its ids per
// expert, and its rows' squared log-sum-exps; one block joins the partial sums in
// a fixed order.  Workspace: [blocks][sums, counts], E of each padded to a multiple of 4, then
// [blocks][sum of squared log-sum-exps, rows].
constexpr int kLossBlocks = 256;   // partial sums that one workgroup then reads (E = 128: 264 KB)
constexpr int LT = 1024, LW = LT / kWave;

struct LossArgs {
  const void *logits;
  const int32_t *ids;
  float *part;
  float *losses, *stats;
  const float *dloss;
  void *d;
  int64_t T;
  int E, k, sigmoid, blocks;
  bool vec;
};

// soft[]: the softmax of a row; q[]: its probabilities (the softmax, or the sigmoids over their
// sum); lse.  An empty row (every logit -inf) gives zeros and false.
template <int LPR, int V>
MOE_DEV bool row_probs(const float (&l)[V], bool sigmoid, float (&soft)[V], float (&q)[V], float &lse) {
  float m = -__builtin_inff();
  float any = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    m = fmaxf(m, l[i]);
    any = l[i] != -__builtin_inff() ? 1.f : any;  // a NaN counts
  }
  const bool some = row_max<LPR>(any) != 0.f;
  m = row_max<LPR>(m);
  float sum = 0.f, qsum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool off = l[i] == -__builtin_inff();
    soft[i] = off ? 0.f : fexp(l[i] - m);
    sum += soft[i];
    if (sigmoid) {
      q[i] = off ? 0.f : shifted_score(l[i], fminf(m, 0.f), true);
      qsum += q[i];
    }
  }
  sum = row_sum<LPR>(sum);
  lse = some ? m + logf(sum) : 0.f;
  const float inv = some ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) soft[i] *= inv;
  if (sigmoid) {
    qsum = row_sum<LPR>(qsum);
    const float qinv = some ? 1.f / qsum : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] *= qinv;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = soft[i];
  }
  return some;
}

// Every lane sums its own V experts over the block's rows; the row groups of a wave and the waves
// join through LDS.
template <typename T, int LPR, int V>
__global__ __launch_bounds__(LT) void loss_fwd_kernel(LossArgs p) {
  using M = RowMap<LPR, V>;
  constexpr int RPW = 64 / LPR, EP = LPR * V;
  __shared__ float psum[LW][EP];  // <= 64 KB (EP <= 1024)
  __shared__ int cnt[EP];
  __shared__ float zs[LW];
  __shared__ int rs[LW];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int sub = lane & (LPR - 1), rw = lane / LPR;
  for (int e = threadIdx.x; e < EP; e += LT) cnt[e] = 0;
  __syncthreads();
  float acc[V] = {}, z = 0.f;
  int rows = 0;
  const int64_t step = (int64_t)gridDim.x * LW * RPW;
  // a block takes runs of LW * RPW consecutive rows
  for (int64_t t0 = (int64_t)blockIdx.x * LW * RPW; t0 < p.T; t0 += step) {
    const int64_t t = t0 + wid * RPW + rw;
    if (t < p.T) {  // (whole rows: the lanes that share one go together)
      float l[V], soft[V], q[V], lse;
      load_row<LPR, V>((const T *)p.logits + t * p.E, p.E, sub, p.vec, l);
      rows += row_probs<LPR, V>(l, p.sigmoid, soft, q, lse);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += q[i];
      z += lse * lse;
    }
    const int64_t i0 = t0 * p.k, i1 = min(p.T, t0 + LW * RPW) * p.k;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += LT) {
      const int id = p.ids[i];
      if (id >= 0 && id < p.E) atomicAdd(&cnt[id], 1);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int d = LPR; d < 64; d <<= 1) acc[i] += __shfl_xor(acc[i], d, kWave);
    if (rw == 0) psum[wid][M::expert(sub, i)] = acc[i];
  }
#pragma unroll
  for (int d = LPR; d < 64; d <<= 1) {
    z += __shfl_xor(z, d, kWave);
    rows += __shfl_xor(rows, d, kWave);
  }
  if (lane == 0) { zs[wid] = z; rs[wid] = rows; }
  __syncthreads();
  // this block's part: sums, then counts, each padded to a multiple of 4
  const int pad = (p.E + 3) & ~3;
  float *part = p.part + (size_t)blockIdx.x * 2 * pad;
  for (int e = threadIdx.x; e < pad; e += LT) {
    float v = 0.f;
    if (e < p.E)
#pragma unroll
      for (int w = 0; w < LW; ++w) v += psum[w][e];
    part[e] = v;
    part[pad + e] = __int_as_float(e < p.E ? cnt[e] : 0);
  }
  if (threadIdx.x == 0) {
    float v = 0.f;
    int r = 0;
    for (int w = 0; w < LW; ++w) { v += zs[w]; r += rs[w]; }
    float *tail = p.part + (size_t)gridDim.x * 2 * pad + 2 * blockIdx.x;
    tail[0] = v;
    tail[1] = __int_as_float(r);
  }
}

// Sums over the block of two values per thread, in a fixed order.
MOE_DEV void block_sums(double &x, double &y, double *red) {
  x = wave_sum(x);
  y = wave_sum(y);
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (lane == 0) {
    red[w] = x;
    red[LW + w] = y;
  }
  __syncthreads();
  x = red[lane & (LW - 1)];
  y = red[LW + (lane & (LW - 1))];
#pragma unroll
  for (int d = LW / 2; d; d >>= 1) {
    x += __shfl_xor(x, d, kWave);
    y += __shfl_xor(y, d, kWave);
  }
  __syncthreads();
}

// Sums runs of the blocks' parts into kLossParts parts of the same form: workgroup (x, y) 64 of the 16-byte
// words (4 threads each) of the y-th run.  Taken where one workgroup would read more than 272 KB: E = 1024
// at 16384 rows 55 -> 26 us for the forward, E = 512 at 32768 38 -> 26, E = 256 at 65536 30 -> 27.5; E = 128 (256 KB)
// gains nothing.
constexpr int kLossParts = 8;
__global__ __launch_bounds__(256) void loss_sum_kernel(LossArgs p, float *out) {
  __shared__ f32x4 red[4][64];
  const int pad = (p.E + 3) & ~3, words = pad / 2;
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), q = threadIdx.x >> 6;
  const int lo = p.blocks * blockIdx.y / kLossParts, hi = p.blocks * (blockIdx.y + 1) / kLossParts;
  const bool counts = c >= pad / 4;
  f32x4 acc = {};
  auto add = [&](f32x4 a, f32x4 b) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = counts ? __int_as_float(__float_as_int(a[i]) + __float_as_int(b[i])) : a[i] + b[i];
    return a;
  };
  if (c < words)
#pragma unroll 8
    for (int b = lo + q; b < hi; b += 4) acc = add(acc, ((const f32x4 *)p.part)[(size_t)b * words + c]);
  red[q][threadIdx.x & 63] = acc;
  __syncthreads();
  if (q == 0 && c < words) {
#pragma unroll
    for (int i = 1; i < 4; ++i) acc = add(acc, red[i][threadIdx.x & 63]);
    ((f32x4 *)out)[(size_t)blockIdx.y * words + c] = acc;
  }
}

// One workgroup joins the blocks' parts, 16 bytes per load: W threads (the power of two from a part's
// words / 4 up) side by side on a part, the LT / W others take every (LT / W)-th part; then a tree over
// those.  In 64 bits (the counts too, which it holds exactly).
// sums: `parts` parts of sums and counts (the blocks' own, or loss_sum_kernel's).
__global__ __launch_bounds__(LT) void loss_join_kernel(LossArgs p, const float *sums_in, int parts) {
  typedef double f64x4 __attribute__((ext_vector_type(4)));
  __shared__ f64x4 sums[LT];
  __shared__ double red[2 * LW];
  const int tid = threadIdx.x, pad = (p.E + 3) & ~3, words = pad / 2;  // 16-byte words of a part
  int W = 1;
  while (W < words) W <<= 1;
  const int c = tid & (W - 1), q = tid / W, Q = LT / W;
  f64x4 acc = {};
  if (c < words) {
    const f32x4 *src = (const f32x4 *)sums_in + c;
    // 8 loads in flight (past the last part: the last one again, not added)
    for (int b0 = q; b0 < parts; b0 += 8 * Q) {
      f32x4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = src[(size_t)min(b0 + j * Q, parts - 1) * words];
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double x = c < pad / 4 ? (double)v[j][i] : (double)__float_as_int(v[j][i]);
          acc[i] += b0 + j * Q < parts ? x : 0.0;
        }
    }
  }
  double z = 0.0, r = 0.0;
  if (tid < p.blocks) {
    const float *tail = p.part + (size_t)p.blocks * 2 * pad + 2 * tid;
    z = tail[0];
    r = (double)__float_as_int(tail[1]);
  }
  sums[tid] = acc;
  for (int d = Q / 2; d; d >>= 1) {
    __syncthreads();
    if (q < d) {
      acc += sums[tid + d * W];
      sums[tid] = acc;
    }
  }
  __syncthreads();
  const double *flat = (const double *)sums;  // [pad] sums, [pad] counts
  const bool mine = tid < p.E;
  const double P = mine ? flat[tid] : 0.0, n = mine ? flat[pad + tid] : 0.0;
  double C = n;
  block_sums(C, r, red);
  const double inv = r > 0.0 ? 1.0 / r : 0.0;
  const float f = C > 0.0 ? (float)((double)p.E * n / C) : 0.f;
  if (mine) p.stats[tid] = f;
  double bal = (double)f * P;
  block_sums(bal, z, red);
  if (tid == 0) {
    p.stats[p.E] = (float)inv;
    p.losses[0] = (float)(bal * inv);
    p.losses[1] = (float)(z * inv);
  }
}
static_assert(kLossBlocks <= LT, "a thread per part");

template <typename T, int LPR, int V>
__global__ __launch_bounds__(NT) void loss_bwd_kernel(LossArgs p) {
  using M = RowMap<LPR, V>;
  constexpr int RPW = 64 / LPR;
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int sub = lane & (LPR - 1), rw = lane / LPR;
  const float inv = p.stats[p.E];
  const float gb = p.dloss[0] * inv, gz = 2.f * p.dloss[1] * inv;
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = M::expert(sub, i) < p.E ? p.stats[M::expert(sub, i)] : 0.f;
  for (int64_t t = ((int64_t)blockIdx.x * NW + wid) * RPW + rw; t < p.T; t += (int64_t)gridDim.x * NW * RPW) {
    float l[V], soft[V], q[V], lse, dot = 0.f;
    load_row<LPR, V>((const T *)p.logits + t * p.E, p.E, sub, p.vec, l);
    row_probs<LPR, V>(l, p.sigmoid, soft, q, lse);
#pragma unroll
    for (int i = 0; i < V; ++i) dot += f[i] * q[i];
    dot = row_sum<LPR>(dot);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float d = gb * q[i] * (f[i] - dot);
      if (p.sigmoid && l[i] != -__builtin_inff()) d *= shifted_score(-l[i], 0.f, true);
      l[i] = d + gz * lse * soft[i];
    }
    store_row<LPR, V>((T *)p.d + t * p.E, p.E, sub, p.vec, l);
  }
}

// f(integral_constant<LPR>, integral_constant<V>) for E experts and at least `lanes` lanes a row
template <int LPR, class F>
void by_values(int E, F &&f) {
  using std::integral_constant;
  const integral_constant<int, LPR> l;
  if (E <= LPR) f(l, integral_constant<int, 1>());
  else if (E <= 2 * LPR) f(l, integral_constant<int, 2>());
  else if (E <= 4 * LPR) f(l, integral_constant<int, 4>());
  else if (E <= 8 * LPR) f(l, integral_constant<int, 8>());
  else f(l, integral_constant<int, 16>());
}
template <class F>
hipError_t by_width(int E, int lanes, F &&f) {
  if (E <= 256 && lanes <= 16) by_values<16>(E, f);
  else if (E <= 512 && lanes <= 32) by_values<32>(E, f);
  else by_values<64>(E, f);
  return hipGetLastError();
}
// the same where any number of lanes does
template <class F>
hipError_t by_width(int E, F &&f) {
  using std::integral_constant;
  if (E <= 256) by_values<16>(E, f);
  else if (E <= 512) f(integral_constant<int, 32>(), integral_constant<int, 16>());
  else f(integral_constant<int, 64>(), integral_constant<int, 16>());
  return hipGetLastError();
}

// A dispatch holds fewer than 2^32 work-items, and a row takes up to 64: calls of more rows than this
// (of a launch, 2^31 work-items at most) take several launches.  f(first row, rows)
constexpr int64_t kLaunchRows = 1 << 25;
template <class F>
hipError_t by_rows(int64_t T, F &&f) {
  for (int64_t t0 = 0; t0 < T; t0 += kLaunchRows) {
    const hipError_t e = f(t0, T - t0 < kLaunchRows ? T - t0 : kLaunchRows);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <class P>
P *at_row(P *p, int64_t row, int64_t bytes) {
  return (P *)((const char *)p + row * bytes);
}

// blocks of `rows` rows each
int row_grid(int64_t T, int rows) { return (int)((T + rows - 1) / rows); }

// rows of E elements on lines of four
bool rows_on_lines(const void *p, int E, int dtype) {
  const size_t es = dtype == MOE_F32 ? 4 : 2;
  return E % 4 == 0 && (uintptr_t)p % (4 * es) == 0;
}

}  // namespace

hipError_t launch_route_fwd(const void *logits, const float *bias, int64_t T, int E, int k,
                            bool sigmoid, int G, int keep, bool top2, bool renorm, float scale,
                            int32_t *ids, float *w, int dtype, hipStream_t st) {
  const int64_t row = (int64_t)E * (dtype == MOE_F32 ? 4 : 2), slots = (int64_t)k * 4;
  return by_rows(T, [&](int64_t t0, int64_t n) {
    const RouteArgs a{at_row(logits, t0, row), bias, at_row(ids, t0, slots), at_row(w, t0, slots), n, E, k, G,
                      keep, sigmoid, top2, renorm, scale,
                      rows_on_lines(logits, E, dtype), bias && rows_on_lines(bias, E, MOE_F32),
                      ((1u << 20) + E / G - 1) / (E / G)};
    return by_width(E, k > G ? k : G, [&](auto L, auto W) {
      constexpr int LPR = decltype(L)::value, V = decltype(W)::value;
      const int grid = row_grid(n, NW * (64 / LPR));
      auto run = [&](auto t) {
        using X = decltype(t);
        if (bias) route_kernel<X, LPR, V, BY_BIASED><<<grid, NT, 0, st>>>(a);
        else if (G > 1 && top2) route_kernel<X, LPR, V, GROUPS_BY_SCORE><<<grid, NT, 0, st>>>(a);
        else route_kernel<X, LPR, V, BY_LOGIT><<<grid, NT, 0, st>>>(a);
      };
      if (dtype == MOE_F32) run(0.f);
      else run((bf16_t)0);
    });
  });
}

hipError_t launch_route_bwd(const float *g, const void *logits, const int32_t *ids, const float *w,
                            int64_t T, int E, int k, bool sigmoid, bool renorm, float scale,
                            void *d, int dtype, hipStream_t st) {
  const int64_t row = (int64_t)E * (dtype == MOE_F32 ? 4 : 2), slots = (int64_t)k * 4;
  return by_rows(T, [&](int64_t t0, int64_t n) {
    const RouteBwdArgs a{at_row(g, t0, slots), at_row(logits, t0, row), at_row(ids, t0, slots),
                         at_row(w, t0, slots), at_row(d, t0, row), n, E, k, sigmoid, renorm, scale,
                         rows_on_lines(logits, E, dtype) && rows_on_lines(d, E, dtype)};
    return by_width(E, [&](auto L, auto W) {
      constexpr int LPR = decltype(L)::value, V = decltype(W)::value;
      const int grid = row_grid(n, NW * (64 / LPR));
      if (dtype == MOE_F32)
        route_bwd_kernel<float, LPR, V><<<grid, NT, 0, st>>>(a);
      else
        route_bwd_kernel<bf16_t, LPR, V><<<grid, NT, 0, st>>>(a);
    });
  });
}

static int loss_blocks(int64_t T, int E) {
  const int lpr = E <= 256 ? 16 : E <= 512 ? 32 : 64;
  const int64_t g = (T + LW * (64 / lpr) - 1) / (LW * (64 / lpr));
  return (int)(g > kLossBlocks ? kLossBlocks : g);
}

// words of a part (sums and counts) and of all parts and tails, on a 16-byte line; whether the parts are
// summed by several workgroups first
static size_t part_words(int E) { return 2 * (size_t)((E + 3) & ~3); }
static size_t all_words(int blocks, int E) { return blocks * part_words(E) + 2 * ((blocks + 1) & ~1); }
static bool sums_first(int blocks, int E) { return blocks * part_words(E) > 272 * 1024 / sizeof(float); }

size_t loss_workspace_bytes(int64_t T, int E) {
  const int blocks = loss_blocks(T, E);
  return (all_words(blocks, E) + (sums_first(blocks, E) ? kLossParts * part_words(E) : 0)) * sizeof(float);
}

hipError_t launch_loss_fwd(const void *logits, const int32_t *ids, int64_t T, int E, int k,
                           bool sigmoid, float *losses, float *stats, int dtype, void *ws,
                           hipStream_t st) {
  const LossArgs a{logits, ids, (float *)ws, losses, stats, nullptr, nullptr, T, E, k, sigmoid,
                   loss_blocks(T, E), rows_on_lines(logits, E, dtype)};
  hipError_t e = hipSuccess;
  if (a.blocks > 0)
    e = by_width(E, [&](auto L, auto W) {
      constexpr int LPR = decltype(L)::value, V = decltype(W)::value;
      if (dtype == MOE_F32)
        loss_fwd_kernel<float, LPR, V><<<a.blocks, LT, 0, st>>>(a);
      else
        loss_fwd_kernel<bf16_t, LPR, V><<<a.blocks, LT, 0, st>>>(a);
    });
  if (e != hipSuccess) return e;
  const float *sums = a.part;
  int parts = a.blocks;
  if (sums_first(a.blocks, E)) {
    float *out = a.part + all_words(a.blocks, E);
    loss_sum_kernel<<<dim3((unsigned)(part_words(E) / 4 + 63) / 64, kLossParts), 256, 0, st>>>(a, out);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    sums = out;
    parts = kLossParts;
  }
  loss_join_kernel<<<1, LT, 0, st>>>(a, sums, parts);
  return hipGetLastError();
}

hipError_t launch_loss_bwd(const float *dloss, const void *logits, const float *stats, int64_t T,
                           int E, bool sigmoid, void *d, int dtype, hipStream_t st) {
  const LossArgs a{logits, nullptr, nullptr, nullptr, const_cast<float *>(stats), dloss, d, T, E, 0,
                   sigmoid, 0, rows_on_lines(logits, E, dtype) && rows_on_lines(d, E, dtype)};
  return by_width(E, [&](auto L, auto W) {
    constexpr int LPR = decltype(L)::value, V = decltype(W)::value;
    const int64_t g = row_grid(T, NW * (64 / LPR));
    const int grid = (int)(g > 4096 ? 4096 : g);
    if (dtype == MOE_F32)
      loss_bwd_kernel<float, LPR, V><<<grid, NT, 0, st>>>(a);
    else
      loss_bwd_kernel<bf16_t, LPR, V><<<grid, NT, 0, st>>>(a);
  });
}

}  // namespace moe
