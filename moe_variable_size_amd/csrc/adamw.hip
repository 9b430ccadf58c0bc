// One AdamW step over many tensors in one launch (per 48 tensors):
//   g' = s g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2,
//   w = w (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps),
// where w is the parameter itself or its fp32 master copy.  m and v are fp32, or 8 bits each.
//
// 8-bit states: per 256 elements of a tensor one fp32 scale, the largest |m| (sqrt v) of the block over 448,
// and E4M3 codes of m and of sqrt(v) over it (the root has half the range of exponents).  A state moves by
// a fraction 1 - b of itself per step, mostly less than half the distance of two codes (1/16 to 1/8): rounded to
// nearest it would stand still.  So codes are rounded up with the probability of the remainder, by a
// hash of (seed, t, tensor, element): right on average, and the same in every run.
//
// Memory bound: 22 bytes per element for bf16 parameters and gradients with fp32 states, 10 and 16 / 256 with 8-bit
// ones.  8 elements per thread make every access 16 or 32 bytes wide, and 32 lanes a block of 256, whose largest value needs no
// LDS.  Tensors go by in one launch, their descriptors in its arguments (48 of them: 6.8 us for 12 small ones;
// a table in memory would have to be copied there first).  277M elements, bf16: 1099 us with fp32 states (5.5 TB/s; a
// large copy reaches 4.8), 501 with 8-bit ones (5.6).  Non-temporal loads and stores of the states: 1157 with fp32 ones.
#include <math.h>

#include <type_traits>

#include "common.hpp"

namespace moe {
namespace {

constexpr int NT = 256;              // threads
constexpr int PER = 8;               // consecutive elements of a thread: 32 lanes hold a block of 256
constexpr int CHUNK = NT * PER;      // elements of a workgroup
constexpr int kTensors = 48;         // of one launch (they travel in its arguments, below 4 KB)
constexpr int64_t kMaxBlocks = 1 << 23;  // workgroups of one launch (2^31 work-items)
constexpr float kLeast = 7.888609052210118e-31f;  // 2^-100: a block whose largest value is below holds zeros

struct Tensor {
  void *p;
  const void *g;
  void *m, *v;
  float *ms, *vs, *master;
  int64_t n;
};
struct Args {
  Tensor t[kTensors];
  int first[kTensors + 1];  // first workgroup of each tensor, then the launch's workgroups
  uint32_t number[kTensors];
  int count_at[kTensors];   // place of each tensor's t in t_dev
  uint64_t wide;            // bit i: tensor i lies on 16-byte lines
  int count;
  float lr, b1, a1, b2, a2, eps, wd;  // a = 1 - b
  float c1, c2;                       // 1 - b^t, for t known to the host
  float ln1, ln2;                     // ln b, for t on the device
  const float *lr_dev, *scale;
  const int32_t *t_dev;
  uint32_t t_low, seed;
};
static_assert(sizeof(Args) <= 4096, "kernel arguments");

MOE_DEV uint32_t mix(uint32_t h) {  // the fractions of sqrt 2 and sqrt 3 as odd factors
  h = (h ^ (h >> 16)) * 0x6A09E667u;
  h = (h ^ (h >> 15)) * 0xBB67AE85u;
  return h ^ (h >> 16);
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// 8 elements from p, on a 16-byte line and all there (whole), or one by one
MOE_DEV void get8(const float *p, bool whole, int left, float (&v)[PER]) {
  if (whole) {
    const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = i < left ? p[i] : 0.f;
  }
}
MOE_DEV void get8(const bf16_t *p, bool whole, int left, float (&v)[PER]) {
  if (whole) {
    const u32x4 a = *(const u32x4 *)p;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = __uint_as_float(i & 1 ? a[i / 2] & 0xffff0000u : a[i / 2] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] = i < left ? bf16_to_f32(p[i]) : 0.f;
  }
}
MOE_DEV void put8(float *p, bool whole, int left, const float (&v)[PER]) {
  if (whole) {
    *(f32x4 *)p = f32x4{v[0], v[1], v[2], v[3]};
    *(f32x4 *)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < left) p[i] = v[i];
  }
}
MOE_DEV void put8(bf16_t *p, bool whole, int left, const float (&v)[PER]) {
  typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
  if (whole) {
    *(bf16x8 *)p = bf16x8{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3],
                          (__bf16)v[4], (__bf16)v[5], (__bf16)v[6], (__bf16)v[7]};
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < left) p[i] = __builtin_bit_cast(bf16_t, (__bf16)v[i]);
  }
}

// 8 codes times their block's scale
MOE_DEV void get8(const uint8_t *p, bool whole, int left, float scale, float (&v)[PER]) {
  u32x2 c = {0, 0};
  if (whole) {
    c = *(const u32x2 *)p;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < left) c[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    v[4 * h] = __builtin_amdgcn_cvt_f32_fp8(c[h], 0) * scale;
    v[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8(c[h], 1) * scale;
    v[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8(c[h], 2) * scale;
    v[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8(c[h], 3) * scale;
  }
}

// The largest |a| of a block (32 lanes); a NaN among them is the largest.
MOE_DEV float block_top(const float (&a)[PER]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = __builtin_elementwise_maximum(top, fabsf(a[i]));
  // neighbours, pairs, then halves and rows of 16 mirrored (once their members are alike); the last step through LDS's crossbar
  auto join = [&](auto ctrl) __attribute__((always_inline)) {
    const int other = __builtin_amdgcn_update_dpp(0, __float_as_int(top), decltype(ctrl)::value, 0xF, 0xF, false);
    top = __builtin_elementwise_maximum(top, __int_as_float(other));
  };
  join(std::integral_constant<int, 0xB1>());   // quad_perm 1 0 3 2
  join(std::integral_constant<int, 0x4E>());   // quad_perm 2 3 0 1
  join(std::integral_constant<int, 0x141>());  // row_half_mirror
  join(std::integral_constant<int, 0x140>());  // row_mirror
  return __builtin_elementwise_maximum(top, __shfl_xor(top, 16, 64));
}

// Codes of four values (at most 448 but for a rounding) into a word.  The instruction adds the random number's upper 20
// bits to the 20 bits that a code drops (shifted alike where it is subnormal), and cuts off: with 16 bits h and a half behind
// them that is floor(y / d + u), u = (h + 1/2) / 2^16.  (u is never 0: the largest value of a block, 448 but for a rounding,
// keeps its code.)  With ten instructions less per code, and the roots' range looked at once per wave, 277M elements take 501 us
// for 611.
MOE_DEV uint32_t codes4(const float *y, const uint32_t (&u)[4]) {
  int c = __builtin_amdgcn_cvt_sr_fp8_f32(y[0], (int)u[0], 0, 0);
  c = __builtin_amdgcn_cvt_sr_fp8_f32(y[1], (int)u[1], c, 1);
  c = __builtin_amdgcn_cvt_sr_fp8_f32(y[2], (int)u[2], c, 2);
  return (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(y[3], (int)u[3], c, 3);
}

// a rounded to codes, and the block's scale (NaN where a value is not finite, so that all of the block becomes one),
// with the low or the high halves of h
template <bool LOW>
MOE_DEV void put8(uint8_t *p, float *scale, bool whole, int left, const float (&a)[PER],
                  const uint32_t (&h)[PER]) {
  const float top = block_top(a);
  const bool none = top < kLeast;
  const float inv = none ? 0.f : 1.f / top * 448.f;
  u32x2 c;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float y[4];
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = a[4 * w + i] * inv;
      u[i] = (LOW ? h[4 * w + i] << 16 : h[4 * w + i] & 0xffff0000u) | 0x8000u;
    }
    c[w] = codes4(y, u);
  }
  if (whole) {
    *(u32x2 *)p = c;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < left) p[i] = (uint8_t)(c[i / 4] >> (8 * (i & 3)));
  }
  if ((threadIdx.x & 31) == 0 && left > 0) *scale = none ? 0.f : top < INFINITY ? top * (1.f / 448.f) : NAN;
}

// The hardware's root, off by a step at most, with small arguments in its range (the exact one takes three times as many
// instructions)
MOE_DEV float root_of(float v) {
  const bool small = v < 0x1p-96f;
  return __builtin_amdgcn_sqrtf(small ? v * 0x1p64f : v) * (small ? 0x1p-32f : 1.f);
}

// States in 8 bits: every operation rounded once, in the formulas' order, none fused, and the root to nearest (the hardware's
// reciprocal root and one correction by the remainder).  A sum or a root that is a step off turns a rounding of codes the other
// way now and then, and in later steps, through a block's largest value, the scale of all of it; like this the states do
// not depend on how the arithmetic is carried out.
MOE_DEV float exact_root(float v) {
  const bool small = v < 0x1p-96f;
  const float x = small ? v * 0x1p64f : v, y = __builtin_amdgcn_rsqf(x), s = x * y, e = fmaf(-s, s, x);
  const float root = fmaf(e, 0.5f * y, s) * (small ? 0x1p-32f : 1.f);
  return e == e ? root : v;  // (of 0, infinity and NaN: they themselves)
}
// the same where no argument of the wave is small or not finite
MOE_DEV float exact_root_in_range(float v) {
  const float y = __builtin_amdgcn_rsqf(v), s = v * y;
  return fmaf(fmaf(-s, s, v), 0.5f * y, s);
}
MOE_DEV float mean_of(float b, float old, float a, float x) {
#pragma clang fp contract(off)
  return b * old + a * x;
}
MOE_DEV float square_of(float b, float old, float a, float x) {
#pragma clang fp contract(off)
  return b * old + a * x * x;
}

// elements at .. at + 7 of tensor t (FULL: the whole workgroup's are there, on 16-byte lines)
template <typename P, typename G, int BITS, bool FULL>
MOE_DEV void step8(const Args &a, const Tensor &t, uint32_t number, int count_at, int64_t at, float s) {
  const int left = FULL ? PER : (int)max((int64_t)0, min((int64_t)PER, t.n - at));
  float g[PER], m[PER], v[PER], w[PER], r[PER];
  get8((const G *)t.g + at, FULL, left, g);
  if (t.master) get8(t.master + at, FULL, left, w);
  else get8((const P *)t.p + at, FULL, left, w);
  if constexpr (BITS == 32) {
    get8((const float *)t.m + at, FULL, left, m);
    get8((const float *)t.v + at, FULL, left, v);
  } else {
    const int64_t b = left > 0 ? at / 256 : 0;
    get8((const uint8_t *)t.m + at, FULL, left, t.ms[b], m);
    get8((const uint8_t *)t.v + at, FULL, left, t.vs[b], v);
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] *= v[i];
  }
  const uint32_t step = a.t_dev ? (uint32_t)a.t_dev[count_at] : a.t_low;
  const float c1 = a.t_dev ? -expm1f((float)a.t_dev[count_at] * a.ln1) : a.c1;
  const float c2 = a.t_dev ? -expm1f((float)a.t_dev[count_at] * a.ln2) : a.c2;
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  const float rate = lr / c1, keep = 1.f - lr * a.wd, root = 1.f / sqrtf(c2);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float x = g[i] * s;
    if constexpr (BITS == 8) {
      m[i] = mean_of(a.b1, m[i], a.a1, x);
      v[i] = square_of(a.b2, v[i], a.a2, x);
    } else {
      m[i] = fmaf(a.b1, m[i], a.a1 * x);
      v[i] = fmaf(a.b2, v[i], a.a2 * x * x);
    }
  }
  if constexpr (BITS == 8) {
    float lo = v[0], hi = v[0];  // (NaN if one is)
#pragma unroll
    for (int i = 1; i < PER; ++i) {
      lo = __builtin_elementwise_minimum(lo, v[i]);
      hi = __builtin_elementwise_maximum(hi, v[i]);
    }
    if (__all(lo >= 0x1p-96f && hi < INFINITY)) {
#pragma unroll
      for (int i = 0; i < PER; ++i) r[i] = exact_root_in_range(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) r[i] = exact_root(v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) r[i] = root_of(v[i]);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    w[i] = fmaf(w[i], keep, -(rate * m[i]) * __builtin_amdgcn_rcpf(fmaf(r[i], root, a.eps)));
  put8((P *)t.p + at, FULL, left, w);
  if (t.master) put8(t.master + at, FULL, left, w);
  if constexpr (BITS == 32) {
    put8((float *)t.m + at, FULL, left, m);
    put8((float *)t.v + at, FULL, left, v);
  } else {
    if constexpr (!FULL) {  // nothing behind the tensor's end counts for its last block
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i >= left) m[i] = r[i] = 0.f;
    }
    const uint32_t key = mix(mix(a.seed + 0x9E3779B9u * step) + number + 0x9E3779B9u * (uint32_t)(at >> 32));
    uint32_t h[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) h[i] = mix(((uint32_t)at + i) ^ key);
    put8<true>((uint8_t *)t.m + at, t.ms + at / 256, FULL, left, m, h);
    put8<false>((uint8_t *)t.v + at, t.vs + at / 256, FULL, left, r, h);
  }
}

template <typename P, typename G, int BITS>
__global__ __launch_bounds__(NT) void adamw_kernel(const Args a) {
  const float s = a.scale ? *a.scale : 1.f;
  if (!(fabsf(s) < INFINITY)) return;  // a step whose gradients are not finite is left out
  int lo = 0, hi = a.count - 1;  // the tensor of this workgroup: the last whose first is not behind it
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first[mid] <= (int)blockIdx.x) lo = mid; else hi = mid - 1;
  }
  const int64_t first = (int64_t)((int)blockIdx.x - a.first[lo]) * CHUNK, at = first + threadIdx.x * PER;
  if ((a.wide >> lo & 1) && first + CHUNK <= a.t[lo].n) step8<P, G, BITS, true>(a, a.t[lo], a.number[lo], a.count_at[lo], at, s);
  else step8<P, G, BITS, false>(a, a.t[lo], a.number[lo], a.count_at[lo], at, s);
}

// one more step for each of the launch's tensors, before it
__global__ __launch_bounds__(64) void count_kernel(const Args a, int32_t *counts) {
  const float s = a.scale ? *a.scale : 1.f;
  if (fabsf(s) < INFINITY && (int)threadIdx.x < a.count) ++counts[a.count_at[threadIdx.x]];
}
static_assert(kTensors <= 64, "a thread per tensor");

template <typename P, typename G>
hipError_t launch(const Args &a, int bits, hipStream_t st) {
  const int grid = a.first[a.count];
  if (bits == 32) adamw_kernel<P, G, 32><<<grid, NT, 0, st>>>(a);
  else adamw_kernel<P, G, 8><<<grid, NT, 0, st>>>(a);
  return hipGetLastError();
}

bool line(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

}  // namespace

hipError_t launch_adamw(const moe_adamw_tensor *tensors, int count, const AdamwOptions &o, int param_dtype,
                        int grad_dtype, int bits, hipStream_t st) {
  Args a;
  a.lr = (float)o.lr;
  a.b1 = (float)o.beta1;
  a.a1 = (float)(1.0 - o.beta1);
  a.b2 = (float)o.beta2;
  a.a2 = (float)(1.0 - o.beta2);
  // (the reciprocal of a number below the normal ones is infinite; v = 0 has then to give m / eps, mostly 0)
  a.eps = o.eps > 0 ? fmaxf((float)o.eps, 0x1p-126f) : 0.f;
  a.wd = (float)o.weight_decay;
  a.ln1 = (float)log(o.beta1);
  a.ln2 = (float)log(o.beta2);
  a.c1 = (float)-expm1((double)o.step * log(o.beta1));
  a.c2 = (float)-expm1((double)o.step * log(o.beta2));
  a.lr_dev = o.lr_dev;
  a.scale = o.grad_scale;
  a.t_dev = o.step_dev;
  a.t_low = (uint32_t)o.step;
  a.seed = o.seed;
  const size_t state = bits == 32 ? 16 : 8;
  int i = 0;
  while (i < count) {
    a.count = 0;
    a.wide = 0;
    a.first[0] = 0;
    for (; i < count && a.count < kTensors; ++i) {
      const moe_adamw_tensor &x = tensors[i];
      if (x.n == 0) continue;
      const int64_t blocks = (x.n + CHUNK - 1) / CHUNK;
      if (a.count && a.first[a.count] + blocks > kMaxBlocks) break;
      const int k = a.count++;
      a.t[k] = Tensor{x.param, x.grad, x.m, x.v, x.m_scale, x.v_scale, x.master, x.n};
      a.number[k] = (uint32_t)x.number;
      a.count_at[k] = o.counts ? (int)x.number : 0;
      a.first[k + 1] = a.first[k] + (int)blocks;
      if (line(x.param, 16) && line(x.grad, 16) && line(x.m, state) && line(x.v, state) && line(x.master, 16))
        a.wide |= 1ull << k;
    }
    if (!a.count) break;
    hipError_t e;
    if (o.counts) {
      count_kernel<<<1, 64, 0, st>>>(a, o.counts);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (param_dtype == MOE_F32)
      e = grad_dtype == MOE_F32 ? launch<float, float>(a, bits, st) : launch<float, bf16_t>(a, bits, st);
    else
      e = grad_dtype == MOE_F32 ? launch<bf16_t, float>(a, bits, st) : launch<bf16_t, bf16_t>(a, bits, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
