// Routing to experts and the losses that keep a router balanced: from a row of
// logits to the expert ids and weights a schedule is built from, and back.
//
// A wave takes a row of E <= 1024 logits, VPL = ceil(E / 64) of them per lane
// (expert e = 64 i + lane in slot i), and keeps the row in registers.
//
// Choice.  Experts are ranked by a 64-bit key that orders like the choice value
// (the logit, or score + bias computed in 64 bits) with NaN above everything
// and an expert that may not be chosen below everything; equal keys go to the
// lower expert.  k rounds of wave-wide maximum take the k best.
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

struct RouteArgs {
  const void *logits;
  const float *bias;
  int32_t *ids;
  float *w;
  int64_t T;
  int E, k, G, keep;
  int sigmoid, top2, renorm;
  float scale;
};

// score of a logit relative to exp(shift): exp(l - shift) (softmax, shift = the
// row's or the chosen maximum) or sigmoid(l) exp(-shift) (shift = min(maximum,
// 0), so that a row of very negative logits keeps a nonzero sum)
MOE_DEV float shifted_score(float l, float shift, bool sigmoid) {
  if (!sigmoid) return expf(l - shift);
  return expf(fminf(l, 0.f) - shift) / (1.f + expf(-fabsf(l)));
}

template <typename T, int VPL>
__global__ __launch_bounds__(NT) void route_kernel(RouteArgs p) {
  extern __shared__ int64_t smem[];  // per wave: E keys, 64 group values
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  int64_t *keys = smem + (size_t)wid * (VPL * 64 + 64), *gval = keys + VPL * 64;
  for (int64_t t = (int64_t)blockIdx.x * NW + wid; t < p.T; t += (int64_t)gridDim.x * NW) {
    const T *row = (const T *)p.logits + t * p.E;
    float l[VPL];
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 64 + lane;
      l[i] = e < p.E ? ldf(row + e) : -__builtin_inff();
      m = fmaxf(m, l[i]);
    }
    m = wave_max(m);
    // choice values
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
      __builtin_amdgcn_wave_barrier();
      __threadfence_block();
      int64_t gk = kBarred;
      if (lane < p.G) {
        int64_t a = kBarred, b = kBarred;  // the two best
        for (int j = 0; j < per; ++j) {
          const int64_t v = keys[lane * per + j];
          if (v > a) { b = a; a = v; } else if (v > b) b = v;
        }
        gk = !p.top2 || b == kBarred ? a : order_key(key_value(a) + key_value(b));
        gval[lane] = gk;
      }
      __builtin_amdgcn_wave_barrier();
      __threadfence_block();
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
      __builtin_amdgcn_wave_barrier();
      __threadfence_block();
    }
    // k rounds
    int id = -1;      // lane j: slot j
    float lj = -__builtin_inff();
    for (int j = 0; j < p.k; ++j) {
      int64_t best = kBarred;
      int at = INT32_MAX;
      float la = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (key[i] > best) { best = key[i]; at = i * 64 + lane; la = l[i]; }
#pragma unroll
      for (int d = 32; d; d >>= 1) {
        const int64_t ok = __shfl_xor(best, d, kWave);
        const int oa = __shfl_xor(at, d, kWave);
        const float ol = __shfl_xor(la, d, kWave);
        if (ok > best || (ok == best && oa < at)) { best = ok; at = oa; la = ol; }
      }
      if (best == kBarred) break;
      if (lane == j) { id = at; lj = la; }
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (at == i * 64 + lane) key[i] = kBarred;
    }
    // weights
    const bool on = id >= 0;
    float wgt;
    if (p.renorm) {
      const float mc = wave_max(on ? lj : -__builtin_inff());
      const float sj = on ? shifted_score(lj, p.sigmoid ? fminf(mc, 0.f) : mc, p.sigmoid) : 0.f;
      float all = wave_sum(sj);
      if (!p.sigmoid) {  // a NaN anywhere in the row is in its softmax
        float bad = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) bad += l[i] != l[i] ? l[i] : 0.f;
        all += wave_sum(bad);
      }
      wgt = sj / all * p.scale;
    } else if (p.sigmoid) {
      wgt = shifted_score(lj, 0.f, true) * p.scale;
    } else {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) sum += l[i] == -__builtin_inff() ? 0.f : expf(l[i] - m);
      wgt = expf(lj - m) / wave_sum(sum) * p.scale;
    }
    if (lane < p.k) {
      p.ids[t * p.k + lane] = id;
      p.w[t * p.k + lane] = on ? wgt : 0.f;
    }
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
};

// g_j = dL/dw_j.  With D = sum_j g_j w_j:
//   renormalised: dl_j = w_j (g_j - D / scale), times 1 - s_j for the sigmoid;
//   plain softmax: dl_i = w_i g_i [i chosen] - p_i D;  plain sigmoid: dl_j = g_j w_j (1 - s_j).
template <typename T, int VPL>
__global__ __launch_bounds__(NT) void route_bwd_kernel(RouteBwdArgs p) {
  __shared__ float rows[NW][VPL * 64];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  float *buf = rows[wid];
  for (int64_t t = (int64_t)blockIdx.x * NW + wid; t < p.T; t += (int64_t)gridDim.x * NW) {
    const T *row = (const T *)p.logits + t * p.E;
    const int id = lane < p.k ? p.ids[t * p.k + lane] : -1;
    const bool on = id >= 0 && id < p.E;
    const float w = on ? p.w[t * p.k + lane] : 0.f, g = on ? p.g[t * p.k + lane] : 0.f;
    const float D = wave_sum(g * w);
    float c = w * (p.renorm ? g - D / p.scale : g);
    if (p.sigmoid && on) {  // 1 - s = sigmoid(-l)
      const float l = ldf(row + id);
      c *= shifted_score(-l, 0.f, true);
    }
    const bool dense = !p.renorm && !p.sigmoid;
    float l[VPL], m = -__builtin_inff(), sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 64 + lane;
      buf[e] = 0.f;
      l[i] = dense && e < p.E ? ldf(row + e) : -__builtin_inff();
      m = fmaxf(m, l[i]);
    }
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
    if (on) atomicAdd(&buf[id], c);  // ids of one row differ; repeated ones add up
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
    if (dense) {
      m = wave_max(m);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        l[i] = l[i] == -__builtin_inff() ? 0.f : expf(l[i] - m);
        sum += l[i];
      }
      sum = wave_sum(sum);
      const float f = sum > 0.f || sum != sum ? D / sum : 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] *= f;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 64 + lane;
      if (e < p.E) stf((T *)p.d + t * p.E + e, buf[e] - (dense ? l[i] : 0.f));
    }
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- losses --------------------------------------------------------------------
// Forward: every block sums its rows' probabilities and counts its ids per
// expert, and its rows' squared log-sum-exps; one block joins the partial sums in
// a fixed order.  Workspace: [blocks][2 E + 2] words: sums, counts, z, rows.
constexpr int kLossBlocks = 256;

struct LossArgs {
  const void *logits;
  const int32_t *ids;
  float *part;
  float *losses, *stats;
  const float *dloss;
  void *d;
  int64_t T;
  int E, k, sigmoid, blocks;
};

// probabilities of a row (softmax, or the sigmoids over their sum); lse; empty
// rows (every logit -inf) give zeros.  soft[]: the softmax, q[]: the probabilities
template <int VPL>
MOE_DEV bool row_probs(const float (&l)[VPL], bool sigmoid, float (&soft)[VPL], float (&q)[VPL],
                       float &lse) {
  float m = -__builtin_inff();
  bool any = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    m = fmaxf(m, l[i]);
    any |= l[i] != -__builtin_inff();
  }
  any = __any(any);
  m = wave_max(m);
  float sum = 0.f, qsum = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool off = l[i] == -__builtin_inff();
    soft[i] = off ? 0.f : expf(l[i] - m);
    sum += soft[i];
    if (sigmoid) {
      q[i] = off ? 0.f : shifted_score(l[i], fminf(m, 0.f), true);
      qsum += q[i];
    }
  }
  sum = wave_sum(sum);
  lse = any ? m + logf(sum) : 0.f;
  const float inv = any ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) soft[i] *= inv;
  if (sigmoid) {
    qsum = wave_sum(qsum);
    const float qinv = any ? 1.f / qsum : 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) q[i] *= qinv;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) q[i] = soft[i];
  }
  return any;
}

template <typename T, int VPL>
__global__ __launch_bounds__(NT) void loss_fwd_kernel(LossArgs p) {
  __shared__ float psum[NW][VPL * 64];
  __shared__ int cnt[VPL * 64];
  __shared__ float zs[NW];
  __shared__ int rs[NW];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < VPL * 64; e += NT) cnt[e] = 0;
  __syncthreads();
  float acc[VPL] = {}, z = 0.f;
  int rows = 0;
  for (int64_t t = (int64_t)blockIdx.x * NW + wid; t < p.T; t += (int64_t)gridDim.x * NW) {
    const T *row = (const T *)p.logits + t * p.E;
    float l[VPL], soft[VPL], q[VPL], lse;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 64 + lane;
      l[i] = e < p.E ? ldf(row + e) : -__builtin_inff();
    }
    rows += row_probs<VPL>(l, p.sigmoid, soft, q, lse);
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] += q[i];
    z += lse * lse;
    if (lane < p.k) {
      const int id = p.ids[t * p.k + lane];
      if (id >= 0 && id < p.E) atomicAdd(&cnt[id], 1);
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) psum[wid][i * 64 + lane] = acc[i];
  if (lane == 0) { zs[wid] = z; rs[wid] = rows; }
  __syncthreads();
  float *part = p.part + (size_t)blockIdx.x * (2 * p.E + 2);
  for (int e = threadIdx.x; e < p.E; e += NT) {
    float v = 0.f;
    for (int w = 0; w < NW; ++w) v += psum[w][e];
    part[e] = v;
    part[p.E + e] = __int_as_float(cnt[e]);
  }
  if (threadIdx.x == 0) {
    float v = 0.f;
    int r = 0;
    for (int w = 0; w < NW; ++w) { v += zs[w]; r += rs[w]; }
    part[2 * p.E] = v;
    part[2 * p.E + 1] = __int_as_float(r);
  }
}

__global__ __launch_bounds__(1024) void loss_join_kernel(LossArgs p) {
  __shared__ double red[1024];
  __shared__ long long ired[1024];
  const int tid = threadIdx.x;
  const int pitch = 2 * p.E + 2;
  double P = 0.0;
  long long c = 0;
  if (tid < p.E)
    for (int b = 0; b < p.blocks; ++b) {
      P += p.part[(size_t)b * pitch + tid];
      c += __float_as_int(p.part[(size_t)b * pitch + p.E + tid]);
    }
  double z = 0.0;
  long long r = 0;
  for (int b = tid; b < p.blocks; b += 1024) {
    z += p.part[(size_t)b * pitch + 2 * p.E];
    r += __float_as_int(p.part[(size_t)b * pitch + 2 * p.E + 1]);
  }
  auto isum = [&](long long v) {
    ired[tid] = v;
    __syncthreads();
    for (int d = 512; d; d >>= 1) {
      if (tid < d) ired[tid] += ired[tid + d];
      __syncthreads();
    }
    const long long s = ired[0];
    __syncthreads();
    return s;
  };
  auto dsum = [&](double v) {
    red[tid] = v;
    __syncthreads();
    for (int d = 512; d; d >>= 1) {
      if (tid < d) red[tid] += red[tid + d];
      __syncthreads();
    }
    const double s = red[0];
    __syncthreads();
    return s;
  };
  const long long C = isum(c), V = isum(r);
  const double inv = V > 0 ? 1.0 / (double)V : 0.0;
  const float f = C > 0 ? (float)((double)p.E * (double)c / (double)C) : 0.f;
  if (tid < p.E) p.stats[tid] = f;
  const double bal = dsum(tid < p.E ? (double)f * P : 0.0), zz = dsum(z);
  if (tid == 0) {
    p.stats[p.E] = (float)inv;
    p.losses[0] = (float)(bal * inv);
    p.losses[1] = (float)(zz * inv);
  }
}

template <typename T, int VPL>
__global__ __launch_bounds__(NT) void loss_bwd_kernel(LossArgs p) {
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const float inv = p.stats[p.E];
  const float gb = p.dloss[0] * inv, gz = 2.f * p.dloss[1] * inv;
  float f[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) f[i] = i * 64 + lane < p.E ? p.stats[i * 64 + lane] : 0.f;
  for (int64_t t = (int64_t)blockIdx.x * NW + wid; t < p.T; t += (int64_t)gridDim.x * NW) {
    const T *row = (const T *)p.logits + t * p.E;
    float l[VPL], soft[VPL], q[VPL], lse;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 64 + lane;
      l[i] = e < p.E ? ldf(row + e) : -__builtin_inff();
    }
    row_probs<VPL>(l, p.sigmoid, soft, q, lse);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) dot += f[i] * q[i];
    dot = wave_sum(dot);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 64 + lane;
      float d = gb * q[i] * (f[i] - dot);
      if (p.sigmoid && l[i] != -__builtin_inff()) d *= shifted_score(-l[i], 0.f, true);
      d += gz * lse * soft[i];
      if (e < p.E) stf((T *)p.d + t * p.E + e, d);
    }
  }
}

// f(integral_constant<VPL>) for E experts
template <class F>
hipError_t by_width(int E, F &&f) {
  if (E <= 64) f(std::integral_constant<int, 1>());
  else if (E <= 128) f(std::integral_constant<int, 2>());
  else if (E <= 256) f(std::integral_constant<int, 4>());
  else if (E <= 512) f(std::integral_constant<int, 8>());
  else f(std::integral_constant<int, 16>());
  return hipGetLastError();
}

int row_grid(int64_t T) {
  const int64_t g = (T + NW - 1) / NW;
  return (int)(g < 1 ? 1 : g > 65536 ? 65536 : g);
}

}  // namespace

hipError_t launch_route_fwd(const void *logits, const float *bias, int64_t T, int E, int k,
                            bool sigmoid, int G, int keep, bool top2, bool renorm, float scale,
                            int32_t *ids, float *w, int dtype, hipStream_t st) {
  RouteArgs a{logits, bias, ids, w, T, E, k, G, keep, sigmoid, top2, renorm, scale};
  return by_width(E, [&](auto V) {
    constexpr int VPL = decltype(V)::value;
    const size_t sm = G > 1 ? (size_t)NW * (VPL * 64 + 64) * sizeof(int64_t) : 0;
    if (dtype == MOE_F32)
      route_kernel<float, VPL><<<row_grid(T), NT, sm, st>>>(a);
    else
      route_kernel<bf16_t, VPL><<<row_grid(T), NT, sm, st>>>(a);
  });
}

hipError_t launch_route_bwd(const float *g, const void *logits, const int32_t *ids, const float *w,
                            int64_t T, int E, int k, bool sigmoid, bool renorm, float scale,
                            void *d, int dtype, hipStream_t st) {
  RouteBwdArgs a{g, logits, ids, w, d, T, E, k, sigmoid, renorm, scale};
  return by_width(E, [&](auto V) {
    constexpr int VPL = decltype(V)::value;
    if (dtype == MOE_F32)
      route_bwd_kernel<float, VPL><<<row_grid(T), NT, 0, st>>>(a);
    else
      route_bwd_kernel<bf16_t, VPL><<<row_grid(T), NT, 0, st>>>(a);
  });
}

static int loss_blocks(int64_t T) {
  const int64_t g = (T + NW - 1) / NW;
  return (int)(g > kLossBlocks ? kLossBlocks : g);
}

size_t loss_workspace_bytes(int64_t T, int E) {
  return (size_t)loss_blocks(T) * (2 * (size_t)E + 2) * sizeof(float);
}

hipError_t launch_loss_fwd(const void *logits, const int32_t *ids, int64_t T, int E, int k,
                           bool sigmoid, float *losses, float *stats, int dtype, void *ws,
                           hipStream_t st) {
  LossArgs a{logits, ids, (float *)ws, losses, stats, nullptr, nullptr, T, E, k, sigmoid,
             loss_blocks(T)};
  hipError_t e = hipSuccess;
  if (a.blocks > 0)
    e = by_width(E, [&](auto V) {
      constexpr int VPL = decltype(V)::value;
      if (dtype == MOE_F32)
        loss_fwd_kernel<float, VPL><<<a.blocks, NT, 0, st>>>(a);
      else
        loss_fwd_kernel<bf16_t, VPL><<<a.blocks, NT, 0, st>>>(a);
    });
  if (e != hipSuccess) return e;
  loss_join_kernel<<<1, 1024, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_loss_bwd(const float *dloss, const void *logits, const float *stats, int64_t T,
                           int E, bool sigmoid, void *d, int dtype, hipStream_t st) {
  LossArgs a{logits, nullptr, nullptr, nullptr, const_cast<float *>(stats), dloss, d, T, E, 0,
             sigmoid, 0};
  return by_width(E, [&](auto V) {
    constexpr int VPL = decltype(V)::value;
    if (dtype == MOE_F32)
      loss_bwd_kernel<float, VPL><<<row_grid(T), NT, 0, st>>>(a);
    else
      loss_bwd_kernel<bf16_t, VPL><<<row_grid(T), NT, 0, st>>>(a);
  });
}

}  // namespace moe
