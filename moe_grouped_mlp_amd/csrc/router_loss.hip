// The router's auxiliary losses, per-expert counts and the gradient with
// respect to its logits.
//
//   p = softmax(x);  lse = log sum exp x;  over the n tokens kept:
//   counts_e = picks of e;  P_e = (1/n) sum p_e
//   L = c_b E sum_e counts_e / (k n) P_e + c_z (1/n) sum lse^2
//   dx_j = p_j (v_j - sum_i p_i v_i + 2 c_z lse / n),
//   v_j = c_b E counts_j / (k n^2) + sum of dprobs over the slots that name j
//
// A token takes L lanes of a wave, L a power of two that leaves a lane at
// most 16 of the E logits, so the logits are read once and stay in
// registers; a wave covers 64 / L tokens.  Lane g of a token holds experts
// 4 (g + L i) + c (VEC: E % 4 == 0 and 16-byte aligned rows, one float4
// each), else g + L i.  The
// loss kernel keeps each lane's sums of p over its tokens in registers, adds
// them over the workgroup in a fixed order and writes one fp32 partial per
// expert and workgroup; a second launch of one workgroup adds these in fp64.
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;   // logits a lane holds

template <int L, typename T, typename F>
MOE_DEV T group_reduce(T v, F f) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = f(v, static_cast<T>(__shfl_xor(v, o, kWave)));
  return v;
}
template <int L>
MOE_DEV float group_sum(float v) {
  return group_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
MOE_DEV float group_max(float v) {
  return group_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}

// Expert of a lane's i-th logit.
template <int L, bool VEC>
MOE_DEV int expert_at(int g, int i) {
  return VEC ? 4 * (g + L * (i / 4)) + i % 4 : g + L * i;
}

// One token's softmax: p[i] of the lane's experts and lse; false (p zero)
// if the logits are all -infinity.  Experts past E have p 0.
template <int L, bool VEC>
MOE_DEV bool token_softmax(const float* __restrict__ row, int E, int g, float (&p)[kPer],
                           float& lse) {
  constexpr float kNegInf = -__builtin_inff();
  if constexpr (VEC) {
    const float4* r4 = reinterpret_cast<const float4*>(row);
#pragma unroll
    for (int q = 0; q < kPer / 4; ++q) {
      float4 v = {kNegInf, kNegInf, kNegInf, kNegInf};
      if (4 * (g + L * q) < E) v = r4[g + L * q];
      p[4 * q] = v.x;
      p[4 * q + 1] = v.y;
      p[4 * q + 2] = v.z;
      p[4 * q + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) p[i] = g + L * i < E ? row[g + L * i] : kNegInf;
  }
  float m = kNegInf;
#pragma unroll
  for (int i = 0; i < kPer; ++i) m = fmaxf(m, p[i]);
  m = group_max<L>(m);
  // the maximum of NaN and a number is the number here; a token of NaN
  // alone keeps m at -infinity and is told from an empty one by its logits
  float nan = 0.0f;
  float z = 0.0f;
  const float mm = m == kNegInf ? 0.0f : m;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    p[i] = expf(p[i] - mm);
    z += p[i];
    nan = p[i] != p[i] ? 1.0f : nan;
  }
  z = group_sum<L>(z);
  if (m == kNegInf && group_max<L>(nan) == 0.0f) return false;
  const float inv = 1.0f / z;
#pragma unroll
  for (int i = 0; i < kPer; ++i) p[i] *= inv;
  lse = mm + logf(z);
  return true;
}

// Partials of one workgroup: prob [E], count [E], then {sum lse^2, n}.
template <int L, bool VEC>
__global__ __launch_bounds__(kThreads) void router_loss_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx,
    const uint8_t* __restrict__ mask, int T, int E, int k, float* __restrict__ part_p,
    int32_t* __restrict__ part_c, float* __restrict__ part_z, int32_t* __restrict__ part_n) {
  constexpr int kTok = kThreads / L;   // tokens the workgroup covers at once
  __shared__ float s_p[kMaxExperts];
  __shared__ int32_t s_c[kMaxExperts];
  __shared__ float s_z[kThreads / kWave];
  __shared__ int32_t s_n[kThreads / kWave];
  const int tid = threadIdx.x, g = tid % L, wave = tid / kWave;
  for (int e = tid; e < E; e += kThreads) {
    s_p[e] = 0.0f;
    s_c[e] = 0;
  }
  __syncthreads();
  float sum[kPer] = {};
  float zsum = 0.0f;
  int32_t n = 0;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTok; t0 < T;
       t0 += static_cast<int64_t>(gridDim.x) * kTok) {
    const int64_t t = t0 + tid / L;
    if (t < T && (!mask || mask[t])) {
      float p[kPer], lse = 0.0f;
      if (token_softmax<L, VEC>(logits + t * E, E, g, p, lse)) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) sum[i] += p[i];
        if (g == 0) {
          zsum += lse * lse;
          ++n;
        }
        for (int s = g; s < k; s += L) {
          const int32_t e = idx[t * k + s];
          if (e >= 0 && e < E) atomicAdd(&s_c[e], 1);   // integers: any order
        }
      }
    }
  }
  // the lanes of a wave that hold the same experts (same g), then the waves
  // one after the other
#pragma unroll
  for (int o = L; o < kWave; o <<= 1) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum[i] += __shfl_xor(sum[i], o, kWave);
  }
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    zsum += __shfl_xor(zsum, o, kWave);
    n += __shfl_xor(n, o, kWave);
  }
  if (tid % kWave == 0) {
    s_z[wave] = zsum;
    s_n[wave] = n;
  }
  for (int w = 0; w < kThreads / kWave; ++w) {
    if (wave == w && tid % kWave < L) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = expert_at<L, VEC>(g, i);
        if (e < E) s_p[e] += sum[i];
      }
    }
    __syncthreads();
  }
  const int64_t at = static_cast<int64_t>(blockIdx.x) * E;
  for (int e = tid; e < E; e += kThreads) {
    part_p[at + e] = s_p[e];
    part_c[at + e] = s_c[e];
  }
  if (tid == 0) {
    float z = 0.0f;
    int32_t m = 0;
    for (int w = 0; w < kThreads / kWave; ++w) {
      z += s_z[w];
      m += s_n[w];
    }
    part_z[blockIdx.x] = z;
    part_n[blockIdx.x] = m;
  }
}

constexpr int kSumThreads = 1024;

MOE_DEV double sum_all(double v, double* s_wave) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  __syncthreads();
  if (threadIdx.x % kWave == 0) s_wave[threadIdx.x / kWave] = v;
  __syncthreads();
  double r = 0.0;
  for (int i = 0; i < kSumThreads / kWave; ++i) r += s_wave[i];
  return r;
}

// Adds the workgroups' partials: S threads share an expert (S the power of
// two that fills the workgroup), each taking every S-th workgroup.
__global__ __launch_bounds__(kSumThreads) void router_loss_sum_kernel(
    const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
    const float* __restrict__ part_z, const int32_t* __restrict__ part_n, int blocks, int E, int k,
    int S, float balance_coef, float z_coef, int32_t* __restrict__ counts,
    int32_t* __restrict__ n_tokens, float* __restrict__ prob_mean, float* __restrict__ loss) {
  __shared__ double s_wave[kSumThreads / kWave];
  const int tid = threadIdx.x;
  double z = 0.0, nd = 0.0;
  for (int b = tid; b < blocks; b += kSumThreads) {
    z += part_z[b];
    nd += part_n[b];
  }
  z = sum_all(z, s_wave);
  nd = sum_all(nd, s_wave);   // an integer below 2^31: exact
  const int sub = tid % S;
  double bal = 0.0;
  for (int e0 = 0; e0 < E; e0 += kSumThreads / S) {
    const int e = e0 + tid / S;
    double p = 0.0;
    int32_t c = 0;
    if (e < E) {
      for (int b = sub; b < blocks; b += S) {
        p += part_p[static_cast<int64_t>(b) * E + e];
        c += part_c[static_cast<int64_t>(b) * E + e];
      }
    }
    for (int o = S / 2; o > 0; o >>= 1) {
      p += __shfl_xor(p, o, kWave);
      c += __shfl_xor(c, o, kWave);
    }
    if (e < E && sub == 0) {
      const double mean = nd > 0.0 ? p / nd : 0.0;
      counts[e] = c;
      prob_mean[e] = static_cast<float>(mean);
      bal += c * mean;
    }
  }
  bal = sum_all(bal, s_wave);
  if (tid == 0) {
    n_tokens[0] = static_cast<int32_t>(nd);
    loss[0] = nd > 0.0 ? static_cast<float>(balance_coef * E * bal / (k * nd)) : 0.0f;
    loss[1] = nd > 0.0 ? static_cast<float>(z_coef * z / nd) : 0.0f;
  }
}

template <int L, bool VEC>
__global__ __launch_bounds__(kThreads) void router_bwd_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx,
    const uint8_t* __restrict__ mask, const float* __restrict__ dprobs,
    const float* __restrict__ dloss, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ n_tokens, int T, int E, int k, float balance_coef, float z_coef,
    float* __restrict__ dlogits) {
  constexpr int kTok = kThreads / L;
  const int tid = threadIdx.x, g = tid % L;
  const double n = n_tokens ? *n_tokens : 0;
  float cb[kPer] = {}, cz = 0.0f;   // the balance term of v, and 2 c_z / n
  if (n > 0.0) {
    const double b = balance_coef * (dloss ? static_cast<double>(dloss[0]) : 1.0) * E / (k * n * n);
    cz = static_cast<float>(2.0 * z_coef * (dloss ? static_cast<double>(dloss[1]) : 1.0) / n);
    if (counts) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int e = expert_at<L, VEC>(g, i);
        if (e < E) cb[i] = static_cast<float>(b * counts[e]);
      }
    }
  }
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTok; t0 < T;
       t0 += static_cast<int64_t>(gridDim.x) * kTok) {
    const int64_t t = t0 + tid / L;
    if (t >= T) continue;   // whole groups: a token's lanes share t
    float p[kPer], lse = 0.0f;
    const bool any = token_softmax<L, VEC>(logits + t * E, E, g, p, lse);
    const bool kept = any && (!mask || mask[t]);
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = kept ? cb[i] : 0.0f;
    if (dprobs) {
      for (int s = 0; s < k; ++s) {
        const int32_t e = idx[t * k + s];
        const float d = dprobs[t * k + s];
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] += expert_at<L, VEC>(g, i) == e ? d : 0.0f;
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) dot += p[i] * v[i];
    dot = group_sum<L>(dot) - (kept ? cz * lse : 0.0f);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = any ? p[i] * (v[i] - dot) : 0.0f;
    float* out = dlogits + t * E;
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < kPer / 4; ++q)
        if (4 * (g + L * q) < E)
          reinterpret_cast<float4*>(out)[g + L * q] =
              float4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (g + L * i < E) out[g + L * i] = v[i];
    }
  }
}

// Lanes per token: at most kPer logits each.
int lanes_of(int E) { return E <= kPer ? 1 : E <= 4 * kPer ? 4 : E <= 16 * kPer ? 16 : 64; }

bool rows_vec(const void* p, int E) {
  return E % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

template <typename F>
void with_lanes(int E, bool vec, F&& f) {
  auto go = [&](auto l) {
    if (vec) f(l, std::true_type{}); else f(l, std::false_type{});
  };
  switch (lanes_of(E)) {
    case 1: go(std::integral_constant<int, 1>{}); break;
    case 4: go(std::integral_constant<int, 4>{}); break;
    case 16: go(std::integral_constant<int, 16>{}); break;
    default: go(std::integral_constant<int, 64>{}); break;
  }
}

}  // namespace

// Workgroups of the loss kernel: one per pass of tokens, at most 256 (their
// partials are what the second launch reads).
int router_loss_blocks(int T, int E) {
  const int tok = kThreads / lanes_of(E);
  const int64_t b = (static_cast<int64_t>(T) + tok - 1) / tok;
  return static_cast<int>(b < 1 ? 1 : b > 256 ? 256 : b);
}

hipError_t launch_router_loss(const moe_router_loss_args& a, hipStream_t s) {
  const int blocks = router_loss_blocks(a.T, a.E);
  float* part_z = static_cast<float*>(a.workspace);
  int32_t* part_n = reinterpret_cast<int32_t*>(part_z + blocks);
  float* part_p = reinterpret_cast<float*>(part_n + blocks);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + static_cast<int64_t>(blocks) * a.E);
  with_lanes(a.E, rows_vec(a.logits, a.E), [&](auto l, auto vec) {
    router_loss_kernel<decltype(l)::value, decltype(vec)::value><<<blocks, kThreads, 0, s>>>(
        a.logits, a.expert_idx, a.token_mask, a.T, a.E, a.k, part_p, part_c, part_z, part_n);
  });
  if (hipError_t e = hipGetLastError()) return e;
  int S = 1;
  while (S < 64 && 2 * S * a.E <= kSumThreads) S *= 2;
  router_loss_sum_kernel<<<1, kSumThreads, 0, s>>>(part_p, part_c, part_z, part_n, blocks, a.E, a.k,
                                                   S, a.balance_coef, a.z_coef, a.counts,
                                                   a.n_tokens, a.prob_mean, a.loss);
  return hipGetLastError();
}

hipError_t launch_router_bwd(const moe_router_bwd_args& a, hipStream_t s) {
  const int tok = kThreads / lanes_of(a.E);
  int64_t blocks = (static_cast<int64_t>(a.T) + tok - 1) / tok;
  if (blocks > 2048) blocks = 2048;
  const bool vec = rows_vec(a.logits, a.E) && rows_vec(a.dlogits, a.E);
  with_lanes(a.E, vec, [&](auto l, auto v) {
    router_bwd_kernel<decltype(l)::value, decltype(v)::value>
        <<<static_cast<int>(blocks), kThreads, 0, s>>>(
            a.logits, a.expert_idx, a.token_mask, a.dprobs, a.dloss, a.counts, a.n_tokens, a.T, a.E,
            a.k, a.balance_coef, a.z_coef, a.dlogits);
  });
  return hipGetLastError();
}

}  // namespace moe
