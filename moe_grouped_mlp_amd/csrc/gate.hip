// The router's choice of experts by scores, its gradient, and the balance
// bias's update.
//
//   score = softmax(x) or 1 / (1 + e^-x);  choice = score + bias (or x)
//   a group's value = its largest choice or the sum of its two largest
//   picks = the k largest choices of the best groups;  w = scale * score / sum
//
// LPT lanes share a token.  Its experts go to them group by group: P = LPT /
// (groups rounded up to a power of two) lanes a group, each with W consecutive
// ids, all in registers (V is what the registers hold), so a token's logits are
// read once and an equal choice of a lower id is one of a lower lane or slot.
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kNoId = 0x7fffffff;

MOE_DEV float neg_inf() { return -__builtin_inff(); }
MOE_DEV double neg_inf64() { return -__builtin_inf(); }

template <typename T>
MOE_DEV float logit_of(T v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else return bf16_to_f32(v);
}

// Where a token's experts are: E experts in n_groups runs of Eg, P (a power of
// two) lanes a run, W ids a lane.
struct Layout {
  int E, Eg, n_groups, P, W;
  int vec;   // rows can be read four logits at a time
};
struct Place {
  int group, id0, n;   // the lane's run, its first id and how many it has
};
MOE_DEV Place place_of(const Layout& l, int lane) {
  Place p;
  p.group = lane / l.P;
  const int at = (lane - p.group * l.P) * l.W;
  p.id0 = p.group * l.Eg + at;
  p.n = p.group < l.n_groups && at < l.Eg ? (l.Eg - at < l.W ? l.Eg - at : l.W) : 0;
  return p;
}

// The lane's logits; slots without an expert and ruled-out ones are -infinity.
template <int V, typename T>
MOE_DEV void load_logits(const T* row, const Layout& l, const Place& p, bool live, float (&x)[V]) {
  if constexpr (V % 4 == 0) {
    if (l.vec) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const bool in = live && i < p.n;   // n is a multiple of 4 here
        if constexpr (std::is_same_v<T, float>) {
          const float4 f = in ? *reinterpret_cast<const float4*>(row + p.id0 + i)
                              : float4{neg_inf(), neg_inf(), neg_inf(), neg_inf()};
          x[i] = f.x;
          x[i + 1] = f.y;
          x[i + 2] = f.z;
          x[i + 3] = f.w;
        } else {
          const uint2 f = in ? *reinterpret_cast<const uint2*>(row + p.id0 + i) : uint2{0xff80ff80u, 0xff80ff80u};
          x[i] = __uint_as_float(f.x << 16);
          x[i + 1] = __uint_as_float(f.x & 0xffff0000u);
          x[i + 2] = __uint_as_float(f.y << 16);
          x[i + 3] = __uint_as_float(f.y & 0xffff0000u);
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = x[i] > neg_inf() ? x[i] : neg_inf();
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float f = live && i < p.n ? logit_of(row[p.id0 + i]) : neg_inf();
    x[i] = f > neg_inf() ? f : neg_inf();
  }
}

// Reductions over the LPT lanes of a token.
template <int LPT, typename T, typename F>
MOE_DEV T over_lanes(T v, F&& f) {
#pragma unroll
  for (int o = 1; o < LPT; o <<= 1) v = f(v, __shfl_xor(v, o, kWave));
  return v;
}
template <int LPT>
MOE_DEV float max_lanes(float v) {
  return over_lanes<LPT>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LPT, typename T>
MOE_DEV T sum_lanes(T v) {
  return over_lanes<LPT>(v, [](T a, T b) { return a + b; });
}

// x - m, 0 for the largest itself (an infinite one too).
MOE_DEV float below(float x, float m) { return x == m ? 0.0f : x - m; }

struct GateP {
  const void* logits;
  const float* bias;
  const uint8_t* mask;
  int32_t* idx;
  float* probs;
  int32_t* counts;
  int64_t ld;
  int T, k;
  float scale;
  Layout l;
  uint8_t sigmoid, top, stay, renorm;   // top: 0 without groups
};

// The k picks by 64-bit choices.  Every lane gets all of them (pick j with j
// its index in the token's lanes): id, or -1.
template <int LPT, int V>
MOE_DEV int picks64(const GateP& g, const Place& p, int lane, const float (&x)[V]) {
  double s[V];   // scores, then choices
  if (g.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = 1.0 / (1.0 + exp(-static_cast<double>(x[i])));
  } else {
    float m = neg_inf();
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, x[i]);
    m = max_lanes<LPT>(m);
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = x[i] > neg_inf() ? (x[i] == m ? 1.0 : exp(static_cast<double>(x[i]) - static_cast<double>(m))) : 0.0;
      z += s[i];
    }
    z = sum_lanes<LPT>(z);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] /= z;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    double c = s[i];
    if (g.bias) {
      const float b = i < p.n ? g.bias[p.id0 + i] : neg_inf();
      c += static_cast<double>(b);
      if (!(c > neg_inf64())) c = neg_inf64();
    }
    s[i] = x[i] > neg_inf() ? c : neg_inf64();
  }
  bool stays = true;
  if (g.top) {
    double a = neg_inf64(), b = neg_inf64();   // the two largest of the group
#pragma unroll
    for (int i = 0; i < V; ++i) {
      b = fmax(b, fmin(a, s[i]));
      a = fmax(a, s[i]);
    }
    for (int o = 1; o < g.l.P; o <<= 1) {
      const double a2 = __shfl_xor(a, o, kWave), b2 = __shfl_xor(b, o, kWave);
      b = fmax(fmin(a, a2), fmax(b, b2));
      a = fmax(a, a2);
    }
    if (g.top == 2 && b > neg_inf64()) a += b;
    int rank = 0;
    for (int o = 0; o < g.l.n_groups; ++o) {
      const double v = __shfl(a, (threadIdx.x & (kWave - 1) & ~(LPT - 1)) + o * g.l.P, kWave);
      rank += v > a || (v == a && o < p.group);
    }
    stays = rank < g.stay;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (!stays) s[i] = neg_inf64();
    else if (!g.bias && s[i] > neg_inf64()) s[i] = x[i];   // the logits decide
  }
  int mine = -1;
  for (int j = 0; j < g.k; ++j) {
    double v = neg_inf64();
    int id = kNoId;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (s[i] > v) {
        v = s[i];
        id = p.id0 + i;
      }
    }
#pragma unroll
    for (int o = 1; o < LPT; o <<= 1) {
      const double v2 = __shfl_xor(v, o, kWave);
      const int id2 = __shfl_xor(id, o, kWave);
      const bool take = v2 > v || (v2 == v && id2 < id);
      v = take ? v2 : v;
      id = take ? id2 : id;
    }
    if (lane == j) mine = id == kNoId ? -1 : id;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (p.id0 + i == id && i < p.n) s[i] = neg_inf64();
  }
  return mine;
}

// 1 / (1 + e^-x), which keeps its bits for large -x.
MOE_DEV float sigmoid_of(float x) {
  const float e = expf(-fabsf(x));
  return (x < 0.0f ? e : 1.0f) / (1.0f + e);
}

// The lane's weight share: its pick's score over the sum of the token's.  The
// scores of picks that are all small are taken times a factor that keeps the
// largest in range.
template <int LPT>
MOE_DEV float renormed(bool sigmoid, bool live, float x) {
  const float top = max_lanes<LPT>(live ? x : neg_inf());
  float s;
  if (!sigmoid) s = expf(below(x, top));
  else s = top < 0.0f ? expf(x - top) / (1.0f + expf(x)) : sigmoid_of(x);
  s = live ? s : 0.0f;
  const float z = sum_lanes<LPT>(s);
  return live ? s / z : 0.0f;
}

template <int LPT, int V, typename T>
__global__ __launch_bounds__(kThreads) void gate_kernel(const GateP g) {
  const int lane = threadIdx.x & (LPT - 1);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / LPT) + threadIdx.x / LPT;
  if (t >= g.T) return;   // whole tokens leave
  const T* row = static_cast<const T*>(g.logits) + t * g.ld;
  const Place p = place_of(g.l, lane);
  float x[V];
  load_logits<V>(row, g.l, p, !g.mask || g.mask[t] != 0, x);
  const int id = picks64<LPT, V>(g, p, lane, x);
  const bool live = id >= 0;
  const float xi = live ? logit_of(row[id]) : neg_inf();
  float w;
  if (g.renorm) {
    w = renormed<LPT>(g.sigmoid, live, xi);
  } else if (g.sigmoid) {
    w = sigmoid_of(xi);
  } else {
    float m = neg_inf();
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, x[i]);
    m = max_lanes<LPT>(m);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) z += expf(below(x[i], m));
    z = sum_lanes<LPT>(z);
    w = expf(below(xi, m)) / z;
  }
  if (lane < g.k) {
    g.idx[t * g.k + lane] = id;
    g.probs[t * g.k + lane] = live ? g.scale * w : 0.0f;
    if (live && g.counts) atomicAdd(g.counts + id, 1);
  }
}

struct GateBwdP {
  const void* logits;
  const int32_t* idx;
  const float* dprobs;
  void* dlogits;
  int64_t ld, ld_d;
  int T, E, k;
  float scale;
  Layout l;
  uint8_t sigmoid, renorm, accumulate, vec_d;
};

// Rows go out through LDS of their own, where the picks' terms are added to
// them.
template <int LPT, int V, typename T>
__global__ __launch_bounds__(kThreads) void gate_bwd_kernel(const GateBwdP g) {
  __shared__ __attribute__((aligned(16))) float s_row[kThreads * V];
  const int lane = threadIdx.x & (LPT - 1);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / LPT) + threadIdx.x / LPT;
  if (t >= g.T) return;
  float* own = s_row + threadIdx.x / LPT * (LPT * V);
  const T* row = static_cast<const T*>(g.logits) + t * g.ld;
  const Place p = place_of(g.l, lane);
  const bool full = !g.sigmoid && !g.renorm;   // every logit has a gradient
  int id = lane < g.k ? g.idx[t * g.k + lane] : -1;
  bool live = id >= 0 && id < g.E;
  float xi = live ? logit_of(row[id]) : neg_inf();
  live = live && xi > neg_inf();
  const float d = live ? g.scale * g.dprobs[t * g.k + lane] : 0.0f;
  float x[V];
  float term, dot = 0.0f;
  if (full) {
    load_logits<V>(row, g.l, p, true, x);
    float m = neg_inf();
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, x[i]);
    m = max_lanes<LPT>(m);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = x[i] > neg_inf() ? expf(below(x[i], m)) : 0.0f;
      z += x[i];
    }
    z = sum_lanes<LPT>(z);
    const float r = z > 0.0f ? 1.0f / z : 0.0f;
    term = live ? expf(below(xi, m)) * r * d : 0.0f;
    dot = sum_lanes<LPT>(term) * r;
  } else if (g.renorm) {
    const float w = renormed<LPT>(g.sigmoid, live, xi);
    const float mean = sum_lanes<LPT>(w * d);
    term = live ? w * (d - mean) : 0.0f;
    if (g.sigmoid) term *= sigmoid_of(-xi);
  } else {
    const float e = expf(-fabsf(xi));   // s (1 - s), either sign
    term = live ? d * (e / ((1.0f + e) * (1.0f + e))) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < p.n) own[p.id0 + i] = full ? -x[i] * dot : 0.0f;
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();   // LDS operations of one wave complete in order
  if (live) atomicAdd(own + id, term);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  T* out = static_cast<T*>(g.dlogits) + t * g.ld_d;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (i >= p.n) continue;
    float v = own[p.id0 + i];
    if (g.accumulate) v += logit_of(out[p.id0 + i]);
    if constexpr (std::is_same_v<T, float>) out[p.id0 + i] = v;
    else out[p.id0 + i] = static_cast<bf16_t>(pack_bf16x2(v, 0.0f));
  }
}

constexpr int kBiasThreads = 1024;
static_assert(kBiasThreads >= kMaxExperts, "a thread for every expert");
__global__ __launch_bounds__(kBiasThreads) void bias_update_kernel(int E, float rate, int reset, int32_t* counts, float* bias) {
  __shared__ int64_t s_sum[kBiasThreads / kWave];
  const int e = threadIdx.x;
  const int64_t n = e < E ? counts[e] : 0;
  int64_t total = n;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o, kWave);
  if ((e & (kWave - 1)) == 0) s_sum[e / kWave] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kBiasThreads / kWave; ++w) total += s_sum[w];
  if (e >= E) return;
  if (n * E != total) bias[e] += n * E < total ? rate : -rate;
  if (reset) counts[e] = 0;
}

int next_pow2(int v) {
  int p = 1;
  while (p < v) p <<= 1;
  return p;
}

// Lanes a token takes and logits a lane holds: the fewest that hold it.
struct Shape {
  int lanes, values;
};
constexpr Shape kShapes[] = {{8, 4}, {16, 4}, {16, 8}, {16, 16}, {64, 8}, {64, 16}, {64, 32}};
int shape_for(int E, int n_groups, Layout* l) {
  l->E = E;
  l->n_groups = n_groups;
  l->Eg = E / n_groups;
  const int g2 = next_pow2(n_groups);
  for (int i = 0; i < static_cast<int>(sizeof(kShapes) / sizeof(Shape)); ++i) {
    if (kShapes[i].lanes < g2) continue;
    l->P = kShapes[i].lanes / g2;
    l->W = ((l->Eg + l->P - 1) / l->P + 3) / 4 * 4;
    if (l->W <= kShapes[i].values) return i;
  }
  return -1;
}

bool can_vec(const Layout& l, const void* p, int64_t ld, int bytes) {
  return l.Eg % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * bytes) == 0;
}

template <typename F>
void with_shape(int i, F&& f) {
  switch (i) {
    case 0: f(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{}); break;
    case 1: f(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{}); break;
    case 2: f(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{}); break;
    case 3: f(std::integral_constant<int, 16>{}, std::integral_constant<int, 16>{}); break;
    case 4: f(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{}); break;
    case 5: f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{}); break;
    default: f(std::integral_constant<int, 64>{}, std::integral_constant<int, 32>{}); break;
  }
}

}  // namespace

hipError_t launch_router_gate(const moe_gate_args& a, hipStream_t s) {
  GateP g{};
  g.logits = a.logits;
  g.bias = a.bias;
  g.mask = a.token_mask;
  g.idx = a.expert_idx;
  g.probs = a.probs;
  g.counts = a.counts;
  g.ld = a.ld ? a.ld : a.E;
  g.T = a.T;
  g.k = a.k;
  g.scale = a.scale;
  g.sigmoid = a.score == MOE_SCORE_SIGMOID;
  const int groups = a.n_groups > 1 && a.topk_groups < a.n_groups ? a.n_groups : 1;   // all stay: no groups
  g.top = groups > 1 ? static_cast<uint8_t>(a.group_top) : 0;
  g.stay = groups > 1 ? static_cast<uint8_t>(a.topk_groups) : 1;
  g.renorm = a.renorm != 0;
  const int shape = shape_for(a.E, groups, &g.l);
  if (shape < 0) return hipErrorInvalidValue;   // (every E <= 1024 with up to 64 groups has one)
  const bool f32 = a.logits_type == MOE_TYPE_F32;
  g.l.vec = can_vec(g.l, a.logits, g.ld, f32 ? 4 : 2);
  with_shape(shape, [&](auto lpt, auto v) {
    constexpr int L = decltype(lpt)::value, V = decltype(v)::value;
    const int64_t blocks = (static_cast<int64_t>(a.T) * L + kThreads - 1) / kThreads;
    if (f32) gate_kernel<L, V, float><<<static_cast<uint32_t>(blocks), kThreads, 0, s>>>(g);
    else gate_kernel<L, V, bf16_t><<<static_cast<uint32_t>(blocks), kThreads, 0, s>>>(g);
  });
  return hipGetLastError();
}

hipError_t launch_router_gate_bwd(const moe_gate_bwd_args& a, hipStream_t s) {
  GateBwdP g{};
  g.logits = a.logits;
  g.idx = a.expert_idx;
  g.dprobs = a.dprobs;
  g.dlogits = a.dlogits;
  g.ld = a.ld ? a.ld : a.E;
  g.ld_d = a.ld_d ? a.ld_d : a.E;
  g.T = a.T;
  g.E = a.E;
  g.k = a.k;
  g.scale = a.scale;
  g.sigmoid = a.score == MOE_SCORE_SIGMOID;
  g.renorm = a.renorm != 0;
  g.accumulate = a.accumulate != 0;
  const int shape = shape_for(a.E, 1, &g.l);
  if (shape < 0) return hipErrorInvalidValue;
  const bool f32 = a.logits_type == MOE_TYPE_F32;
  g.l.vec = can_vec(g.l, a.logits, g.ld, f32 ? 4 : 2);
  g.vec_d = can_vec(g.l, a.dlogits, g.ld_d, f32 ? 4 : 2);
  with_shape(shape, [&](auto lpt, auto v) {
    constexpr int L = decltype(lpt)::value, V = decltype(v)::value;
    const int64_t blocks = (static_cast<int64_t>(a.T) * L + kThreads - 1) / kThreads;
    if (f32) gate_bwd_kernel<L, V, float><<<static_cast<uint32_t>(blocks), kThreads, 0, s>>>(g);
    else gate_bwd_kernel<L, V, bf16_t><<<static_cast<uint32_t>(blocks), kThreads, 0, s>>>(g);
  });
  return hipGetLastError();
}

hipError_t launch_bias_update(const moe_bias_update_args& a, hipStream_t s) {
  bias_update_kernel<<<1, kBiasThreads, 0, s>>>(a.E, a.rate, a.reset, a.counts, a.bias);
  return hipGetLastError();
}

}  // namespace moe
