// The router's auxiliary losses, per-expert counts and the gradient with
// respect to its logits.
//
//   p = softmax(x);  lse = log sum exp x;  over the n tokens kept:
//   counts_e = picks of e;  P_e = (1/n) sum p_e
//   L = c_b E sum_e counts_e / (k n) P_e + c_z (1/n) sum lse^2
//   dx_j = p_j (v_j - sum_i p_i v_i + 2 c_z lse / n),
//   v_j = c_b E counts_j / (k n^2) + sum of dprobs over the slots that name j
//
// A token takes L lanes of a wave with P logits each (4, or 16 for more than 64
// experts), so the logits are read once and stay in registers; a wave covers
// 64 / L tokens.  Lane g of a token holds experts 4 (g + L i) + c (VEC:
// E % 4 == 0 and 16-byte aligned rows, one float4 each), else g + L i.  The loss
// kernel keeps each lane's sums of p over its tokens in registers, adds them
// over the workgroup in a fixed order and writes one partial per expert and
// workgroup; a second launch adds these, unless there is one workgroup only,
// which then does all of it.  Sums over tokens are fp64 throughout (a token's own
// sums over its experts fp32).
//
// Bound by latencies: a workgroup makes one or a few passes, so all it reads
// goes out at once, before the first use.  16384 tokens of 256 experts: 10.8 us
// for the partials (16.8 MB read; with fp32 sums and exponentials within two steps
// 8.8), 4.8 for their sums, 13.3 for the gradient (33.6 MB, 2.5 TB/s); 256 tokens
// of 4: 3.6 and 2.8 in one launch each.
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

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

constexpr float kNegInf = -__builtin_inff();

// The lane's logits of a token; those past E are -infinity (loads are made from
// a clamped place: one behind a condition is waited for before the next).
template <int L, int P, bool VEC>
MOE_DEV void token_load(const float* __restrict__ row, int E, int g, float (&p)[P]) {
  if constexpr (VEC) {
    const float4* r4 = reinterpret_cast<const float4*>(row);
#pragma unroll
    for (int q = 0; q < P / 4; ++q) {
      const float4 v = r4[min(g + L * q, E / 4 - 1)];
      p[4 * q] = v.x;
      p[4 * q + 1] = v.y;
      p[4 * q + 2] = v.z;
      p[4 * q + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = row[min(g + L * i, E - 1)];
  }
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (expert_at<L, VEC>(g, i) >= E) p[i] = kNegInf;
}

// The token's softmax in place of its logits, and lse; false if the logits are
// all -infinity.  Experts past E have p 0.
template <int L, int P>
MOE_DEV bool token_softmax(float (&p)[P], float& lse) {
  float m = kNegInf;
#pragma unroll
  for (int i = 0; i < P; ++i) m = fmaxf(m, p[i]);
  m = group_max<L>(m);
  // the maximum of NaN and a number is the number here; a token of NaN
  // alone keeps m at -infinity and is told from an empty one by its logits
  float nan = 0.0f;
  float z = 0.0f;
  const float mm = m == kNegInf ? 0.0f : m;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    p[i] = expf(p[i] - mm);
    z += p[i];
    nan = p[i] != p[i] ? 1.0f : nan;
  }
  z = group_sum<L>(z);
  if (m == kNegInf && group_max<L>(nan) == 0.0f) return false;
  const float inv = 1.0f / z;
#pragma unroll
  for (int i = 0; i < P; ++i) p[i] *= inv;
  lse = mm + logf(z);
  return true;
}

constexpr int kMaxLossBlocks = 256;   // workgroups of the loss kernel at most
constexpr int kLossThreads = 1024;
// threads of a single workgroup that covers all tokens in one pass: starting
// and joining 16 waves costs more than 4 (256 tokens of 4 experts, sums in fp32:
// 4.8 us with 16, 3.4 with 4)
constexpr int kFewThreads = 256;

// Sum over the workgroup's THREADS, in every thread.
template <int THREADS, typename T>
MOE_DEV T sum_all(T v, T* s_wave) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  __syncthreads();
  if (threadIdx.x % kWave == 0) s_wave[threadIdx.x / kWave] = v;
  __syncthreads();
  T r = 0;
#pragma unroll
  for (int i = 0; i < THREADS / kWave; ++i) r += s_wave[i];
  return r;
}

constexpr int kSumExperts = 16;   // experts of a workgroup of the second launch
__host__ __device__ constexpr int sum_blocks(int E) { return (E + kSumExperts - 1) / kSumExperts; }

// The workspace: the balance terms (fp64) and the count of the second launch's
// workgroups, then the loss kernel's partials: sums, then counts.
struct LossWs {
  double* terms;
  int32_t* done;
  double *part_z, *part_p;    // a workgroup's sum of lse^2; its sum of p per expert
  int32_t *part_n, *part_c;   // its tokens; its picks per expert
  MOE_DEV LossWs(void* p, int E, int blocks)
      : terms(static_cast<double*>(p)),
        done(reinterpret_cast<int32_t*>(terms + sum_blocks(E))),
        part_z(terms + sum_blocks(E) + 1),
        part_p(part_z + blocks),
        part_n(reinterpret_cast<int32_t*>(part_p + static_cast<int64_t>(blocks) * E)),
        part_c(part_n + blocks) {}
};

// (Arguments past about 104 bytes, a kernel's own and those that reading the
// grid's size adds, cost a launch 0.6 to 1 us of the host's time: hence one
// workspace pointer, and `blocks` by value.)
struct LossOut {
  float balance_coef, z_coef;
  int32_t *counts, *n_tokens;
  float *prob_mean, *loss;
  // over n tokens: bal = sum of counts * mean p, z = sum of lse^2
  MOE_DEV void write(int E, int k, double n, double bal, double z) const {
    n_tokens[0] = static_cast<int32_t>(n);
    loss[0] = n > 0.0 ? static_cast<float>(balance_coef * E * bal / (k * n)) : 0.0f;
    loss[1] = n > 0.0 ? static_cast<float>(z_coef * z / n) : 0.0f;
  }
};

// Partials of one workgroup: {sum of p, picks} per expert, {sum lse^2, n}.
template <int THREADS, int L, int P, bool VEC>
__global__ __launch_bounds__(THREADS) void router_loss_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx,
    const uint8_t* __restrict__ mask, int T, int E, int k, int blocks, void* ws, LossOut out) {
  constexpr int kWaves = THREADS / kWave, kTok = THREADS / L;   // tokens the workgroup covers at once
  constexpr int kOwnPicks = (kMaxTopK + L - 1) / L;
  __shared__ double s_p[kWaves * L * P];   // the waves' sums, expert-major: at most 128 KB
  __shared__ int32_t s_c[L * P];
  __shared__ double s_z[kWaves];
  __shared__ int32_t s_n[kWaves];
  __shared__ double s_wave[kWaves];
  const int tid = threadIdx.x, g = tid % L, wave = tid / kWave;
  for (int e = tid; e < E; e += THREADS) s_c[e] = 0;
  __syncthreads();
  double sum[P] = {};
  double zsum = 0.0;
  int32_t n = 0;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTok; t0 < T;
       t0 += static_cast<int64_t>(blocks) * kTok) {
    const int64_t t = t0 + tid / L;
    if (t >= T) continue;   // whole groups: a token's lanes share t
    float p[P], lse = 0.0f;
    int32_t pick[kOwnPicks];
    token_load<L, P, VEC>(logits + t * E, E, g, p);
#pragma unroll
    for (int s = 0; s < kOwnPicks; ++s) pick[s] = idx[t * k + min(g + s * L, k - 1)];
    const bool keep = !mask || mask[t];
    if (token_softmax<L, P>(p, lse) && keep) {
#pragma unroll
      for (int i = 0; i < P; ++i) sum[i] += p[i];
      if (g == 0) {
        zsum = __builtin_fma(static_cast<double>(lse), static_cast<double>(lse), zsum);
        ++n;
      }
#pragma unroll
      for (int s = 0; s < kOwnPicks; ++s)
        if (g + s * L < k && pick[s] >= 0 && pick[s] < E) atomicAdd(&s_c[pick[s]], 1);   // integers: any order
    }
  }
  // the lanes of a wave that hold the same experts (same g), then the waves
  // in their order
#pragma unroll
  for (int o = L; o < kWave; o <<= 1) {
#pragma unroll
    for (int i = 0; i < P; ++i) sum[i] += __shfl_xor(sum[i], o, kWave);
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
  if (tid % kWave < L) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = expert_at<L, VEC>(g, i);
      if (e < E) s_p[wave * L * P + e] = sum[i];
    }
  }
  __syncthreads();
  double z = 0.0;
  int32_t m = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    z += s_z[w];
    m += s_n[w];
  }
  static_assert(L * P <= THREADS, "an expert a thread");
  double v = 0.0;
  if (tid < E) {
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += s_p[w * L * P + tid];
  }
  if (blocks == 1) {   // these are the whole sums
    const double mean = m > 0 ? v / m : 0.0;
    if (tid < E) {
      out.counts[tid] = s_c[tid];
      out.prob_mean[tid] = static_cast<float>(mean);
    }
    const double bal = sum_all<THREADS>(tid < E ? s_c[tid] * mean : 0.0, s_wave);
    if (tid == 0) out.write(E, k, m, bal, z);
    return;
  }
  const LossWs w(ws, E, blocks);
  if (tid < E) {
    w.part_p[static_cast<int64_t>(blockIdx.x) * E + tid] = v;
    w.part_c[static_cast<int64_t>(blockIdx.x) * E + tid] = s_c[tid];
  }
  if (tid == 0) {
    w.part_z[blockIdx.x] = z;
    w.part_n[blockIdx.x] = m;
    if (blockIdx.x == 0) *w.done = 0;
  }
}

// Adds the workgroups' partials: 16 experts a workgroup, 16 threads each, all
// loads of a thread in flight.  The last workgroup to end adds the balance
// terms in their order; done was set to 0 by the first launch.
__global__ __launch_bounds__(kThreads) void router_loss_sum_kernel(void* ws, int blocks, int E, int k,
                                                                   LossOut out) {
  const LossWs w(ws, E, blocks);
  constexpr int kWaves = kThreads / kWave;
  __shared__ double s_z[kWaves];
  __shared__ int32_t s_n[kWaves];
  __shared__ double s_p[kThreads];
  __shared__ int32_t s_c[kThreads];
  constexpr int kRows = kThreads / kSumExperts, U = kMaxLossBlocks / kRows;
  const int tid = threadIdx.x, e = blockIdx.x * kSumExperts + tid % kSumExperts;
  // (loads from a clamped place, the value dropped after: a load behind a
  // condition is waited for before the next one, 9.8 us in all against 4.7)
  double vp[U];
  int32_t vc[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t at = static_cast<int64_t>(min(tid / kSumExperts + u * kRows, blocks - 1)) * E + min(e, E - 1);
    vp[u] = w.part_p[at];
    vc[u] = w.part_c[at];
  }
  static_assert(kMaxLossBlocks == kThreads, "one partial a thread");
  double z = w.part_z[min(tid, blocks - 1)];
  int32_t n = w.part_n[min(tid, blocks - 1)];
  if (tid >= blocks) z = 0.0, n = 0;
  double p = 0.0;
  int32_t c = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (tid / kSumExperts + u * kRows >= blocks || e >= E) vp[u] = 0.0, vc[u] = 0;
    p += vp[u];
    c += vc[u];
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    z += __shfl_xor(z, o, kWave);
    n += __shfl_xor(n, o, kWave);
  }
  s_p[tid] = p;
  s_c[tid] = c;
  if (tid % kWave == 0) {
    s_z[tid / kWave] = z;
    s_n[tid / kWave] = n;
  }
  __syncthreads();
  if (tid >= kWave) return;   // the first wave does the rest
  z = 0.0;
  n = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    z += s_z[i];
    n += s_n[i];
  }
  double bal = 0.0;
  if (tid < kSumExperts && e < E) {
    p = 0.0;
    c = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      p += s_p[i * kSumExperts + tid];
      c += s_c[i * kSumExperts + tid];
    }
    const double mean = n > 0 ? p / n : 0.0;
    out.counts[e] = c;
    out.prob_mean[e] = static_cast<float>(mean);
    bal = c * mean;
  }
#pragma unroll
  for (int o = kSumExperts / 2; o > 0; o >>= 1) bal += __shfl_xor(bal, o, kWave);
  int last = 0;
  if (tid == 0) {
    __hip_atomic_store(&w.terms[blockIdx.x], bal, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int before = __hip_atomic_fetch_add(w.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    last = before == sum_blocks(E) - 1;
  }
  if (!__shfl(last, 0, kWave)) return;
  static_assert(kMaxExperts / kSumExperts <= kWave, "a workgroup's term a lane");
  double all = tid < sum_blocks(E)
                   ? __hip_atomic_load(&w.terms[tid], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                   : 0.0;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) all += __shfl_xor(all, o, kWave);
  if (tid == 0) out.write(E, k, n, all, z);
}

template <int L, int P, bool VEC>
__global__ __launch_bounds__(kThreads) void router_bwd_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ idx,
    const uint8_t* __restrict__ mask, const float* __restrict__ dprobs,
    const float* __restrict__ dloss, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ n_tokens, int T, int E, int k, int blocks, float balance_coef,
    float z_coef, float* __restrict__ dlogits) {
  constexpr int kTok = kThreads / L;
  // the picks' gradients of a token, spread to the lanes of their experts
  // through LDS: comparing every logit with every pick costs three times the
  // rest of the kernel for 256 experts
  constexpr bool kSpread = L >= kMaxTopK;
  __shared__ __attribute__((aligned(16))) float s_d[kSpread ? kThreads * P : 4];
  const int tid = threadIdx.x, g = tid % L;
  float* row_d = s_d + (kSpread ? tid / L * L * P : 0);
  // what the loss terms take, read now and used when the first token is there
  const int32_t n_read = n_tokens ? *n_tokens : 0;
  const float dl0 = dloss ? dloss[0] : 1.0f, dl1 = dloss ? dloss[1] : 1.0f;
  int32_t count[P] = {};
  if (counts) {
#pragma unroll
    for (int i = 0; i < P; ++i) count[i] = counts[min(expert_at<L, VEC>(g, i), E - 1)];   // (past E its p is 0)
  }
  float cb[P] = {}, cz = 0.0f;   // the balance term of v, and 2 c_z / n
  bool ready = false;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTok; t0 < T;
       t0 += static_cast<int64_t>(blocks) * kTok) {
    const int64_t t = t0 + tid / L;
    if (t >= T) continue;   // whole groups: a token's lanes share t
    // the picks: one a lane, or all in every lane of a small group
    constexpr int kOwnPicks = L >= kMaxTopK ? 1 : kMaxTopK;
    int32_t pe[kOwnPicks];
    float pd[kOwnPicks] = {};
#pragma unroll
    for (int s = 0; s < kOwnPicks; ++s) {
      const int at = L >= kMaxTopK ? g : s;
      pe[s] = idx[t * k + min(at, k - 1)];
      if (at >= k || !dprobs) pe[s] = -1;
    }
    if (dprobs) {
#pragma unroll
      for (int s = 0; s < kOwnPicks; ++s) pd[s] = dprobs[t * k + min(L >= kMaxTopK ? g : s, k - 1)];
    }
    float p[P], lse = 0.0f;
    token_load<L, P, VEC>(logits + t * E, E, g, p);
    const bool keep = !mask || mask[t];
    const bool any = token_softmax<L, P>(p, lse);
    const bool kept = any && keep;
    if (!ready) {
      ready = true;
      if (n_read > 0) {
        const double n = n_read, b = balance_coef * static_cast<double>(dl0) * E / (k * n * n);
        cz = static_cast<float>(2.0 * z_coef * static_cast<double>(dl1) / n);
#pragma unroll
        for (int i = 0; i < P; ++i) cb[i] = static_cast<float>(b * count[i]);
      }
    }
    float v[P];
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = kept ? cb[i] : 0.0f;
    if (dprobs) {
      if constexpr (kSpread) {
        // lane s < k: the sum over the slots with its expert, written by the
        // first of them (one wave: LDS operations complete in order)
        float4* row4 = reinterpret_cast<float4*>(row_d);
#pragma unroll
        for (int q = 0; q < P / 4; ++q) row4[g + L * q] = float4{0.0f, 0.0f, 0.0f, 0.0f};
        float d = 0.0f;
        bool first = pe[0] >= 0 && pe[0] < E;
#pragma unroll
        for (int s = 0; s < kMaxTopK; ++s) {
          const int32_t e = __shfl(pe[0], s, L);
          const float ds = __shfl(pd[0], s, L);
          if (e == pe[0]) {
            d += ds;
            first = first && s >= g;
          }
        }
        asm volatile("" ::: "memory");
        if (first) row_d[pe[0]] = d;
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] += row_d[expert_at<L, VEC>(g, i)];
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
      } else {
#pragma unroll
        for (int s = 0; s < kMaxTopK; ++s) {
          if (s < k) {
#pragma unroll
            for (int i = 0; i < P; ++i)
              v[i] += expert_at<L, VEC>(g, i) == pe[s % kOwnPicks] ? pd[s % kOwnPicks] : 0.0f;
          }
        }
      }
    }
    // a token that is left out and has no gradient of its own gets zeros, whatever
    // its logits are: padding may hold NaN
    bool zero = !any;
    if (!keep) {
      float own = 0.0f;
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (expert_at<L, VEC>(g, i) < E && v[i] != 0.0f) own = 1.0f;   // (also for NaN)
      zero = zero || group_max<L>(own) == 0.0f;
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) dot += p[i] * v[i];
    dot = group_sum<L>(dot) - (kept ? cz * lse : 0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = zero ? 0.0f : p[i] * (v[i] - dot);
    float* out = dlogits + t * E;
    if constexpr (VEC) {
#pragma unroll
      for (int q = 0; q < P / 4; ++q)
        if (4 * (g + L * q) < E)
          reinterpret_cast<float4*>(out)[g + L * q] =
              float4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (g + L * i < E) out[g + L * i] = v[i];
    }
  }
}

// Lanes per token.
int lanes_of(int E) { return E <= 4 ? 1 : E <= 16 ? 4 : E <= 256 ? 16 : 64; }

bool rows_vec(const void* p, int E) {
  return E % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

template <typename F>
void with_lanes(int E, bool vec, F&& f) {
  auto go = [&](auto l, auto per) {
    if (vec) f(l, per, std::true_type{}); else f(l, per, std::false_type{});
  };
  std::integral_constant<int, 4> four;
  std::integral_constant<int, 16> sixteen;
  switch (lanes_of(E)) {
    case 1: go(std::integral_constant<int, 1>{}, four); break;
    case 4: go(four, four); break;
    case 16: if (E <= 64) go(sixteen, four); else go(sixteen, sixteen); break;
    default: go(std::integral_constant<int, 64>{}, sixteen); break;
  }
}

}  // namespace

// Workgroups of the loss kernel: one per pass of tokens, at most 256 (their
// partials are what the second launch reads).
static int loss_blocks(int T, int E) {
  const int tok = kLossThreads / lanes_of(E);
  const int64_t b = (static_cast<int64_t>(T) + tok - 1) / tok;
  return static_cast<int>(b < 1 ? 1 : b > kMaxLossBlocks ? kMaxLossBlocks : b);
}

size_t router_loss_workspace_bytes(int T, int E) {
  const size_t blocks = loss_blocks(T, E), parts = blocks + blocks * static_cast<size_t>(E);
  return 8 * (sum_blocks(E) + 1 + parts) + 4 * parts;
}

hipError_t launch_router_loss(const moe_router_loss_args& a, hipStream_t s) {
  const int blocks = loss_blocks(a.T, a.E);
  const LossOut out{a.balance_coef, a.z_coef, a.counts, a.n_tokens, a.prob_mean, a.loss};
  with_lanes(a.E, rows_vec(a.logits, a.E), [&](auto l, auto per, auto vec) {
    constexpr int kL = decltype(l)::value, kP = decltype(per)::value;
    auto go = [&](auto kernel, int threads) {
      kernel<<<blocks, threads, 0, s>>>(a.logits, a.expert_idx, a.token_mask, a.T, a.E, a.k, blocks,
                                        a.workspace, out);
    };
    if constexpr (kL * kP <= kFewThreads) {
      if (static_cast<int64_t>(a.T) * kL <= kFewThreads)
        return go(router_loss_kernel<kFewThreads, kL, kP, decltype(vec)::value>, kFewThreads);
    }
    go(router_loss_kernel<kLossThreads, kL, kP, decltype(vec)::value>, kLossThreads);
  });
  if (blocks == 1) return hipGetLastError();
  if (hipError_t e = hipGetLastError()) return e;
  router_loss_sum_kernel<<<sum_blocks(a.E), kThreads, 0, s>>>(a.workspace, blocks, a.E, a.k, out);
  return hipGetLastError();
}

hipError_t launch_router_bwd(const moe_router_bwd_args& a, hipStream_t s) {
  const int tok = kThreads / lanes_of(a.E);
  int64_t blocks = (static_cast<int64_t>(a.T) + tok - 1) / tok;
  if (blocks > 2048) blocks = 2048;
  const bool vec = rows_vec(a.logits, a.E) && rows_vec(a.dlogits, a.E);
  with_lanes(a.E, vec, [&](auto l, auto per, auto v) {
    router_bwd_kernel<decltype(l)::value, decltype(per)::value, decltype(v)::value>
        <<<static_cast<int>(blocks), kThreads, 0, s>>>(
            a.logits, a.expert_idx, a.token_mask, a.dprobs, a.dloss, a.counts, a.n_tokens, a.T, a.E,
            a.k, static_cast<int>(blocks), a.balance_coef, a.z_coef, a.dlogits);
  });
  return hipGetLastError();
}

}  // namespace moe
